"""A paged cache in 4 bits: append, reading back and attention against fp64,
element by element, with bounds that count the roundings (see fp4_ref)."""
import numpy as np
import pytest
import torch

import fp4_ref as f4
import long_context_mask_gb300 as bsa
import paged_ref as ref
from gpu_util import status_ok
from test_gpu_paged import LENS, bits, lists_for

pytestmark = pytest.mark.gpu
BOUNDS, OVERFLOW, NONFINITE = 6, 3, 7


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def raw(x):
    return x.view(torch.uint8)


def same_bytes(a, b):
    return all(torch.equal(raw(x), raw(y)) for x, y in zip(a, b))


# ------------------------------------------------------------------ append

def run_append(b, c, q, k, v, means=True, **kw):
    q_out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda") if q is not None else None
    k_mean = torch.full((b.n_pages, b.H_kv, b.D), 7.0, dtype=torch.bfloat16, device="cuda") if means else None
    bsa.paged_append_fp4(k, v, *c.arrays(), *b.arrays(), q=q, q_out=q_out, k_mean=k_mean, **c.gains(), **kw)
    return q_out, k_mean


def check_append(b, c, q, k, v, before, q_out, k_mean, rope=None, interleaved=False, q_norm=None, k_norm=None, eps=1e-6):
    starts = b.q_start.tolist()
    slots = torch.zeros((b.n_pages, b.page), dtype=torch.bool, device="cuda")
    filled = {}
    kg, vg = c.k_gain, c.v_gain
    for s, (n, length) in enumerate(zip(b.new, b.length)):
        if n == 0:
            continue
        pos = torch.arange(length - n, length, device="cuda")
        t = slice(starts[s], starts[s] + n)
        page, at = b.table[s].long()[pos // b.page], pos % b.page
        y, size = ref.turned(q[t], pos, rope, interleaved, q_norm, eps)
        bound = 2.0 ** -8 * y.abs() * 1.01 + ((b.D + 8) / 2 * (q_norm is not None) + 4) * 2.0 ** -24 * size
        assert ((q_out[t].double() - y).abs() <= bound).all()
        # keys: the norm's factor is rounded once and two products follow (3 half steps), the
        # rotation's two products and sum
        y, size = ref.turned(k[t], pos, rope, interleaved, k_norm, eps)
        err = ((4 * (k_norm is not None)) + 3 * (rope is not None)) * 2.0 ** -24 * size
        f4.check_quantised(y, err, c.k[page, :, at], raw(c.k_scale)[page, :, at], kg)
        f4.check_quantised(v[t].double(), 0 * v[t].double(), c.v[page, :, at], raw(c.v_scale)[page, :, at], vg)
        slots[page, at] = True
        for j in range((length - n) // 128, length // 128):
            which = b.table[s, j * 128 // b.page:(j + 1) * 128 // b.page].long()
            filled[int(which[-1])] = which
    for now, was in zip(c.arrays(), before):
        assert torch.equal(raw(now).transpose(1, 2)[~slots], raw(was).transpose(1, 2)[~slots])
    outside = torch.ones(b.tokens, dtype=torch.bool, device="cuda")
    outside[starts[0]:starts[-1]] = False
    assert (q_out[outside] == 7.0).all()
    c.refresh()
    if k_mean is not None:
        for page in range(b.n_pages):
            if page not in filled:
                assert (k_mean[page] == 7.0).all()
                continue
            keys = b.k_cache[filled[page]]
            mean, size = keys.mean((0, 2)), keys.abs().mean((0, 2))
            # 128 additions in fp32, the gain, one rounding to bf16
            assert ((k_mean[page].double() - mean).abs() <= 2.0 ** -8 * mean.abs() * 1.01 + 2.0 ** -16 * size).all()


@pytest.mark.parametrize("gains", [False, True])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("H,K,D,page,rot,inter,norm", [
    (4, 2, 128, 16, 128, False, False), (4, 2, 128, 128, 128, False, True), (14, 2, 64, 32, 32, True, False),
    (3, 3, 64, 64, 48, False, True), (8, 1, 128, 16, 64, True, True), (6, 2, 128, 64, 0, False, False),
    (2, 2, 64, 128, 64, False, True), (2, 2, 64, 16, 16, False, True)])
def test_append(lens, H, K, D, page, rot, inter, norm, gains):
    b = ref.make(*LENS[lens], H=H, H_kv=K, D=D, page=page, seed=1, pad_tokens=3, first=2, poison=False)
    c = f4.Cache(b, 1, gains=gains, dirty=False)
    q, k, v = ref.rows(b, H, 2), f4.random_rows(b, K, 3), f4.random_rows(b, K, 4)
    kw = dict(rope=ref.rope_table(1000, rot) if rot else None, interleaved=inter)
    if norm:
        g = torch.Generator().manual_seed(5)
        kw.update(q_norm=torch.randn(D, generator=g).to(torch.bfloat16).cuda(),
                  k_norm=torch.randn(D, generator=g).to(torch.bfloat16).cuda(), eps=1e-5)
    before = c.clone()
    q_out, k_mean = run_append(b, c, q, k, v, **kw)
    status_ok()
    check_append(b, c, q, k, v, before, q_out, k_mean, **kw)


def test_every_half_goes_to_the_even_level():
    """Each level and each middle between two, under scales of every size (bf16 holds them exactly)."""
    steps = [0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0]
    to = [0.0, 0.0, 0.5, 1.0, 1.0, 1.0, 1.5, 2.0, 2.0, 2.0, 3.0, 4.0, 4.0, 4.0, 6.0]
    scales = f4.e4m3(torch.arange(1, 127))
    n = len(scales)
    for D in (64, 128):
        b = ref.make([n], [n], H=1, H_kv=1, D=D, page=16, seed=2, poison=False)
        c = f4.Cache(b, 2)
        x = torch.tensor([*steps[:14], 6.0, -0.25] * (D // 16), dtype=torch.float64)
        want = torch.tensor([*to[:14], 6.0, 0.0] * (D // 16), dtype=torch.float64)
        sign = torch.where(torch.arange(D) % 3 == 0, -1.0, 1.0).double()
        sign[15::16] = 1.0
        rows = (x * sign)[None] * scales[:, None]
        kv = rows.to(torch.bfloat16)[:, None].cuda()
        assert torch.equal(kv.double().cpu()[:, 0], rows)
        bsa.paged_append_fp4(kv, kv, *c.arrays(), *b.arrays())
        status_ok()
        c.refresh()
        assert torch.equal(b.keys(0, 0).cpu(), (want * sign)[None] * scales[:, None])
        assert torch.equal(b.keys(0, 0, b.v_cache).cpu(), (want * sign)[None] * scales[:, None])


def test_what_four_bits_cannot_hold():
    """Beyond the range: the largest; not finite: the largest or 0, and told; too small: 0."""
    b = ref.make([6], [6], H=1, H_kv=1, D=64, page=16, seed=3, poison=False)
    c = f4.Cache(b, 3)
    x = torch.zeros((6, 1, 64), dtype=torch.bfloat16, device="cuda")
    x[0, 0, 3], x[0, 0, 4] = 1e30, -1.0                 # beyond 2688
    x[1, 0, 20], x[1, 0, 21] = 2.0 ** -13, -2.0 ** -14  # max / 6 below half the smallest scale
    x[2] = 1e-38
    bsa.paged_append_fp4(x, x, *c.arrays(), *b.arrays())
    status_ok()
    got = b.keys(0, 0, c.refresh().b.v_cache)
    assert got[0, 3] == 2688.0 and got[0, 4] == 0.0 and (got[1:] == 0).all()
    one = 6 * 0.171875  # a group of ones: e4m3(1 / 6) is 11 / 64, between 10 / 64 and 11 / 64 (10.67 / 64), and 1 / (11 / 64) > 5
    for bad, want in ((float("inf"), 2688.0), (-float("inf"), -2688.0), (float("nan"), 0.0)):
        for which in (0, 1):
            y = torch.ones_like(x)
            y[4, 0, 40] = bad
            kv = (y, torch.ones_like(x)) if which == 0 else (torch.ones_like(x), y)
            bsa.paged_append_fp4(*kv, *c.arrays(), *b.arrays())
            assert bsa.device_status() == NONFINITE
            c.refresh()
            got = b.keys(0, 0, b.k_cache if which == 0 else b.v_cache)
            assert got[4, 40] == want and (got[:4] == one).all() and (got[4, :32] == one).all() and torch.isfinite(got).all()


def test_append_of_views_and_in_place():
    b = ref.make([5, 200], [40, 200], H=6, H_kv=2, D=128, page=32, seed=3, poison=False)
    c, c2 = f4.Cache(b, 4), f4.Cache(b, 4)
    qkv = ref.rows(b, 10, 6)
    rope = ref.rope_table(256, 128)
    before = c.clone()
    q, k, v = qkv[:, :6], qkv[:, 6:8], qkv[:, 8:]
    q_out, k_mean = run_append(b, c, q, k, v, rope=rope)
    check_append(b, c, q, k, v, before, q_out, k_mean, rope=rope)
    whole = qkv.clone()
    bsa.paged_append_fp4(whole[:, 6:8], whole[:, 8:], *c2.arrays(), *b.arrays(), q=whole[:, :6], q_out=whole[:, :6],
                         rope=rope)                                        # rotated where it stands, no means
    status_ok()
    assert torch.equal(bits(whole[:, :6].contiguous()), bits(q_out)) and torch.equal(whole[:, 6:], qkv[:, 6:])
    assert same_bytes(c.arrays(), c2.arrays())
    # the queries that the append into bf16 pages gives
    pages = [torch.zeros((b.n_pages, 2, 32, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    other = torch.empty_like(q_out)
    bsa.paged_append(k, v, *pages, *b.arrays(), q=q, q_out=other, rope=rope)
    assert torch.equal(bits(other), bits(q_out))


def test_append_chunks_leave_the_same_bytes():
    """300 tokens at once, and as 1, 126, 1, 2, 128, 42."""
    b = ref.make([300], [300], H=4, H_kv=2, D=128, page=16, seed=7, poison=False)
    c, c2 = f4.Cache(b, 5, gains=True), f4.Cache(b, 5, gains=True)
    q, k, v = ref.rows(b, 4, 8), ref.rows(b, 2, 9), ref.rows(b, 2, 10)
    norm = (1 + 0.1 * torch.randn(128, generator=torch.Generator().manual_seed(1))).to(torch.bfloat16).cuda()
    kw = dict(rope=ref.rope_table(300, 128), q_norm=norm, k_norm=norm)
    q_out, k_mean = run_append(b, c, q, k, v, **kw)
    mean2, q2, at = torch.full_like(k_mean, 7.0), torch.empty_like(q_out), 0
    for n in (1, 126, 1, 2, 128, 42):
        t = slice(at, at + n)
        bsa.paged_append_fp4(k[t], v[t], *c2.arrays(), b.table, i32([0, n]), i32([at + n]), q=q[t], q_out=q2[t],
                             k_mean=mean2, **c2.gains(), **kw)
        at += n
    status_ok()
    assert same_bytes(c.arrays(), c2.arrays()) and torch.equal(bits(q2), bits(q_out))
    assert torch.equal(bits(mean2), bits(k_mean))


def test_append_reports_and_leaves_out_what_makes_no_sense():
    b = ref.make([2, 2, 2], [40, 50, 60], H=2, H_kv=1, D=64, page=32, seed=11, poison=False)
    q, k, v = ref.rows(b, 2, 1), ref.rows(b, 1, 2), ref.rows(b, 1, 3)

    def go(table=None, q_start=None, kv_len=None):
        c = f4.Cache(b, 6)
        before = c.clone()
        bsa.paged_append_fp4(k, v, *c.arrays(), b.table if table is None else table,
                             b.q_start if q_start is None else i32(q_start), b.kv_len if kv_len is None else i32(kv_len))
        return bsa.device_status(), [raw(x) != raw(y) for x, y in zip(c.arrays(), before)]

    good = go()
    assert good[0] == 0
    for page in (-1, b.n_pages, 1 << 30):
        table = b.table.clone()
        table[1, 1] = page
        st, changed = go(table=table)
        assert st == BOUNDS
        for x, y in zip(changed, good[1]):
            assert torch.equal(x[b.table[0, :2].long()], y[b.table[0, :2].long()]) and not (x & ~y).any()
            assert not x[b.table[1, 1].long()].any()
    for bad in ([40, -1, 60], [40, 65, 60], [40, 1, 60]):
        st, changed = go(kv_len=bad)
        assert st == BOUNDS and all(torch.equal(x[b.table[2, :2].long()], y[b.table[2, :2].long()]) for x, y in zip(changed, good[1]))
    for bad in ([0, 2, -5, 2], [0, 2, 7, 2], [2, 1, 3, 6], [0, 6, 0, 6]):
        assert go(q_start=bad)[0] == BOUNDS


# ------------------------------------------------------------------ reading back

@pytest.mark.parametrize("gains", [False, True])
@pytest.mark.parametrize("H,K,D,page", [(4, 2, 128, 16), (2, 2, 64, 32), (8, 1, 128, 128), (40, 40, 128, 64), (3, 3, 64, 16)])
def test_read(H, K, D, page, gains):
    b = ref.make([0, 3, 128, 1, 257, 64, 65], [50, 131, 256, 384, 300, 64, 1000], H=H, H_kv=K, D=D, page=page, seed=8, first=2,
                 pad_tokens=3)
    c = f4.Cache(b, 8, gains=gains)
    k = torch.full((b.tokens, K, D), 7.0, dtype=torch.bfloat16, device="cuda")
    both = torch.full((b.tokens, 2 * K + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    bsa.paged_read_fp4(*c.arrays(), *b.arrays(), k, both[:, :K], **c.gains())
    bsa.paged_read_fp4(*c.arrays(), *b.arrays(), None, both[:, K:2 * K], **c.gains())
    only = torch.full_like(k, 7.0)
    bsa.paged_read_fp4(*c.arrays(), *b.arrays(), only, **c.gains())
    status_ok()
    starts = b.q_start.tolist()
    live = torch.zeros(b.tokens, dtype=torch.bool, device="cuda")
    for s, (n, length) in enumerate(zip(b.new, b.length)):
        t = slice(starts[s], starts[s] + n)
        live[t] = True
        for h in range(K):
            for got, cache in ((k, b.k_cache), (both, b.v_cache)):
                want = b.keys(s, h, cache)[length - n:]
                # (level * scale is exact; the gain's product and its rounding)
                x = want.float().to(torch.bfloat16).double() if not gains else want
                err = (got[t, h].double() - x).abs()
                assert (err <= (2.0 ** -8 * 1.01 * x.abs() if gains else 0 * x)).all()
    assert (k[~live] == 7.0).all() and (both[~live] == 7.0).all() and (both[:, 2 * K] == 7.0).all()
    assert torch.equal(bits(both[:, K:2 * K].contiguous()), bits(both[:, :K].contiguous())) and torch.equal(bits(only), bits(k))


def test_read_of_all_codes_and_scales():
    """All 16 codes under all 256 bytes of a scale."""
    b = ref.make([256], [256], H=1, H_kv=1, D=64, page=64, seed=9, poison=False)
    c = f4.Cache(b, 9)
    order = b.pages_of(0)
    row = torch.tensor([i | (i + 1) << 4 for i in range(0, 16, 2)], dtype=torch.uint8, device="cuda").repeat(4)
    c.k[:] = row
    raw(c.k_scale)[order] = torch.arange(256, dtype=torch.uint8, device="cuda").reshape(4, 1, 64, 1).expand(4, 1, 64, 4)
    c.refresh()
    out = torch.empty((256, 1, 64), dtype=torch.bfloat16, device="cuda")
    bsa.paged_read_fp4(*c.arrays(), *b.arrays(), out)
    status_ok()
    assert torch.equal(out[:, 0].double(), b.keys(0, 0))


def test_read_of_any_range_and_shared_pages():
    """Two requests for the same sequence's tokens: 100 .. 199 and 0 .. 149."""
    b = ref.make([300], [300], H=2, H_kv=2, D=128, page=32, seed=10)
    c = f4.Cache(b, 10)
    out = torch.empty((250, 2, 128), dtype=torch.bfloat16, device="cuda")
    bsa.paged_read_fp4(*c.arrays(), b.table.expand(2, -1).contiguous(), i32([0, 100, 250]), i32([200, 150]), None, out)
    status_ok()
    for h in range(2):
        v = b.keys(0, h, b.v_cache)
        assert torch.equal(out[:100, h].double(), v[100:200]) and torch.equal(out[100:, h].double(), v[:150])


def test_read_reports_what_makes_no_sense():
    b = ref.make([2, 2, 2], [40, 50, 60], H=1, H_kv=1, D=64, page=32, seed=11)
    c = f4.Cache(b, 11)

    def go(table=b.table, q_start=b.q_start, kv_len=b.kv_len):
        out = torch.full((6, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        bsa.paged_read_fp4(*c.arrays(), table, q_start, kv_len, out)
        return bsa.device_status(), out

    good = go()[1]
    table = b.table.clone()
    table[1, 1] = b.n_pages
    st, out = go(table=table)
    assert st == BOUNDS and (out[2:4] == 7.0).all() and torch.equal(out[:2], good[:2]) and torch.equal(out[4:], good[4:])
    for bad in ([40, -1, 60], [40, 65, 60]):
        st, out = go(kv_len=i32(bad))
        assert st == BOUNDS and (out[2:4] == 7.0).all() and torch.equal(out[4:], good[4:])
    st, out = go(kv_len=i32([40, 1, 60]))          # two tokens asked for, one there
    assert st == BOUNDS and (out[2] == 7.0).all() and torch.equal(out[4:], good[4:])
    assert torch.equal(out[3, 0].double(), f4.held(c.k, c.k_scale)[b.table[1, 0].long(), 0, 0])
    for bad in ([0, 2, -5, 2], [0, 2, 7, 2], [2, 1, 3, 6], [0, 6, 0, 6]):
        assert go(q_start=i32(bad))[0] == BOUNDS


# ------------------------------------------------------------------ attention

SHAPES = [(4, 2, 128, 16), (8, 8, 64, 128), (14, 2, 64, 16), (32, 8, 128, 64), (16, 1, 128, 32), (5, 1, 64, 64),
          (128, 1, 128, 128), (40, 2, 128, 16)]
ATT = dict(one=([1], [1]), step=([1] * 7, [1, 15, 16, 17, 128, 129, 1000]), prompt=([300], [300]),
           mixed=([0, 3, 129, 1, 257, 64, 2], [50, 131, 256, 3000, 300, 64, 2]))


def run_forward(b, c, q, **kw):
    o = torch.full((b.tokens, b.H, b.D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.tokens, b.H), 7.0, device="cuda")
    bsa.forward_paged_fp4(q, *c.arrays(), *b.arrays(), o, lse, **c.gains(), **kw)
    return o, lse


def untouched(b, o, lse):
    out = torch.ones(b.tokens, dtype=torch.bool, device="cuda")
    out[b.q_start[0].item():b.q_start[-1].item()] = False
    return bool((o[out] == 7.0).all() and (lse[out] == 7.0).all())


@pytest.mark.parametrize("gains", [False, True])
@pytest.mark.parametrize("lens", ATT)
@pytest.mark.parametrize("H,K,D,page", SHAPES)
def test_attention(lens, H, K, D, page, gains):
    b = ref.make(*ATT[lens], H=H, H_kv=K, D=D, page=page, seed=21, first=2, pad_tokens=3)
    c = f4.Cache(b, 21, gains=gains)
    q = ref.rows(b, H, 22)
    o, lse = run_forward(b, c, q, max_new=max(b.new) if gains else 0)
    status_ok()
    f4.check_attention(b, q, o, lse)
    assert untouched(b, o, lse)


@pytest.mark.parametrize("causal,window,sinks", [(False, 0, 0), (True, 100, 0), (True, 200, 40), (True, 1, 0),
                                                 (False, 100, 5), (True, 128, 300), (True, 1 << 30, 4)])
@pytest.mark.parametrize("H,K,D,page", SHAPES[:4])
def test_masks(causal, window, sinks, H, K, D, page):
    b = ref.make([1, 40, 0, 150, 3], [700, 1040, 30, 2000, 3], H=H, H_kv=K, D=D, page=page, seed=23, first=1, pad_tokens=1)
    c = f4.Cache(b, 23, gains=True)
    q = ref.rows(b, H, 24)
    o, lse = run_forward(b, c, q, causal=causal, window=window, sinks=sinks)
    status_ok()
    f4.check_attention(b, q, o, lse, causal=causal, window=window, sinks=sinks)
    assert untouched(b, o, lse)


@pytest.mark.parametrize("max_new", [0, 1, 2, 3, 4, 1000])
def test_the_hint_does_not_matter(max_new):
    """Sequences with more and with fewer new tokens than told."""
    b = ref.make([1, 3, 90, 2], [500, 1000, 700, 2], H=8, H_kv=2, D=128, page=32, seed=25)
    c = f4.Cache(b, 25)
    q = ref.rows(b, 8, 26)
    o, lse = run_forward(b, c, q, max_new=max_new)
    status_ok()
    f4.check_attention(b, q, o, lse)


def test_rows_without_a_key():
    """New tokens before position 0, empty sequences, lists that are empty: 0 and -inf."""
    b = ref.make([5, 4], [5, 4], H=4, H_kv=2, D=128, page=16, seed=27)
    c = f4.Cache(b, 27)
    q = ref.rows(b, 4, 28)
    o = torch.full((9, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((9, 4), 7.0, device="cuda")
    bsa.forward_paged_fp4(q, *c.arrays(), b.table, b.q_start, i32([2, 0]), o, lse)
    status_ok()
    assert (o[:3] == 0).all() and torch.isneginf(lse[:3]).all() and (o[5:] == 0).all() and torch.isneginf(lse[5:]).all()
    sel = torch.zeros((9, 2, 3), dtype=torch.int32, device="cuda")
    cnt = torch.zeros((9, 2), dtype=torch.int32, device="cuda")
    bsa.forward_paged_fp4(q, *c.arrays(), *b.arrays(), o, lse, sel=sel, sel_cnt=cnt)
    status_ok()
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_scale_and_large_scores():
    b = ref.make([1, 90], [2000, 700], H=4, H_kv=2, D=64, page=32, seed=29)
    c = f4.Cache(b, 29)
    q = ref.rows(b, 4, 30)
    for scale in (0.02, 1.0, 7.0):
        o, lse = run_forward(b, c, q, scale=scale)
        status_ok()
        f4.check_attention(b, q, o, lse, scale=scale)


@pytest.mark.parametrize("e", [-126, -60, -20, 20, 60, 100])
def test_queries_of_any_size(e):
    """Rows of 2^e, of mixed sizes, and of zeros (the scale takes 2^e out again)."""
    b = ref.make([1, 30], [300, 200], H=4, H_kv=2, D=128, page=64, seed=31)
    c = f4.Cache(b, 31)
    q = ref.rows(b, 4, 32)
    q[2, 1] = 0
    q[3, 2, 5:] *= 2.0 ** -18
    big = (q.double() * 2.0 ** e).to(torch.bfloat16)
    scale = 0.1 * 2.0 ** -e
    o, lse = run_forward(b, c, big, scale=scale)
    status_ok()
    f4.check_attention(b, big, o, lse, scale=scale)


def test_rising_scores_raise_the_maximum():
    """Keys that matter more and more: scores that pass the maximum so far by a little and by a lot."""
    b = ref.make([1, 40], [1500, 900], H=2, H_kv=1, D=64, page=16, seed=33)
    c = f4.Cache(b, 33)
    for s in range(2):
        for p in range(b.length[s]):
            v = min(448.0, 2.0 ** (p / 100 - 6))
            c.k_scale[b.table[s, p // 16].long(), :, p % 16] = torch.tensor(v).to(torch.float8_e4m3fn)
    c.refresh()
    q = ref.rows(b, 2, 34)
    o, lse = run_forward(b, c, q)
    status_ok()
    f4.check_attention(b, q, o, lse)


def test_queries_may_be_views():
    b = ref.make([4, 60], [400, 600], H=8, H_kv=2, D=128, page=64, seed=35)
    c = f4.Cache(b, 35)
    qkv = ref.rows(b, 12, 36)
    o, lse = run_forward(b, c, qkv[:, :8])
    o2, lse2 = run_forward(b, c, qkv[:, :8].contiguous())
    status_ok()
    assert torch.equal(bits(o), bits(o2)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("seed", range(6))
def test_random_batches(seed):
    g = np.random.default_rng(200 + seed)
    H, K = [(4, 2), (7, 1), (12, 12), (40, 8), (24, 4), (96, 1)][seed]
    n = int(g.integers(1, 60))
    new = [int(x) for x in g.integers(0, 90, n)]
    length = [int(a + g.integers(0, 900)) for a in new]
    b = ref.make(new, length, H=H, H_kv=K, D=int(g.choice([64, 128])), page=int(g.choice([16, 32, 64, 128])), seed=seed)
    if b.tokens == 0:
        return
    c = f4.Cache(b, seed)
    q = ref.rows(b, H, seed)
    o, lse = run_forward(b, c, q)
    status_ok()
    f4.check_attention(b, q, o, lse)


def test_many_sequences():
    """More sequences than threads of a block, most of them without new tokens."""
    g = np.random.default_rng(9)
    new = [int(x) for x in (g.random(3000) < 0.2) * g.integers(1, 3, 3000)]
    length = [int(a + g.integers(0, 40)) for a in new]
    b = ref.make(new, length, H=2, H_kv=1, D=64, page=16, seed=31)
    c = f4.Cache(b, 37)
    q = ref.rows(b, 2, 32)
    o, lse = run_forward(b, c, q)
    status_ok()
    f4.check_attention(b, q, o, lse)


def test_a_query_that_is_not_finite_stays_alone():
    b = ref.make([70, 3], [500, 300], H=8, H_kv=2, D=128, page=64, seed=40)
    c = f4.Cache(b, 40)
    q = ref.rows(b, 8, 41)
    o0, lse0 = run_forward(b, c, q)
    q[11, 3, 7], q[40, 0, 0] = float("nan"), float("inf")
    o, lse = run_forward(b, c, q)
    status_ok()
    same = torch.ones(b.tokens, 8, dtype=torch.bool, device="cuda")
    same[11, 3] = same[40, 0] = False
    assert torch.equal(bits(o)[same], bits(o0)[same]) and torch.equal(lse[same], lse0[same])
    assert torch.isnan(o[~same].float()).all()


def test_the_same_call_gives_the_same_bits():
    b = ref.make([1, 1, 130], [15000, 7000, 4000], H=8, H_kv=2, D=128, page=64, seed=33)
    c = f4.Cache(b, 42)
    q = ref.rows(b, 8, 34)
    first = run_forward(b, c, q)
    f4.check_attention(b, q, *first)
    for _ in range(5):
        again = run_forward(b, c, q)
        assert torch.equal(bits(first[0]), bits(again[0])) and torch.equal(first[1], again[1])
    status_ok()


def test_attention_reports_what_makes_no_sense():
    b = ref.make([2, 2, 2], [40, 50, 60], H=2, H_kv=1, D=64, page=32, seed=35, poison=False)
    c = f4.Cache(b, 43)
    q = ref.rows(b, 2, 36)
    good = run_forward(b, c, q)

    def go(table=b.table, q_start=b.q_start, kv_len=b.kv_len):
        o = torch.full((b.tokens, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((b.tokens, 2), 7.0, device="cuda")
        bsa.forward_paged_fp4(q, *c.arrays(), table, q_start, kv_len, o, lse)
        return bsa.device_status(), o

    for page in (-1, b.n_pages, 1 << 30):
        table = b.table.clone()
        table[1, 1] = page
        st, o = go(table=table)
        assert st == BOUNDS
        assert torch.equal(bits(o[:2]), bits(good[0][:2])) and torch.equal(bits(o[4:]), bits(good[0][4:]))
    for bad in ([40, -1, 60], [40, 65, 60]):
        st, o = go(kv_len=i32(bad))
        assert st == BOUNDS and (o[2:4] == 7.0).all() and torch.equal(bits(o[:2]), bits(good[0][:2]))
    for bad in ([0, 2, -5, 2], [0, 2, 7, 2], [2, 1, 3, 6], [0, 6, 0, 6]):
        assert go(q_start=i32(bad))[0] == BOUNDS


# ------------------------------------------------------------------ lists

@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,K,D,page", SHAPES)
def test_attention_over_lists(H, K, D, page, causal):
    b = ref.make([1, 40, 0, 150, 3], [700, 1040, 30, 2000, 3], H=H, H_kv=K, D=D, page=page, seed=41, first=1, pad_tokens=2)
    c = f4.Cache(b, 44, gains=True)
    q = ref.rows(b, H, 42)
    sel, cnt, want = lists_for(b, np.random.default_rng(43), 5, empty=0.1)
    o, lse = run_forward(b, c, q, sel=sel, sel_cnt=cnt, causal=causal)
    status_ok()
    f4.check_attention(b, q, o, lse, sel=want, causal=causal)
    assert untouched(b, o, lse)


def test_lists_report_what_makes_no_sense():
    b = ref.make([2, 3], [300, 500], H=4, H_kv=2, D=128, page=64, seed=46)
    c = f4.Cache(b, 45)
    q = ref.rows(b, 4, 47)
    sel, cnt, want = lists_for(b, np.random.default_rng(48), 3)
    for (t, h, e, x) in ((0, 0, 0, 3), (0, 0, 0, -1), (4, 1, 0, 1 << 30)):
        s2, c2, w2 = sel.clone(), cnt.clone(), [[list(y) for y in z] for z in want]
        s2[t, h, e] = x
        c2[t, h] = max(int(cnt[t, h]), 1)
        rest = s2[t, h, 1:int(c2[t, h])].tolist()
        w2[t][h] = sorted(set(rest))
        o, lse = run_forward(b, c, q, sel=s2, sel_cnt=c2)
        assert bsa.device_status() == BOUNDS
        f4.check_attention(b, q, o, lse, sel=w2)
    c2 = cnt.clone()
    c2[1, 1] = 4
    run_forward(b, c, q, sel=sel.clamp(min=0), sel_cnt=c2)
    assert bsa.device_status() == OVERFLOW
    c2[1, 1] = -1
    run_forward(b, c, q, sel=sel.clamp(min=0), sel_cnt=c2)
    assert bsa.device_status() == BOUNDS


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("D,page", [(128, 16), (64, 128)])
def test_a_conversation(D, page):
    """Prompts, then tokens one by one: append, choose blocks, attend over all and over the
    chosen ones, read back; against fp64 over what the cache holds."""
    H, K, steps, prompts = 8, 2, 5, [300, 127, 1]
    b = ref.make(prompts, [n + steps for n in prompts], H=H, H_kv=K, D=D, page=page, seed=51, poison=False)
    c = f4.Cache(b, 51, gains=True)
    k_mean = torch.zeros((b.n_pages, K, D), dtype=torch.bfloat16, device="cuda")
    rope = ref.rope_table(1000, D)
    lengths = list(prompts)
    for step in range(steps + 1):
        new = prompts if step == 0 else [1] * 3
        if step:
            lengths = [n + 1 for n in lengths]
        b.new, b.length, b.tokens = list(new), list(lengths), sum(new)
        b.q_start, b.kv_len = i32(np.cumsum([0, *new]).tolist()), i32(lengths)
        qkv = ref.rows(b, H + 2 * K, 60 + step)
        q = torch.empty((b.tokens, H, D), dtype=torch.bfloat16, device="cuda")
        bsa.paged_append_fp4(qkv[:, H:H + K], qkv[:, H + K:], *c.arrays(), *b.arrays(), q=qkv[:, :H], q_out=q, rope=rope,
                             k_mean=k_mean, **c.gains())
        c.refresh()
        o, lse = run_forward(b, c, q, max_new=max(new))
        sel = torch.empty((b.tokens, K, 3), dtype=torch.int32, device="cuda")
        cnt = torch.empty((b.tokens, K), dtype=torch.int32, device="cuda")
        bsa.select_paged(q, k_mean, *b.arrays(), sel, cnt, page_size=page, topk=1)
        o2, lse2 = run_forward(b, c, q, sel=sel, sel_cnt=cnt)
        back = torch.empty((b.tokens, K, D), dtype=torch.bfloat16, device="cuda")
        bsa.paged_read_fp4(*c.arrays(), *b.arrays(), None, back, **c.gains())
        status_ok()
        f4.check_attention(b, q, o, lse)
        lists = [[sel[t, h, :int(cnt[t, h])].tolist() for h in range(K)] for t in range(b.tokens)]
        assert lists == ref.select(b, q, k_mean, 1, 1, 1)
        f4.check_attention(b, q, o2, lse2, sel=lists)
        for s, t in enumerate(b.q_start.tolist()[:-1]):
            for h in range(K):
                want = b.keys(s, h, b.v_cache)[b.length[s] - new[s]:]
                assert ((back[t:t + new[s], h].double() - want).abs() <= 2.0 ** -8 * 1.01 * want.abs()).all()


def test_captured_and_replayed_as_the_sequences_grow():
    """One graph of append, attention and reading back, replayed while the lengths in device memory grow;
    the same again outside of a graph, on another stream and with scratch of its own."""
    H, K, D = 8, 2, 128
    b = ref.make([1, 1], [700, 140], H=H, H_kv=K, D=D, page=32, seed=53, max_pages=24, poison=False)
    b.table = i32(np.random.default_rng(1).permutation(48).reshape(2, 24).tolist())
    b.n_pages = 48
    c, c2 = f4.Cache(b, 53), f4.Cache(b, 53)
    qkv = ref.rows(b, H + 2 * K, 54)
    rope = ref.rope_table(1000, D)
    ws = torch.empty(bsa.forward_paged_fp4_workspace_size(2, 2, 24, 32, H, K, D), dtype=torch.uint8, device="cuda")

    def step(cache, **kw):
        q = torch.empty((2, H, D), dtype=torch.bfloat16, device="cuda")
        o, lse = torch.empty_like(q), torch.empty((2, H), device="cuda")
        back = torch.empty((2, K, D), dtype=torch.bfloat16, device="cuda")
        stream = {k: v for k, v in kw.items() if k == "stream"}
        bsa.paged_append_fp4(qkv[:, H:H + K], qkv[:, H + K:], *cache.arrays(), *b.arrays(), q=qkv[:, :H], q_out=q, rope=rope,
                             **stream)
        bsa.forward_paged_fp4(q, *cache.arrays(), *b.arrays(), o, lse, max_new=1, **kw)
        bsa.paged_read_fp4(*cache.arrays(), *b.arrays(), back, **stream)
        return o, lse, back

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(c, workspace=ws)
    for x, y in zip(c.arrays(), c2.arrays()):
        raw(x).copy_(raw(y))
    for i in range(4):
        b.kv_len.copy_(i32([700 + i, 140 + i]))
        qkv.copy_(ref.rows(b, H + 2 * K, 55 + i))
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.default_stream()):
            other = torch.cuda.Stream()
            other.wait_stream(torch.cuda.current_stream())
            want = step(c2, stream=other)
            torch.cuda.synchronize()
        status_ok()
        assert all(torch.equal(x, y) for x, y in zip(out, want))
        assert same_bytes(c.arrays(), c2.arrays())


def test_caches_beyond_32_bits():
    """Codes of more than 2^32 bytes: rows at the far end."""
    K, D, page, pages = 8, 128, 128, 72000      # 4.7 GB of codes each
    free = torch.cuda.mem_get_info()[0]
    if free < 40 << 30:
        pytest.skip("memory")
    shape = (pages, K, page)
    k, v = (torch.zeros((*shape, 64), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((*shape, 8), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    b = ref.make([200, 1], [300, 150], H=8, H_kv=K, D=D, page=page, seed=57, poison=False)
    far = torch.tensor([pages - 1 - i for i in range(b.n_pages)], device="cuda")
    b.table = torch.where(b.table >= 0, far[b.table.clamp(min=0).long()].to(torch.int32), b.table).contiguous()
    whole = ref.make([300, 150], [300, 150], H=8, H_kv=K, D=D, page=page, seed=57, poison=False)
    rows = ref.rows(whole, 2 * K, 59)
    bsa.paged_append_fp4(rows[:, :K], rows[:, K:], k, ks, v, vs, b.table, whole.q_start, b.kv_len)
    q = ref.rows(b, 8, 60)
    o = torch.empty((b.tokens, 8, D), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((b.tokens, 8), device="cuda")
    bsa.forward_paged_fp4(q, k, ks, v, vs, *b.arrays(), o, lse)
    out = torch.empty((b.tokens, K, D), dtype=torch.bfloat16, device="cuda")
    bsa.paged_read_fp4(k, ks, v, vs, *b.arrays(), out)
    status_ok()
    first = pages - b.n_pages
    b.k_cache, b.v_cache = f4.held(k[first:], ks[first:]), f4.held(v[first:], vs[first:])
    b.table = torch.where(b.table >= 0, b.table - first, b.table)
    f4.check_attention(b, q, o, lse)
    for h in range(K):
        assert torch.equal(out[:200, h].double(), b.keys(0, h)[100:])
        f4.check_quantised(rows[:300, h].double(), 0 * rows[:300, h].double(), k[first:][b.pages_of(0), h].reshape(-1, 64)[:300],
                           raw(ks)[first:][b.pages_of(0), h].reshape(-1, 8)[:300])
