"""A cache in 4 bits: rows of one call apart from one another, and the far ends of weights, gains and
roundings, against fp64 or bit by bit."""
import numpy as np
import pytest
import torch

import fp4_ref as f4
import long_context_mask_gb300 as bsa
import paged_ref as ref
from gpu_util import status_ok
from test_gpu_paged import bits, lists_for
from test_gpu_paged_fp4 import run_append, run_forward

pytestmark = pytest.mark.gpu
INF = float("inf")


# ------------------------------------------------------------------ row tiles without a key

@pytest.mark.parametrize("D,page", [(64, 64), (128, 128)])
def test_short_row_tiles_before_row_tiles_without_a_key(D, page):
    """A thread block's run of some 40 row tiles (a token each): again and again one of one or two key tiles, and
    eight or nine without any, by lists that are empty; and tokens before position 0."""
    H, n = 128, 152 * 40 + 5
    b = ref.make([n], [n], H=H, H_kv=1, D=D, page=page, seed=140)
    c = f4.Cache(b, 140)
    q = ref.rows(b, H, 141)
    t = torch.arange(n)
    own = t // 128
    sel = torch.stack([torch.zeros_like(own), own], 1)[:, None].to(torch.int32).contiguous().cuda()
    cnt = torch.where((t % 9 == 0) | (t % 90 == 4), torch.where(own > 0, 1 + t % 2, torch.ones_like(t)), torch.zeros_like(t))
    lists = [[[0, int(own[x])][:int(cnt[x])]] for x in range(n)]
    cnt = cnt[:, None].to(torch.int32).contiguous().cuda()
    first = None
    for _ in range(20):
        o, lse = run_forward(b, c, q, sel=sel, sel_cnt=cnt)
        status_ok()
        if first is None:
            first = o, lse
            f4.check_attention(b, q, o, lse, sel=lists)
        assert torch.equal(bits(o), bits(first[0])) and torch.equal(lse, first[1])
    short = torch.tensor([140], dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((n, H), device="cuda")
    bsa.forward_paged_fp4(q, *c.arrays(), b.table, b.q_start, short, o, lse)
    status_ok()
    assert (o[:n - 140] == 0).all() and torch.isneginf(lse[:n - 140]).all() and torch.isfinite(lse[n - 140:]).all()


@pytest.mark.parametrize("max_new", [0, 1])
@pytest.mark.parametrize("H,K,D", [(1, 1, 128), (2, 2, 64), (4, 1, 64), (12, 1, 128)])
def test_a_token_whose_scores_are_all_minus_infinity(H, K, D, max_new):
    """It is a row without a key, with no other row beside it too."""
    b = ref.make([1, 1], [700, 40], H=H, H_kv=K, D=D, page=64, seed=147)
    c = f4.Cache(b, 147)
    c.k = (c.k & 0x77) | 0x11
    raw = c.k_scale.view(torch.uint8)
    raw.copy_(torch.where(raw == 0, torch.full_like(raw, 0x20), raw))
    q = ref.rows(b, H, 148)
    q[..., 17] = -INF
    o, lse = run_forward(b, c, q, max_new=max_new)
    status_ok()
    assert (o == 0).all() and torch.isneginf(lse).all()


# ------------------------------------------------------------------ rows apart from one another

def rising(new, length, H, K, D, page, seed):
    """A batch whose scores grow along the keys, past every maximum again and again; values 16 and 17 of a key
    are positive, so that a query's infinity there makes scores of its sign alone."""
    b = ref.make(new, length, H=H, H_kv=K, D=D, page=page, seed=seed)
    c = f4.Cache(b, seed)
    raw = c.k_scale.view(torch.uint8)
    for s, n in enumerate(b.length):
        p = torch.arange(n, device="cuda")
        size = torch.exp2(6.0 * p / n - 5.0).to(torch.float8_e4m3fn).view(torch.uint8)
        raw[b.table[s].long()[p // page], :, p % page] = size[:, None, None]
    c.k[..., 8] = (c.k[..., 8] & 0x77) | 0x11
    return b, c.refresh()


def with_row(q, rows, value):
    """q with the given rows ([tokens, heads] truth values) not finite, or 64 times as large."""
    x = q.clone()
    if value is None:
        x[rows] *= 64
    else:
        x[..., 17] = torch.where(rows, torch.full_like(x[..., 17], value), x[..., 17])
    return x


def check_apart(b, c, q, bad, **kw):
    """No other row has other bits for what the bad rows hold."""
    o0, lse0 = run_forward(b, c, q, **kw)
    status_ok()
    for value in (None, float("nan"), INF, -INF):
        o, lse = run_forward(b, c, with_row(q, bad, value), **kw)
        status_ok()
        assert torch.equal(bits(o)[~bad], bits(o0)[~bad]) and torch.equal(lse[~bad], lse0[~bad]), value
        seen = bad & torch.isfinite(lse0)
        if value == -INF:
            assert (o[bad] == 0).all() and torch.isneginf(lse[bad]).all()
        elif value is not None:
            assert torch.isnan(o[seen].float()).all() and torch.isnan(lse[seen]).all()
    return o0, lse0


@pytest.mark.parametrize("new,H,K,D,page", [(1, 8, 2, 128, 64), (1, 8, 1, 64, 16), (1, 32, 2, 128, 128), (2, 8, 2, 64, 32)])
def test_rows_of_few_tokens_do_not_show_in_one_another(new, H, K, D, page):
    """Row tiles of 8 and of 16, some four to eight key tiles to a warp."""
    b, c = rising([new] * 12, [16000 + 700 * s for s in range(12)], H, K, D, page, 142)
    q = ref.rows(b, H, 143)
    bad = torch.zeros((b.tokens, H), dtype=torch.bool, device="cuda")
    bad[:, 1::H // K] = True
    o, lse = check_apart(b, c, q, bad, max_new=new)
    f4.check_attention(b, q, o, lse)


@pytest.mark.parametrize("kw", [{}, dict(window=900, sinks=300), dict(causal=False), "lists"])
@pytest.mark.parametrize("H,K,D,page", [(8, 2, 128, 64), (14, 2, 64, 16)])
def test_rows_of_many_tokens_do_not_show_in_one_another(H, K, D, page, kw):
    b, c = rising([200, 70], [5000, 3000], H, K, D, page, 144)
    q = ref.rows(b, H, 145)
    want = {}
    if kw == "lists":
        sel, cnt, listed = lists_for(b, np.random.default_rng(146), 12)
        kw, want = dict(sel=sel, sel_cnt=cnt), dict(sel=listed)
    bad = torch.zeros((b.tokens, H), dtype=torch.bool, device="cuda")
    bad[2::5, 1], bad[3::7, H - 1] = True, True
    o, lse = check_apart(b, c, q, bad, **kw)
    f4.check_attention(b, q, o, lse, **(want or kw))


# ------------------------------------------------------------------ gains and roundings

@pytest.mark.parametrize("new,heads", [(1, 4), (1, 12), (40, 4)])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 128)])
def test_the_smallest_and_largest_gains_of_attention(D, page, new, heads):
    """A long row of even weights, out of one page that the table names again and again: O is the mean
    value, a normal number with any gain.  The bound is test_the_longest_sequence_out_of_one_page's (of fewer additions)."""
    b = ref.make([new], [page], H=2 * heads, H_kv=2, D=D, page=page, seed=151, poison=False)
    c = f4.Cache(b, 151)
    c.v &= 0x77
    c.v_scale.copy_(torch.full(c.v_scale.shape, 128.0).to(torch.float8_e4m3fn))
    c.v_gain = torch.tensor([2.0 ** -126, 2.0 ** 117], device="cuda")
    c.refresh()
    q = torch.zeros((new, 2 * heads, D), dtype=torch.bfloat16, device="cuda")
    copies = (29 << 16) // page   # (a sum whose reciprocal is no power of two)
    table = b.table[:, :1].expand(1, copies).contiguous()
    o, lse = torch.empty_like(q), torch.empty((new, 2 * heads), device="cuda")
    bsa.forward_paged_fp4(q, *c.arrays(), table, b.q_start, torch.tensor([29 << 16], dtype=torch.int32, device="cuda"), o, lse,
                          causal=False, max_new=new, **c.gains())
    status_ok()
    O = b.v_cache[b.table[0, 0].long()].double().mean(1).repeat_interleave(heads, 0)  # [2 * heads, D]
    assert ((o.double() - O).abs() <= (2.0 ** -8 * 1.01 + 2.0 ** -11 + 2.0 ** -11 + 2.0 ** -12) * O.abs()).all()
    assert ((lse.double() - np.log(29 << 16)).abs() <= 2.0 ** -12 + 8 * 2.0 ** -24 * 15).all()


# ------------------------------------------------------------------ weights far below a row's largest

@pytest.mark.parametrize("even", [False, True])
@pytest.mark.parametrize("nats", [12, 15, 17])
@pytest.mark.parametrize("new", [1, 3, 40])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
def test_small_weights_beside_a_sink(D, page, new, nats, even):
    """The first key takes nearly all of the weight and has a value of 0: O is what the others leave, of many weights or
    (even) of one.

    fp4_ref.check_attention's bound with its last term as small as it has to be: a weight is rounded where its row's
    largest is at least 2^6, so what fp16's smallest step 2^-24 takes is at most 2^-25 / 2^6 of that."""
    b = ref.make([new, new], [8192, 30 if new < 30 else 60], H=4, H_kv=1, D=D, page=page, seed=149)
    c = f4.Cache(b, 149)
    c.v &= 0x77
    c.k[..., :8] = 0                                # values 0 .. 15 are the sink's alone
    per = 16 * 6 * D ** -0.5                        # nats to a scale of 1 there, against queries of 1
    size = torch.tensor(nats / per).to(torch.float8_e4m3fn)
    for s in range(2):
        at = b.table[s, 0].long()
        c.k[at, :, 0], c.v[at, :, 0] = 0, 0
        c.k[at, :, 0, :8] = 0x77
        c.k_scale[at, :, 0, 0] = size
    c.refresh()
    q = ref.rows(b, 4, 150)
    q[..., :16] = 1
    if even:
        q[..., 16:] = 0
    for kw in (dict(max_new=0), dict(max_new=new)):
        o, lse = run_forward(b, c, q, **kw)
        status_ok()
        O, L, A, R = ref.attend(b, q)
        assert float((L - size.double().item() * per).amax()) < 0.2  # (the sink has the weight)
        d = (D + 16) * 2.0 ** -24 * (R + 1)
        bound = 2.0 ** -8 * 1.01 * O.abs() + (2.0 ** -11 * 1.01 + 2 * d[..., None]) * A + 2.0 ** -31 * f4.visible(b)
        err = (o.double() - O).abs()
        assert (err <= bound).all(), f"{float((err / bound).max()):.2f} of the bound"


def nearest_bf16(x):
    """fp64 numbers whose nearest bf16 is a normal one, rounded to it once, halves to even."""
    i = x.contiguous().view(torch.int64)
    i = i + ((1 << 44) - 1) + (i >> 45 & 1)
    return (i & ~((1 << 45) - 1)).view(torch.float64)


def test_reading_back_rounds_once():
    """Every level under every scale, times 4096 gains: the bf16 number nearest to the product.  Among them 0.625 times
    0x1.78ccccp-4, whose nearest fp32 number lies halfway between two of bf16's."""
    K = 4096
    b = ref.make([32], [32], H=K, H_kv=K, D=64, page=16, seed=152, poison=False)
    c = f4.Cache(b, 152)
    order = b.pages_of(0)
    c.k[:] = torch.tensor([i | (i + 1) << 4 for i in range(0, 16, 2)], dtype=torch.uint8, device="cuda").repeat(4)
    scale = torch.arange(128, dtype=torch.uint8, device="cuda").clamp(1, 126).reshape(2, 1, 16, 4).expand(2, K, 16, 4)
    c.k_scale.view(torch.uint8)[order] = scale
    g = torch.Generator().manual_seed(153)
    c.k_gain = (torch.rand(K, generator=g) + 0.5).cuda()
    c.k_gain[7] = float.fromhex("0x1.78ccccp-4")
    c.refresh()
    out = torch.empty((32, K, 64), dtype=torch.bfloat16, device="cuda")
    bsa.paged_read_fp4(*c.arrays(), *b.arrays(), out, **c.gains())
    status_ok()
    held = b.k_cache[order].double().permute(0, 2, 1, 3).reshape(32, K, 64)
    # (levels, scales and gains are multiples in fp64 without a rounding: 6 + 24 bits)
    off = out.double() != nearest_bf16(held)
    assert not off.any(), f"{int(off.sum())} of {off.numel()} values are not the nearest"
    half = (held[:, 7] == 0.625 * c.k_gain[7].double()).nonzero()
    assert len(half) and float(out[half[0, 0], 7, half[0, 1]]) == 0.057373046875


def test_mean_keys_with_large_and_small_gains():
    """Sums of 128 keys that 32 bits cannot hold, or hold with few bits only, where the means are normal numbers."""
    b = ref.make([256], [256], H=4, H_kv=4, D=64, page=32, seed=154, poison=False)
    c = f4.Cache(b, 154)
    c.k_gain = torch.tensor([2.0 ** -126, 1.0, 2.0 ** 120, 2.0 ** 124], device="cuda")
    k = ((ref.rows(b, 4, 155).double().abs() + 8) * c.k_gain.double()[:, None]).to(torch.bfloat16)
    _, k_mean = run_append(b, c, None, k, k)
    status_ok()
    c.refresh()
    for j in range(2):
        pages = b.table[0, 4 * j:4 * j + 4].long()
        keys = b.k_cache[pages]
        mean, size = keys.mean((0, 2)), keys.abs().mean((0, 2))
        # (as in check_append)
        assert ((k_mean[pages[-1]].double() - mean).abs() <= 2.0 ** -8 * mean.abs() * 1.01 + 2.0 ** -16 * size).all()


def test_finite_numbers_beyond_the_range_are_no_error():
    """However far: a quotient by the gain that 32 bits cannot hold is a magnitude beyond 2688 gains as any other."""
    b = ref.make([3], [3], H=2, H_kv=2, D=64, page=16, seed=156, poison=False)
    c = f4.Cache(b, 156)
    c.k_gain = torch.tensor([2.0 ** -66, 2.0 ** -126], device="cuda")
    c.v_gain = c.k_gain.flip(0).contiguous()
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    x[0, :, 5], x[0, :, 6], x[2, :, 40] = 1e30, 2.0 ** -60, -3e38
    bsa.paged_append_fp4(x, x, *c.arrays(), *b.arrays(), **c.gains())
    status_ok()
    c.refresh()
    for cache, gain in ((b.k_cache, c.k_gain), (b.v_cache, c.v_gain)):
        for h in range(2):
            got = b.keys(0, h, cache) / gain[h].double()
            want = torch.zeros_like(got)
            want[0, 5], want[2, 40] = 2688.0, -2688.0
            want[0, 6] = 2688.0 if gain[h] == 2.0 ** -126 else 0.0   # (2^66 gains, 64 gains under a scale of 448)
            assert torch.equal(got, want)
    x[1, 1, 9] = INF
    bsa.paged_append_fp4(x, x, *c.arrays(), *b.arrays(), **c.gains())
    assert bsa.device_status() == 7
