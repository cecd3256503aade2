"""Paged cache: append, attention and block selection against fp64, element by
element, with bounds that count the roundings (see paged_ref)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import long_context_mask_gb300 as bsa
import paged_ref as ref
from gpu_util import status_ok

pytestmark = pytest.mark.gpu
BOUNDS, OVERFLOW = 6, 3


def bits(t):
    return t.view(torch.int16)


# ------------------------------------------------------------------ append

def run_append(b, q, k, v, means=True, **kw):
    q_out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=b.device)
    k_mean = torch.full((b.n_pages, b.H_kv, b.D), 7.0, dtype=torch.bfloat16, device=b.device) if means else None
    bsa.paged_append(k, v, b.k_cache, b.v_cache, *b.arrays(), q=q, q_out=q_out, k_mean=k_mean, **kw)
    return q_out, k_mean


def check_append(b, q, k, v, before_k, before_v, q_out, k_mean, rope=None, interleaved=False, q_norm=None,
                 k_norm=None, eps=1e-6):
    starts = b.q_start.tolist()
    want_v, slots, filled = before_v.clone(), torch.zeros_like(before_k, dtype=torch.bool), {}
    for s, (n, length) in enumerate(zip(b.new, b.length)):
        pos = torch.arange(length - n, length, device=b.device)
        t = slice(starts[s], starts[s] + n)
        page, at = b.table[s].long()[pos // b.page], pos % b.page
        for got, x, w in ((q_out[t], q[t], q_norm), (b.k_cache[page, :, at], k[t], k_norm)):
            y, size = ref.turned(x, pos, rope, interleaved, w, eps)
            # one rounding to bf16, and fp32: the norm's sum of D squares, root, quotient
            # and products (D + 8) / 2 steps, the rotation's two products and sum
            bound = 2.0 ** -8 * y.abs() * 1.01 + ((b.D + 8) / 2 * (w is not None) + 4) * 2.0 ** -24 * size
            if w is None and rope is None:
                bound = torch.zeros_like(bound)
            assert ((got.double() - y).abs() <= bound).all()
        want_v[page, :, at] = v[t]
        slots[page, :, at] = True
        for j in range((length - n) // 128, length // 128):
            which = b.table[s, j * 128 // b.page:(j + 1) * 128 // b.page].long()
            filled[int(which[-1])] = which
    assert torch.equal(bits(b.v_cache), bits(want_v))
    assert torch.equal(bits(b.k_cache)[~slots], bits(before_k)[~slots])
    outside = torch.ones(b.tokens, dtype=torch.bool, device=b.device)
    outside[starts[0]:starts[-1]] = False
    assert (q_out[outside] == 7.0).all()
    if k_mean is not None:
        for page in range(b.n_pages):
            if page not in filled:
                assert (k_mean[page] == 7.0).all()
                continue
            keys = b.k_cache[filled[page]].double()
            mean, size = keys.mean((0, 2)) * 1.0, keys.abs().mean((0, 2))
            # 128 additions in fp32, one rounding
            assert ((k_mean[page].double() - mean).abs() <= 2.0 ** -8 * mean.abs() * 1.01 + 2.0 ** -17 * size).all()


LENS = dict(one=([1], [1]), step=([1] * 5, [1, 127, 128, 129, 1000]), prompt=([300], [300]),
            chunks=([0, 3, 128, 1, 257, 64], [50, 131, 256, 384, 300, 64]))


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("H,K,D,page,rot,inter,norm", [
    (4, 2, 128, 16, 128, False, False), (4, 2, 128, 128, 128, False, True), (14, 2, 64, 32, 32, True, False),
    (3, 3, 64, 64, 48, False, True), (8, 1, 128, 16, 64, True, True), (6, 2, 128, 64, 0, False, False),
    (2, 2, 64, 128, 16, False, True)])
def test_append(lens, H, K, D, page, rot, inter, norm):
    b = ref.make(*LENS[lens], H=H, H_kv=K, D=D, page=page, seed=1, pad_tokens=3, first=2, poison=False)
    q, k, v = ref.rows(b, H, 2), ref.rows(b, K, 3), ref.rows(b, K, 4)
    kw = dict(rope=ref.rope_table(1000, rot) if rot else None, interleaved=inter)
    if norm:
        g = torch.Generator().manual_seed(5)
        kw.update(q_norm=torch.randn(D, generator=g).to(torch.bfloat16).cuda(),
                  k_norm=torch.randn(D, generator=g).to(torch.bfloat16).cuda(), eps=1e-5)
    bk, bv = b.k_cache.clone(), b.v_cache.clone()
    q_out, k_mean = run_append(b, q, k, v, **kw)
    status_ok()
    check_append(b, q, k, v, bk, bv, q_out, k_mean, **kw)


def test_append_of_views_and_in_place():
    b = ref.make([5, 200], [40, 200], H=6, H_kv=2, D=128, page=32, seed=3, poison=False)
    qkv = ref.rows(b, 10, 6)
    rope = ref.rope_table(256, 128)
    bk, bv = b.k_cache.clone(), b.v_cache.clone()
    q, k, v = qkv[:, :6], qkv[:, 6:8], qkv[:, 8:]
    q_out, k_mean = run_append(b, q, k, v, rope=rope)
    check_append(b, q, k, v, bk, bv, q_out, k_mean, rope=rope)
    k1, v1 = b.k_cache.clone(), b.v_cache.clone()
    whole = qkv.clone()
    bsa.paged_append(whole[:, 6:8], whole[:, 8:], b.k_cache, b.v_cache, *b.arrays(), q=whole[:, :6],
                     q_out=whole[:, :6], rope=rope)                         # rotated where it stands, no means
    status_ok()
    assert torch.equal(bits(whole[:, :6]), bits(q_out)) and torch.equal(whole[:, 6:], qkv[:, 6:])
    assert torch.equal(bits(b.k_cache), bits(k1)) and torch.equal(bits(b.v_cache), bits(v1))
    bsa.paged_append(k, v, b.k_cache, b.v_cache, *b.arrays(), rope=rope)    # no queries
    assert torch.equal(bits(b.k_cache), bits(k1))


def test_append_chunks_leave_the_same_bits():
    """300 tokens at once, and as 1, 126, 1, 2, 128, 42."""
    b = ref.make([300], [300], H=4, H_kv=2, D=128, page=16, seed=7, poison=False)
    q, k, v = ref.rows(b, 4, 8), ref.rows(b, 2, 9), ref.rows(b, 2, 10)
    rope = ref.rope_table(300, 128)
    q_out, k_mean = run_append(b, q, k, v, rope=rope)
    kc, vc = b.k_cache.clone(), b.v_cache.clone()
    b.k_cache.zero_()
    b.v_cache.zero_()
    mean2, q2, at = torch.full_like(k_mean, 7.0), torch.empty_like(q_out), 0
    for n in (1, 126, 1, 2, 128, 42):
        start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        length = torch.tensor([at + n], dtype=torch.int32, device="cuda")
        t = slice(at, at + n)
        bsa.paged_append(k[t], v[t], b.k_cache, b.v_cache, b.table, start, length, q=q[t], q_out=q2[t], rope=rope,
                         k_mean=mean2)
        at += n
    status_ok()
    used = b.table[0].long()
    assert torch.equal(bits(b.k_cache[used, :, :12]), bits(kc[used, :, :12])) and torch.equal(bits(q2), bits(q_out))
    assert torch.equal(bits(b.v_cache[used[:18]]), bits(vc[used[:18]])) and torch.equal(bits(mean2), bits(k_mean))


def test_append_reports_and_leaves_out_what_makes_no_sense():
    b = ref.make([2, 2, 2], [40, 50, 60], H=2, H_kv=1, D=64, page=32, seed=11, poison=False)
    q, k, v = ref.rows(b, 2, 1), ref.rows(b, 1, 2), ref.rows(b, 1, 3)

    def go(table=None, q_start=None, kv_len=None, **kw):
        bk = b.k_cache.clone()
        q_out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        bsa.paged_append(k, v, b.k_cache, b.v_cache, b.table if table is None else table,
                         b.q_start if q_start is None else q_start, b.kv_len if kv_len is None else kv_len, q=q,
                         q_out=q_out, **kw)
        st = bsa.device_status()
        return st, (bits(b.k_cache) != bits(bk)).any(-1).any(1), q_out

    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for page in (-1, b.n_pages, 1 << 30):
        table = b.table.clone()
        table[1, 1] = page
        st, changed, q_out = go(table=table)
        assert st == BOUNDS and int(changed.sum()) == 4 and not (q_out == 7.0).any()
        b.k_cache.zero_()
    for kw in (dict(kv_len=i32([40, -1, 60])), dict(kv_len=i32([40, 65, 60])), dict(q_start=i32([0, 2, -5, 2])),
               dict(q_start=i32([0, 2, 7, 2])), dict(q_start=i32([2, 1, 3, 6]))):
        assert go(**kw)[0] == BOUNDS
    b.k_cache.zero_()
    st, changed, q_out = go(kv_len=i32([40, 1, 60]))          # two new tokens, one position
    assert st == BOUNDS and int(changed.sum()) == 5 and (q_out[2] == 7.0).all() and not (q_out[3] == 7.0).any()
    st, _, _ = go(rope=ref.rope_table(59, 64))                # position 59 has no angles
    assert st == BOUNDS
    assert go(rope=ref.rope_table(60, 64))[0] == 0


# ------------------------------------------------------------------ attention

def run_forward(b, q, **kw):
    o = torch.full((b.tokens, b.H, b.D), 7.0, dtype=torch.bfloat16, device=b.device)
    lse = torch.full((b.tokens, b.H), 7.0, device=b.device)
    bsa.forward_paged(q, b.k_cache, b.v_cache, *b.arrays(), o, lse, **kw)
    return o, lse


def untouched(b, o, lse):
    out = torch.ones(b.tokens, dtype=torch.bool, device=b.device)
    out[b.q_start[0].item():b.q_start[-1].item()] = False
    return bool((o[out] == 7.0).all() and (lse[out] == 7.0).all())


SHAPES = [(4, 2, 128, 128), (4, 2, 128, 16), (14, 2, 64, 32), (3, 3, 64, 64), (16, 1, 128, 64), (128, 1, 64, 16),
          (40, 8, 128, 128)]
ATT = dict(one=([1], [1]), edge=([1] * 6, [1, 2, 127, 128, 129, 257]), step=([1] * 9, [1000, 3, 64, 700, 511, 1, 1500, 128, 90]),
           prompt=([300, 5], [300, 5]), chunks=([0, 3, 128, 1, 257, 64], [50, 131, 256, 1384, 300, 64]),
           long=([1, 2], [20001, 9000]))


@pytest.mark.parametrize("lens", ATT)
@pytest.mark.parametrize("H,K,D,page", SHAPES)
def test_attention(lens, H, K, D, page):
    """Causal, with NaN in every slot that holds no token."""
    b = ref.make(*ATT[lens], H=H, H_kv=K, D=D, page=page, seed=21, pad_tokens=3, first=2)
    q = ref.rows(b, H, 22)
    o, lse = run_forward(b, q)
    status_ok()
    ref.check_attention(b, q, o, lse)
    assert untouched(b, o, lse)


@pytest.mark.parametrize("causal,window,sinks", [(False, 0, 0), (True, 100, 0), (True, 200, 40), (True, 1, 0),
                                                 (False, 130, 300), (True, 4000, 64), (True, 128, 1000)])
@pytest.mark.parametrize("H,K,D,page", SHAPES[:3])
def test_masks(causal, window, sinks, H, K, D, page):
    b = ref.make([1, 40, 200, 3], [700, 1040, 600, 3], H=H, H_kv=K, D=D, page=page, seed=23)
    q = ref.rows(b, H, 24)
    kw = dict(causal=causal, window=window, sinks=sinks)
    o, lse = run_forward(b, q, **kw)
    status_ok()
    ref.check_attention(b, q, o, lse, **kw)


def test_rows_without_a_key():
    """An empty sequence, and a chunk longer than what the cache holds."""
    b = ref.make([2, 40, 3], [0, 10, 200], H=4, H_kv=2, D=128, page=16, seed=25)
    q = ref.rows(b, 4, 26)
    o, lse = run_forward(b, q)                     # causal: the first 30 tokens stand before position 0
    status_ok()
    assert torch.isneginf(lse[:32]).all() and not o[:32].any() and torch.isfinite(lse[32:]).all()
    ref.check_attention(b, q, o, lse)
    o, lse = run_forward(b, q, causal=False)       # every token sees what there is
    assert torch.isneginf(lse[:2]).all() and not o[:2].any()
    ref.check_attention(b, q, o, lse, causal=False)


def test_scale_and_large_scores():
    """Scores of hundreds: the running maximum moves by more than 2^64."""
    b = ref.make([1, 70], [900, 1500], H=4, H_kv=2, D=128, page=32, seed=27)
    q = ref.rows(b, 4, 28)
    for scale in (1.0, 4.0, 1e-3):
        o, lse = run_forward(b, q, scale=scale)
        status_ok()
        ref.check_attention(b, q, o, lse, scale=scale)
    # growing keys: every tile's maximum is a new one
    for s, n in enumerate(b.length):
        for p in range((n + 31) // 32):
            rows = min(32, n - 32 * p)
            b.k_cache[b.table[s, p], :, :rows] = (q[s, 0].float() * (0.02 * p)).to(torch.bfloat16)
    o, lse = run_forward(b, q, scale=1.0)
    status_ok()
    ref.check_attention(b, q, o, lse, scale=1.0)


def test_queries_may_be_views():
    b = ref.make([5, 33], [40, 533], H=6, H_kv=2, D=128, page=32, seed=29)
    qkv = ref.rows(b, 10, 30)
    o, lse = run_forward(b, qkv[:, 2:8])
    o2, lse2 = run_forward(b, qkv[:, 2:8].contiguous())
    status_ok()
    assert torch.equal(bits(o), bits(o2)) and torch.equal(lse, lse2)
    ref.check_attention(b, qkv[:, 2:8], o, lse)


@pytest.mark.parametrize("seed", range(6))
def test_random_batches(seed):
    g = np.random.default_rng(100 + seed)
    H, K = [(4, 2), (7, 1), (12, 12), (40, 8), (24, 4), (96, 1)][seed]
    n = int(g.integers(1, 60))
    new = [int(x) for x in g.integers(0, 90, n)]
    length = [int(a + g.integers(0, 900)) for a in new]
    b = ref.make(new, length, H=H, H_kv=K, D=int(g.choice([64, 128])), page=int(g.choice([16, 32, 64, 128])), seed=seed)
    if b.tokens == 0:
        return
    q = ref.rows(b, H, seed)
    o, lse = run_forward(b, q)
    status_ok()
    ref.check_attention(b, q, o, lse)


def test_many_sequences():
    """More sequences than threads of a block, most of them without new tokens."""
    g = np.random.default_rng(9)
    new = [int(x) for x in (g.random(3000) < 0.2) * g.integers(1, 3, 3000)]
    length = [int(a + g.integers(0, 40)) for a in new]
    b = ref.make(new, length, H=2, H_kv=1, D=64, page=16, seed=31)
    q = ref.rows(b, 2, 32)
    o, lse = run_forward(b, q)
    status_ok()
    ref.check_attention(b, q, o, lse)


HIDDEN = dict(future=dict(), window=dict(window=150, sinks=5), lists="lists")


@pytest.mark.parametrize("kind", HIDDEN)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("H,K,D,page", [(4, 2, 128, 128), (14, 2, 64, 16), (2, 2, 128, 32)])
def test_what_a_row_does_not_see_does_not_reach_it(H, K, D, page, bad, kind):
    """Keys and values that are not finite, at places that some rows of a tile see and
    others do not: those that do not get what they get without them."""
    b = ref.make([120, 40, 1], [1500, 300, 700], H=H, H_kv=K, D=D, page=page, seed=37)
    q = ref.rows(b, H, 38)
    kw, sel = HIDDEN[kind], None
    if kind == "lists":
        s, c, sel = lists_for(b, np.random.default_rng(39), 6)
        kw = dict(sel=s, sel_cnt=c)
    places = [(0, 1439, 3), (0, 1290, 0), (0, 2, 1), (1, 270, 5), (1, 299, 7), (2, 400, 2)]  # sequence, position, column
    good = b.k_cache.clone(), b.v_cache.clone()
    o0, lse0 = run_forward(b, q, **kw)
    ref.check_attention(b, q, o0, lse0, **(dict(sel=sel) if sel else kw))
    sees = torch.zeros(b.tokens, K, dtype=torch.bool, device="cuda")
    starts = b.q_start.tolist()
    for s, pos, col in places:
        for cache in (b.k_cache, b.v_cache):
            cache[b.table[s, pos // page], :, pos % page, col] = bad
        for i in range(b.new[s]):
            p = b.length[s] - b.new[s] + i
            see = pos <= p and (kind != "window" or pos > p - 150 or pos < 5)
            for h in range(K):
                sees[starts[s] + i, h] |= see and (sel is None or pos // 128 in sel[starts[s] + i][h])
    o, lse = run_forward(b, q, **kw)
    status_ok()
    hit = sees.repeat_interleave(H // K, 1)
    assert hit.any() and not hit.all()
    assert torch.isfinite(o[~hit].float()).all()
    b.k_cache, b.v_cache = good
    keep = o.clone(), lse.clone()
    keep[0][hit], keep[1][hit] = o0[hit], lse0[hit]
    ref.check_attention(b, q, *keep, **(dict(sel=sel) if sel else kw))
    if bad != bad:
        assert torch.isnan(o[hit].float()).any(-1).all() and torch.isnan(lse[hit]).all()


def test_a_query_that_is_not_finite_stays_alone():
    b = ref.make([70, 3], [500, 300], H=8, H_kv=2, D=128, page=64, seed=40)
    q = ref.rows(b, 8, 41)
    o0, lse0 = run_forward(b, q)
    q[11, 3, 7], q[40, 0, 0] = float("nan"), float("inf")
    o, lse = run_forward(b, q)
    status_ok()
    same = torch.ones(b.tokens, 8, dtype=torch.bool, device="cuda")
    same[11, 3] = same[40, 0] = False
    assert torch.equal(bits(o)[same], bits(o0)[same]) and torch.equal(lse[same], lse0[same])
    assert torch.isnan(o[~same].float()).all()


def test_the_same_call_gives_the_same_bits():
    b = ref.make([1, 1, 130], [15000, 7000, 4000], H=8, H_kv=2, D=128, page=64, seed=33)
    q = ref.rows(b, 8, 34)
    first = run_forward(b, q)
    for _ in range(5):
        again = run_forward(b, q)
        assert torch.equal(bits(first[0]), bits(again[0])) and torch.equal(first[1], again[1])
    status_ok()


def test_attention_reports_what_makes_no_sense():
    b = ref.make([2, 2, 2], [40, 50, 60], H=2, H_kv=1, D=64, page=32, seed=35, poison=False)
    q = ref.rows(b, 2, 36)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    good = run_forward(b, q)

    def go(**kw):
        a = dict(table=b.table, q_start=b.q_start, kv_len=b.kv_len)
        a.update(kw)
        o = torch.full((b.tokens, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((b.tokens, 2), 7.0, device="cuda")
        bsa.forward_paged(q, b.k_cache, b.v_cache, a["table"], a["q_start"], a["kv_len"], o, lse)
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

def lists_for(b, g, width, empty=0.0):
    """Random lists (unordered, repeated entries, blocks behind the token) as tensors and as sets."""
    sel = torch.full((b.tokens, b.H_kv, width), -1, dtype=torch.int32)
    cnt = torch.zeros((b.tokens, b.H_kv), dtype=torch.int32)
    want = [[[] for _ in range(b.H_kv)] for _ in range(b.tokens)]
    starts = b.q_start.tolist()
    for s, (n, length) in enumerate(zip(b.new, b.length)):
        blocks = (length + 127) // 128
        for t in range(starts[s], starts[s] + n):
            for h in range(b.H_kv):
                c = 0 if blocks == 0 or g.random() < empty else int(g.integers(0, width + 1))
                pick = g.integers(0, max(blocks, 1), c)
                sel[t, h, :c] = torch.from_numpy(pick.astype(np.int32))
                cnt[t, h] = c
                want[t][h] = sorted(set(pick.tolist()))
    return sel.cuda(), cnt.cuda(), want


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,K,D,page", SHAPES)
def test_attention_over_lists(H, K, D, page, causal):
    b = ref.make([1, 40, 0, 150, 3], [700, 1040, 30, 2000, 3], H=H, H_kv=K, D=D, page=page, seed=41, first=1, pad_tokens=2)
    q = ref.rows(b, H, 42)
    sel, cnt, want = lists_for(b, np.random.default_rng(43), 5, empty=0.1)
    o, lse = run_forward(b, q, sel=sel, sel_cnt=cnt, causal=causal)
    status_ok()
    ref.check_attention(b, q, o, lse, sel=want, causal=causal)
    assert untouched(b, o, lse)


def test_all_blocks_listed_is_the_plain_call():
    b = ref.make([1, 30], [1000, 700], H=4, H_kv=2, D=128, page=64, seed=44)
    q = ref.rows(b, 4, 45)
    every = torch.arange(8, dtype=torch.int32, device="cuda").expand(b.tokens, 2, 8).contiguous()
    cnt = torch.full((b.tokens, 2), 8, dtype=torch.int32, device="cuda")
    cnt[1:] = 6
    o, lse = run_forward(b, q, sel=every, sel_cnt=cnt)
    o2, lse2 = run_forward(b, q)
    status_ok()
    assert torch.equal(bits(o), bits(o2)) and torch.equal(lse, lse2)


def test_lists_report_what_makes_no_sense():
    b = ref.make([2, 3], [300, 500], H=4, H_kv=2, D=128, page=64, seed=46)
    q = ref.rows(b, 4, 47)
    sel, cnt, want = lists_for(b, np.random.default_rng(48), 3)
    for change, code in (((0, 0, 0, 3), BOUNDS), ((0, 0, 0, -1), BOUNDS), ((4, 1, 0, 1 << 30), BOUNDS)):
        s2, c2 = sel.clone(), cnt.clone()
        s2[change[0], change[1], change[2]] = change[3]
        c2[change[0], change[1]] = 1
        o, lse = run_forward(b, q, sel=s2, sel_cnt=c2)
        assert bsa.device_status() == code
        w2 = [[list(x) for x in r] for r in want]
        w2[change[0]][change[1]] = []                       # the one entry is left out
        ref.check_attention(b, q, o, lse, sel=w2)
    for n, code in ((4, OVERFLOW), (-1, BOUNDS)):
        c2 = cnt.clone()
        c2[1, 1] = n
        run_forward(b, q, sel=sel.clamp(min=0), sel_cnt=c2)
        assert bsa.device_status() == code


# ------------------------------------------------------------------ selection

def mean_keys(b, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((b.n_pages, b.H_kv, b.D), generator=g).to(torch.bfloat16).cuda()


def run_select(b, q, k_mean, width=None, **kw):
    width = kw["topk"] + kw["sink_blocks"] + kw["local_blocks"] if width is None else width
    sel = torch.full((b.tokens, b.H_kv, width), 77, dtype=torch.int32, device="cuda")
    cnt = torch.full((b.tokens, b.H_kv), 77, dtype=torch.int32, device="cuda")
    bsa.select_paged(q, k_mean, *b.arrays(), sel, cnt, page_size=b.page, **kw)
    return sel, cnt


def check_select(b, q, k_mean, sel, cnt, topk, sink_blocks, local_blocks):
    want = ref.select(b, q, k_mean, topk, sink_blocks, local_blocks)
    a, e = b.q_start[0].item(), b.q_start[-1].item()
    sh, ch = sel.cpu().numpy(), cnt.cpu().numpy()
    for t in range(b.tokens):
        for h in range(b.H_kv):
            if not a <= t < e:
                assert ch[t, h] == 77 and (sh[t, h] == 77).all()
                continue
            w = want[t][h]
            assert sh[t, h, :len(w)].tolist() == w and ch[t, h] == len(w) and (sh[t, h, len(w):] == -1).all(), (t, h)
    return want


@pytest.mark.parametrize("topk,sinks,local", [(4, 1, 1), (0, 1, 1), (1, 0, 1), (7, 2, 3), (300, 0, 1), (16, 5, 9)])
@pytest.mark.parametrize("H,K,D,page", SHAPES)
def test_selection(H, K, D, page, topk, sinks, local):
    b = ref.make([1, 20, 0, 140, 3, 2], [4000, 2100, 30, 3900, 3, 128], H=H, H_kv=K, D=D, page=page, seed=51, first=1,
                 pad_tokens=2, poison=False)
    q, km = ref.rows(b, H, 52), mean_keys(b, 53)
    kw = dict(topk=topk, sink_blocks=sinks, local_blocks=local)
    sel, cnt = run_select(b, q, km, width=topk + sinks + local + 2, **kw)
    status_ok()
    check_select(b, q, km, sel, cnt, **kw)


@pytest.mark.parametrize("kind", ["equal", "zero", "steps", "close"])
def test_close_and_equal_scores(kind):
    """Ties go to the lower block, and scores that fp32 cannot tell apart are told apart."""
    b = ref.make([30], [128 * 400 + 7], H=4, H_kv=2, D=128, page=128, seed=54, poison=False)
    q, km = ref.rows(b, 4, 55), mean_keys(b, 56)
    at = b.table[0].long()
    if kind == "equal":
        km[:] = km[0]
    elif kind == "zero":
        km.zero_()
    elif kind == "steps":
        for j in range(400):
            km[at[j]] = km[at[j % 9]]                       # nine different scores, 44 blocks each
    else:
        km[:] = km[0]
        # one value of each mean moved by one bf16 step where q is tiny: the scores differ by about 2^-30
        q[..., 5] = 2.0 ** -22
        km[..., 5] = 1.0
        for j in range(400):
            km[at[j], :, 5] = 1.0 + (j * 37 % 101) / 128
    kw = dict(topk=16, sink_blocks=1, local_blocks=1)
    sel, cnt = run_select(b, q, km, **kw)
    status_ok()
    check_select(b, q, km, sel, cnt, **kw)


def test_selection_of_the_longest_cache():
    b = ref.make([2], [1 << 20], H=2, H_kv=1, D=64, page=128, seed=57, poison=False)
    q, km = ref.rows(b, 2, 58), mean_keys(b, 59)
    for topk in (5, 8000):
        kw = dict(topk=topk, sink_blocks=1, local_blocks=2)
        sel, cnt = run_select(b, q, km, **kw)
        status_ok()
        check_select(b, q, km, sel, cnt, **kw)


def test_selection_with_nan_and_infinite_means():
    b = ref.make([3], [128 * 40], H=2, H_kv=1, D=64, page=64, seed=60, poison=False)
    q, km = ref.rows(b, 2, 61), mean_keys(b, 62)
    at = b.table[0, 1::2].long()
    km[at[7]] = float("nan")
    sel, cnt = run_select(b, q, km, topk=38, sink_blocks=0, local_blocks=1)   # all but one of 39: not the NaN
    status_ok()
    assert sel[2, 0].tolist() == [j for j in range(40) if j != 7]
    km[at[7]] = 1.0
    km[at[9], 0, 0] = float("inf")
    sel, cnt = run_select(b, q, km, topk=1, sink_blocks=0, local_blocks=1)
    status_ok()
    pos = q[:, :, 0].double().sum(1) > 0
    assert [9 in sel[t, 0].tolist() for t in range(3)] == pos.tolist()


def test_selection_reports_what_makes_no_sense():
    b = ref.make([2, 2], [1000, 1200], H=2, H_kv=1, D=64, page=32, seed=63, poison=False)
    q, km = ref.rows(b, 2, 64), mean_keys(b, 65)
    table = b.table.clone()
    table[1, 7] = b.n_pages
    b2 = ref.Batch(**{**b.__dict__, "table": table})
    sel, cnt = run_select(b2, q, km, topk=2, sink_blocks=0, local_blocks=1)
    assert bsa.device_status() == BOUNDS and (cnt == 3).all()
    b2 = ref.Batch(**{**b.__dict__, "kv_len": torch.tensor([1000, 5000], dtype=torch.int32, device="cuda")})
    sel, cnt = run_select(b2, q, km, topk=2, sink_blocks=0, local_blocks=1)
    assert bsa.device_status() == BOUNDS and (cnt[2:] == 77).all() and (cnt[:2] == 3).all()


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("page", [16, 128])
def test_a_conversation(page):
    """A prompt in two chunks, then single tokens, each selected over what the
    earlier calls left, against the same tokens at once and fp64."""
    H, K, D, n = 8, 2, 128, 1100
    g = torch.Generator().manual_seed(70)
    q, k, v = (torch.randn((n, h, D), generator=g).to(torch.bfloat16).cuda() for h in (H, K, K))
    rope = ref.rope_table(n, D)
    pages = (n + page - 1) // page
    table = torch.randperm(pages + 3, generator=g)[:pages].to(torch.int32).cuda()[None].contiguous()
    kc, vc = (torch.full((pages + 3, K, page, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    km = torch.full((pages + 3, K, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    qr, o = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty((n, H), device="cuda")
    kw = dict(topk=3, sink_blocks=1, local_blocks=2)
    sel = torch.empty((n, K, 6), dtype=torch.int32, device="cuda")
    cnt = torch.empty((n, K), dtype=torch.int32, device="cuda")
    at = 0
    for step in [500, 590] + [1] * 10:
        t = slice(at, at + step)
        batch = (table, torch.tensor([0, step], dtype=torch.int32, device="cuda"),
                 torch.tensor([at + step], dtype=torch.int32, device="cuda"))
        bsa.paged_append(k[t], v[t], kc, vc, *batch, q=q[t], q_out=qr[t], rope=rope, k_mean=km)
        bsa.select_paged(qr[t], km, *batch, sel[t], cnt[t], page_size=page, **kw)
        bsa.forward_paged(qr[t], kc, vc, *batch, o[t], lse[t], sel=sel[t], sel_cnt=cnt[t])
        at += step
    status_ok()
    b = ref.Batch([n], [n], H, K, D, page, "cuda", table=table, q_start=torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                  kv_len=torch.tensor([n], dtype=torch.int32, device="cuda"), k_cache=kc, v_cache=vc, n_pages=pages + 3, tokens=n)
    want = check_select(b, qr, km, sel, cnt, **kw)
    ref.check_attention(b, qr, o, lse, sel=want)
    pos = torch.arange(n, device="cuda")
    y, size = ref.turned(k, pos, rope, False, None, 0.0)
    got = torch.stack([b.keys(0, h) for h in range(K)], 1)
    assert ((got - y).abs() <= 2.0 ** -8 * y.abs() * 1.01 + 2.0 ** -22 * size).all()
    # the whole text at once leaves the same cache
    k2, v2, m2, q2 = torch.full_like(kc, float("nan")), torch.full_like(vc, float("nan")), torch.full_like(km, float("nan")), torch.empty_like(q)
    bsa.paged_append(k, v, k2, v2, *b.arrays(), q=q, q_out=q2, rope=rope, k_mean=m2)
    status_ok()
    for x, z in ((kc, k2), (vc, v2), (km, m2), (qr, q2)):
        assert torch.equal(bits(x), bits(z))


def test_captured_and_replayed_as_the_sequences_grow():
    """One graph of append, select and attend; lengths, tables and tokens change between replays."""
    H, K, D, page, S = 8, 2, 128, 32, 5
    g = torch.Generator().manual_seed(80)
    length0 = [300, 129, 1, 1000, 64]
    b = ref.make([1] * S, length0, H=H, H_kv=K, D=D, page=page, seed=81, max_pages=40, spare=30)
    free = [p for p in range(b.n_pages) if p not in set(b.table[b.table >= 0].tolist())]
    km = torch.zeros((b.n_pages, K, D), dtype=torch.bfloat16, device="cuda")
    for s, n in enumerate(length0):
        for j in range(n // 128):
            which = b.table[s, j * 4:(j + 1) * 4].long()
            km[which[-1]] = b.k_cache[which].float().mean((0, 2)).to(torch.bfloat16)
    q, k, v = ref.rows(b, H, 82), ref.rows(b, K, 83), ref.rows(b, K, 84)
    rope = ref.rope_table(2000, D)
    qr, o = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty((S, H), device="cuda")
    kw = dict(topk=2, sink_blocks=1, local_blocks=1)
    sel = torch.empty((S, K, 4), dtype=torch.int32, device="cuda")
    cnt = torch.empty((S, K), dtype=torch.int32, device="cuda")

    def step():
        bsa.paged_append(k, v, b.k_cache, b.v_cache, *b.arrays(), q=q, q_out=qr, rope=rope, k_mean=km)
        bsa.select_paged(qr, km, *b.arrays(), sel, cnt, page_size=page, **kw)
        bsa.forward_paged(qr, b.k_cache, b.v_cache, *b.arrays(), o, lse, sel=sel, sel_cnt=cnt)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens = list(length0)
    for turn in range(6):
        if turn:
            lens = [n + 1 for n in lens]
            for s, n in enumerate(lens):
                at = (n - 1) // page
                if b.table[s, at] < 0:
                    b.table[s, at] = free.pop()
            b.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
            for t, h in ((q, H), (k, K), (v, K)):
                t.copy_(torch.randn((S, h, D), generator=g).to(torch.bfloat16))
        o.fill_(7.0)
        graph.replay()
        status_ok()
        b.length = lens
        want = check_select(b, qr, km, sel, cnt, **kw)
        ref.check_attention(b, qr, o, lse, sel=want)


def test_two_graphs_share_a_workspace_and_streams_do_not():
    """Graphs replayed one after the other on one workspace, and two streams at once on one each."""
    bs = [ref.make([1, 60], [9000, 3000 + 500 * x], H=8, H_kv=2, D=128, page=64, seed=90 + x) for x in range(2)]
    qs = [ref.rows(b, 8, 92 + x) for x, b in enumerate(bs)]
    want = [run_forward(b, q) for b, q in zip(bs, qs)]
    need = max(bsa.forward_paged_workspace_size(2, b.tokens, b.table.shape[1], 64, 8, 2, 128) for b in bs)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [(torch.empty_like(o), torch.empty_like(lse)) for o, lse in want]
    graphs = []
    for b, q, (o, lse) in zip(bs, qs, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            bsa.forward_paged(q, b.k_cache, b.v_cache, *b.arrays(), o, lse, workspace=ws)
        graphs.append(graph)
    for x in (0, 1, 1, 0, 1):
        outs[x][0].zero_()
        graphs[x].replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(outs[x][0]), bits(want[x][0])) and torch.equal(outs[x][1], want[x][1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for o, lse in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for st, sp, b, q, (o, lse) in zip(streams, spaces, bs, qs, outs):
            bsa.forward_paged(q, b.k_cache, b.v_cache, *b.arrays(), o, lse, workspace=sp, stream=st)
    torch.cuda.synchronize()
    for (o, lse), (wo, wl) in zip(outs, want):
        assert torch.equal(bits(o), bits(wo)) and torch.equal(lse, wl)
    status_ok()


# ------------------------------------------------------------------ the far ends

def test_caches_beyond_32_bits():
    """The same batch in pages at the end of a cache of 2.3e9 values gives the same bits."""
    H, K, D, page, pages = 8, 2, 128, 128, 70000
    b = ref.make([1, 130, 257], [3000, 1500, 257], H=H, H_kv=K, D=D, page=page, seed=100)
    q, k, v = ref.rows(b, H, 101), ref.rows(b, K, 102), ref.rows(b, K, 103)
    rope = ref.rope_table(3000, D)
    km = torch.randn((b.n_pages, K, D), generator=torch.Generator().manual_seed(104)).to(torch.bfloat16).cuda()
    at = pages - b.n_pages
    far = dict(table=torch.where(b.table >= 0, b.table + at, b.table), means=torch.zeros((pages, K, D), dtype=torch.bfloat16, device="cuda"))
    far["means"][at:] = km
    for x in ("k_cache", "v_cache"):
        far[x] = torch.zeros((pages, K, page, D), dtype=torch.bfloat16, device="cuda")
        far[x][at:] = getattr(b, x)
    assert far["k_cache"].numel() > 1 << 31
    outs = []
    for kc, vc, table, means in ((b.k_cache, b.v_cache, b.table, km), (far["k_cache"], far["v_cache"], far["table"], far["means"])):
        batch = (table, b.q_start, b.kv_len)
        qr, o = torch.empty_like(q), torch.empty_like(q)
        lse, o2, lse2 = torch.empty((b.tokens, H), device="cuda"), torch.empty_like(q), torch.empty((b.tokens, H), device="cuda")
        sel = torch.empty((b.tokens, K, 6), dtype=torch.int32, device="cuda")
        cnt = torch.empty((b.tokens, K), dtype=torch.int32, device="cuda")
        bsa.paged_append(k, v, kc, vc, *batch, q=q, q_out=qr, rope=rope, k_mean=means)
        bsa.select_paged(qr, means, *batch, sel, cnt, page_size=page, topk=4)
        bsa.forward_paged(qr, kc, vc, *batch, o, lse, sel=sel, sel_cnt=cnt)
        bsa.forward_paged(qr, kc, vc, *batch, o2, lse2)
        status_ok()
        first = 0 if kc is b.k_cache else at
        outs.append((qr, o, o2, lse, lse2, sel, cnt, means[first:], kc[first:].nan_to_num(3.0), vc[first:].nan_to_num(3.0)))
    for x, y in zip(*outs):
        assert torch.equal(x, y)
    assert not far["k_cache"][:at].any() and not far["v_cache"][:at].any() and not far["means"][:at].any()


def test_windows_of_any_length():
    """A window longer than any sequence is none, with tokens before position 0 too."""
    b = ref.make([1, 300, 200], [700, 300, 150], H=4, H_kv=2, D=64, page=32, seed=105)
    q = ref.rows(b, 4, 106)
    o, lse = run_forward(b, q)
    for window in (1 << 20, 2 ** 31 - 1):
        for sinks in (0, 2 ** 31 - 1):
            o2, lse2 = run_forward(b, q, window=window, sinks=sinks)
            assert torch.equal(bits(o2), bits(o)) and torch.equal(lse2, lse)
    status_ok()
    ref.check_attention(b, q, o, lse)


def test_scratch_of_another_stream_is_not_reused_early():
    """Calls on a stream that is busy, without a workspace, while the current one allocates and writes."""
    b = ref.make([1, 60, 2], [9000, 3000, 20000], H=8, H_kv=2, D=128, page=64, seed=107)
    q = ref.rows(b, 8, 108)
    km = torch.randn((b.n_pages, 2, 128), generator=torch.Generator().manual_seed(109)).to(torch.bfloat16).cuda()
    sel = torch.empty((b.tokens, 2, 10), dtype=torch.int32, device="cuda")
    cnt = torch.empty((b.tokens, 2), dtype=torch.int32, device="cuda")

    def go(o, lse, stream=None):
        bsa.select_paged(q, km, *b.arrays(), sel, cnt, page_size=64, topk=8, stream=stream)
        bsa.forward_paged(q, b.k_cache, b.v_cache, *b.arrays(), o, lse, sel=sel, sel_cnt=cnt, stream=stream)

    want, got = [(torch.empty_like(q), torch.empty((b.tokens, 8), device="cuda")) for _ in range(2)]
    go(*want)
    sel0, cnt0 = sel.clone(), cnt.clone()
    sizes = (bsa.select_paged_workspace_size(3, b.tokens, b.table.shape[1], 64, 8, 2, 128),
             bsa.forward_paged_workspace_size(3, b.tokens, b.table.shape[1], 64, 8, 2, 128, 10))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    go(*got, stream=side)
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    status_ok()
    assert len(junk) == 6 and torch.equal(sel, sel0) and torch.equal(cnt, cnt0)
    assert torch.equal(bits(got[0]), bits(want[0])) and torch.equal(got[1], want[1])


def test_rows_next_to_values_that_are_not_finite_over_a_long_cache():
    """Every row has an infinite value at its first key and all but the last of a sequence a NaN
    behind their own: 128 rows of 2^19 keys are computed from their own keys by one thread block,
    which takes longer than a wait may last without progress."""
    n, L, S = 128, 1 << 19, 152
    dev = "cuda"
    k = torch.zeros((L // 128, 1, 128, 64), dtype=torch.bfloat16, device=dev)
    v = torch.ones_like(k)
    v[0, 0, 0, 0] = float("inf")
    v[-1, 0, -1, 1] = float("nan")
    table = torch.arange(L // 128, dtype=torch.int32, device=dev).repeat(S, 1)
    start = torch.arange(S + 1, dtype=torch.int32, device=dev) * n
    length = torch.full((S,), L, dtype=torch.int32, device=dev)
    q = torch.randn((S * n, 1, 64), generator=torch.Generator().manual_seed(110)).to(torch.bfloat16).to(dev)
    o, lse = torch.empty_like(q), torch.empty((S * n, 1), device=dev)
    bsa.forward_paged(q, k, v, table, start, length, o, lse)
    status_ok()
    want = torch.ones((S, n, 64), device=dev)
    want[:, :, 0] = float("inf")
    want[:, -1, 1] = float("nan")
    got = o.view(S, n, 64).float()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
    fin = want.isfinite()
    assert ((got - want)[fin].abs() <= 2.0 ** -7).all()
    keys = torch.arange(L - n + 1, L + 1, dtype=torch.float64, device=dev)
    # a sum of ones in fp32, its parts at most 2^19: exact; a logarithm and a product
    assert ((lse.view(S, n).double() - keys.log()).abs() <= 8 * 2.0 ** -24 * (1 + keys.log())).all()


def test_very_many_heads():
    b = ref.make([1, 3], [5, 200], H=16384, H_kv=16384, D=64, page=128, seed=111, poison=False)
    q, k, v = ref.rows(b, 16384, 112), ref.rows(b, 16384, 113), ref.rows(b, 16384, 114)
    rope = ref.rope_table(200, 64)
    bk, bv = b.k_cache.clone(), b.v_cache.clone()
    q_out, k_mean = run_append(b, q, k, v, rope=rope)
    status_ok()
    check_append(b, q, k, v, bk, bv, q_out, k_mean, rope=rope)
    o, lse = run_forward(b, q_out)
    sel = torch.empty((b.tokens, 16384, 2), dtype=torch.int32, device="cuda")
    cnt = torch.empty((b.tokens, 16384), dtype=torch.int32, device="cuda")
    bsa.select_paged(q_out, k_mean, *b.arrays(), sel, cnt, page_size=128, topk=1, sink_blocks=0)
    o2, lse2 = run_forward(b, q_out, sel=sel, sel_cnt=cnt)  # (all blocks there are)
    status_ok()
    assert torch.equal(cnt[0], torch.ones_like(cnt[0])) and torch.equal(cnt[1:], torch.full_like(cnt[1:], 2))
    # both within the bound of ref.check_attention, where A is at most the largest |v| and
    # the fp32 term, 2 (D + 16) 2^-24 (R + 1) A with R < 20 and |v| < 6, below 2^-10
    far = 2.0 ** -7 * 1.01 * (b.v_cache.abs().max().float() + 1.01 * o.float().abs()) + 2.0 ** -9
    assert ((o2.float() - o.float()).abs() <= far).all()
    for h in (0, 1, 9000, 16383):  # against the reference, a head at a time
        one = ref.Batch(b.new, b.length, 1, 1, 64, 128, "cuda", table=b.table, q_start=b.q_start, kv_len=b.kv_len,
                        k_cache=b.k_cache[:, h:h + 1], v_cache=b.v_cache[:, h:h + 1], n_pages=b.n_pages, tokens=b.tokens)
        ref.check_attention(one, q_out[:, h:h + 1], o[:, h:h + 1], lse[:, h:h + 1])
        ref.check_attention(one, q_out[:, h:h + 1], o2[:, h:h + 1], lse2[:, h:h + 1])


FIRST_CALL = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch, paged_ref as ref, long_context_mask_gb300 as bsa
b = ref.make([1, 60], [900, 300], H=8, H_kv=2, D=128, page=64, seed=120, poison=False)
q, k, v = ref.rows(b, 8, 1), ref.rows(b, 2, 2), ref.rows(b, 2, 3)
km = torch.zeros((b.n_pages, 2, 128), dtype=torch.bfloat16, device="cuda")
qr, o, lse = torch.empty_like(q), torch.empty_like(q), torch.empty((b.tokens, 8), device="cuda")
sel = torch.empty((b.tokens, 2, 6), dtype=torch.int32, device="cuda")
cnt = torch.empty((b.tokens, 2), dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    bsa.paged_append(k, v, b.k_cache, b.v_cache, *b.arrays(), q=q, q_out=qr, k_mean=km)
    bsa.select_paged(qr, km, *b.arrays(), sel, cnt, page_size=64, topk=4)
    bsa.forward_paged(qr, b.k_cache, b.v_cache, *b.arrays(), o, lse, sel=sel, sel_cnt=cnt)
graph.replay()
torch.cuda.synchronize()
assert bsa.device_status() == 0
ref.check_attention(b, qr, o, lse, sel=ref.select(b, qr, km, 4, 1, 1))
"""


def test_the_first_calls_of_a_process_may_be_captured():
    """Nothing has been loaded or set up before the capture begins."""
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALL.format(root=os.path.dirname(tests), tests=tests)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=240)
    assert r.returncode == 0, r.stderr[-2000:]
