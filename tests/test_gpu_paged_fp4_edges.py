"""A paged cache in 4 bits at its edges: first calls, graphs and streams that share or do
not share, the largest sizes, pages that are there twice, and queries that are not finite."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import fp4_ref as f4
import long_context_mask_gb300 as bsa
import paged_ref as ref
from gpu_util import status_ok
from test_gpu_paged import bits, lists_for
from test_gpu_paged_fp4 import check_append, run_append, run_forward, untouched

pytestmark = pytest.mark.gpu
TESTS = os.path.dirname(os.path.abspath(__file__))


def in_a_process(code):
    r = subprocess.run([sys.executable, "-c", code.format(root=os.path.dirname(TESTS), tests=TESTS)], capture_output=True,
                       text=True, timeout=240)
    assert r.returncode == 0, r.stderr[-2000:]


# ------------------------------------------------------------------ first calls

CAPTURED = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch, fp4_ref as f4, paged_ref as ref, long_context_mask_gb300 as bsa
b = ref.make([1, 60], [900, 300], H=8, H_kv=2, D=128, page=16, seed=120, poison=False)
c = f4.Cache(b, 1)
q, k, v = ref.rows(b, 8, 1), ref.rows(b, 2, 2), ref.rows(b, 2, 3)
qr, o, lse = torch.empty_like(q), torch.empty_like(q), torch.empty((b.tokens, 8), device="cuda")
o2, lse2, back = torch.empty_like(q), torch.empty_like(lse), torch.empty_like(v)
sel = torch.arange(2, dtype=torch.int32, device="cuda").repeat(b.tokens, 2, 1)
cnt = torch.full((b.tokens, 2), 2, dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    bsa.paged_append_fp4(k, v, *c.arrays(), *b.arrays(), q=q, q_out=qr)
    bsa.forward_paged_fp4(qr, *c.arrays(), *b.arrays(), o, lse)
    bsa.forward_paged_fp4(qr, *c.arrays(), *b.arrays(), o2, lse2, sel=sel, sel_cnt=cnt)
    bsa.paged_read_fp4(*c.arrays(), *b.arrays(), None, back)
graph.replay()
torch.cuda.synchronize()
assert bsa.device_status() == 0
c.refresh()
f4.check_attention(b, qr, o, lse)
f4.check_attention(b, qr, o2, lse2, sel=[[[0, 1]] * 2] * b.tokens)
assert torch.equal(back[0, 1].double(), b.keys(0, 1, b.v_cache)[-1])
"""

THREADS = """
import sys, threading
sys.path[:0] = [{root!r}, {tests!r}]
import torch, fp4_ref as f4, paged_ref as ref, long_context_mask_gb300 as bsa
n = 8
bs = [ref.make([1, 40], [900, 300], H=8, H_kv=2, D=64 + 64 * (x % 2), page=16 << x % 3, seed=x, poison=False) for x in range(n)]
cs = [f4.Cache(b, x) for x, b in enumerate(bs)]
qs = [ref.rows(b, 8, 1) for b in bs]
outs = [(torch.empty_like(q), torch.empty((41, 8), device="cuda"), torch.empty((41, 2, b.D), dtype=torch.bfloat16, device="cuda"))
        for b, q in zip(bs, qs)]
streams = [torch.cuda.Stream() for _ in bs]
failed, together = [], threading.Barrier(n)
torch.cuda.synchronize()
bsa.load_library()

def go(x):
    b, c, q, (o, lse, back) = bs[x], cs[x], qs[x], outs[x]
    try:
        with torch.cuda.stream(streams[x]):
            together.wait()
            bsa.forward_paged_fp4(q, *c.arrays(), *b.arrays(), o, lse)
            bsa.paged_read_fp4(*c.arrays(), *b.arrays(), back)
    except Exception as e:
        failed.append(e)

threads = [threading.Thread(target=go, args=(x,)) for x in range(n)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not failed, failed
assert bsa.device_status() == 0
for b, q, (o, lse, back) in zip(bs, qs, outs):
    f4.check_attention(b, q, o, lse)
    assert all(torch.equal(back[1:, h].double(), b.keys(1, h)[260:]) for h in range(2))
"""


def test_the_first_calls_of_a_process_may_be_captured():
    """Nothing has been loaded or set up before the capture begins."""
    in_a_process(CAPTURED)


def test_first_calls_from_several_threads_at_once():
    in_a_process(THREADS)


# ------------------------------------------------------------------ graphs and streams

def test_two_graphs_share_a_workspace_and_streams_do_not():
    """Graphs replayed one after the other on one workspace, and two streams at once on one each."""
    bs = [ref.make([1, 60, 2], [9000, 3000 + 500 * x, 800], H=8, H_kv=2, D=128, page=32, seed=90 + x) for x in range(2)]
    cs = [f4.Cache(b, 90 + x) for x, b in enumerate(bs)]
    qs = [ref.rows(b, 8, 92 + x) for x, b in enumerate(bs)]
    want = [run_forward(b, c, q) for b, c, q in zip(bs, cs, qs)]
    need = max(bsa.forward_paged_fp4_workspace_size(3, b.tokens, b.table.shape[1], 32, 8, 2, 128) for b in bs)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [(torch.empty_like(o), torch.empty_like(lse)) for o, lse in want]
    graphs = []
    for b, c, q, (o, lse) in zip(bs, cs, qs, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            bsa.forward_paged_fp4(q, *c.arrays(), *b.arrays(), o, lse, workspace=ws)
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
        for st, sp, b, c, q, (o, lse) in zip(streams, spaces, bs, cs, qs, outs):
            bsa.forward_paged_fp4(q, *c.arrays(), *b.arrays(), o, lse, workspace=sp, stream=st)
    torch.cuda.synchronize()
    for (o, lse), (wo, wl) in zip(outs, want):
        assert torch.equal(bits(o), bits(wo)) and torch.equal(lse, wl)
    status_ok()


def test_a_workspace_of_exactly_its_size_is_enough():
    b = ref.make([1, 40, 0, 150, 3], [700, 1040, 30, 2000, 3], H=14, H_kv=2, D=64, page=16, seed=61)
    c = f4.Cache(b, 61)
    q = ref.rows(b, 14, 62)
    sel, cnt, want = lists_for(b, np.random.default_rng(63), 5)
    for lists in ({}, dict(sel=sel, sel_cnt=cnt)):
        need = bsa.forward_paged_fp4_workspace_size(5, b.tokens, b.table.shape[1], 16, 14, 2, 64, 5 if lists else 0)
        space = torch.full((need + 4096,), 0xa5, dtype=torch.uint8, device="cuda")
        o, lse = run_forward(b, c, q, workspace=space[:need], **lists)
        status_ok()
        f4.check_attention(b, q, o, lse, **(dict(sel=want) if lists else {}))
        assert (space[need:] == 0xa5).all()
        with pytest.raises(bsa.BsaError):
            run_forward(b, c, q, workspace=space[:need - 1], **lists)


# ------------------------------------------------------------------ masks, with the hint of few rows

@pytest.mark.parametrize("kw", [dict(window=100, sinks=5), dict(window=1), dict(causal=False, window=64), dict(causal=False)])
@pytest.mark.parametrize("H,K,D,page", [(14, 2, 64, 16), (8, 1, 128, 32), (12, 2, 128, 64), (16, 1, 64, 128)])
def test_masks_of_few_rows(H, K, D, page, kw):
    """Row tiles of 8 and of 16, as the hint chooses them."""
    b = ref.make([1, 2, 0, 2, 1], [700, 1040, 30, 2, 129], H=H, H_kv=K, D=D, page=page, seed=64, first=1, pad_tokens=1)
    c = f4.Cache(b, 64, gains=True)
    q = ref.rows(b, H, 65)
    for max_new in (0, 1, 2):
        o, lse = run_forward(b, c, q, max_new=max_new, **kw)
        status_ok()
        f4.check_attention(b, q, o, lse, **kw)
        assert untouched(b, o, lse)


@pytest.mark.parametrize("kw", [{}, dict(window=100, sinks=5), dict(causal=False)])
@pytest.mark.parametrize("H,K,D,page", [(14, 2, 64, 16), (32, 8, 128, 128), (3, 3, 128, 32), (128, 1, 64, 64)])
def test_one_sequence_with_room_for_many_tokens(H, K, D, page, kw):
    """A single sequence, whose tokens the host knows only as a number they do not exceed."""
    for new, length in ((0, 50), (1, 1), (1, 1500), (2, 129), (5, 700), (40, 40), (300, 1000)):
        b = ref.make([new], [length], H=H, H_kv=K, D=D, page=page, seed=80 + new, first=1, pad_tokens=330 - new)
        c = f4.Cache(b, 80)
        q = ref.rows(b, H, 81)
        o, lse = run_forward(b, c, q, **kw)
        status_ok()
        if new:
            f4.check_attention(b, q, o, lse, **kw)
        assert untouched(b, o, lse)


# ------------------------------------------------------------------ the far ends

@pytest.mark.parametrize("D,page", [(64, 16), (128, 128)])
def test_as_many_sequences_as_there_may_be(D, page):
    """16384 sequences, few of them with new tokens, one with a prompt: append, all forms of attention, read."""
    g = np.random.default_rng(66)
    new = [int(x) for x in (g.random(16384) < 0.02) * g.integers(1, 3, 16384)]
    new[9000] = 200
    length = [int(a + (g.integers(0, 40) if a else 0)) for a in new]
    b = ref.make(new, length, H=2, H_kv=1, D=D, page=page, seed=66)
    c = f4.Cache(b, 66)
    q, kv = ref.rows(b, 2, 67), ref.rows(b, 2, 68)
    before = c.clone()
    q_out, k_mean = run_append(b, c, q, kv[:, :1], kv[:, 1:])
    status_ok()
    check_append(b, c, q, kv[:, :1], kv[:, 1:], before, q_out, k_mean)
    for kw in (dict(max_new=0), dict(max_new=1), dict(window=9, sinks=2)):
        o, lse = run_forward(b, c, q, **kw)
        status_ok()
        kw.pop("max_new", None)
        f4.check_attention(b, q, o, lse, **kw)
    sel, cnt, want = lists_for(b, np.random.default_rng(69), 2)
    o, lse = run_forward(b, c, q, sel=sel, sel_cnt=cnt)
    status_ok()
    f4.check_attention(b, q, o, lse, sel=want)
    back = torch.empty((b.tokens, 1, D), dtype=torch.bfloat16, device="cuda")
    bsa.paged_read_fp4(*c.arrays(), *b.arrays(), back)
    status_ok()
    at = 0
    for s, n in enumerate(new):
        if n:
            assert torch.equal(back[at:at + n, 0].double(), b.keys(s, 0)[b.length[s] - n:])
            at += n


@pytest.mark.parametrize("new,max_new", [(1, 1), (2, 0), (3, 0)])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 128)])
def test_the_longest_sequence_out_of_one_page(new, max_new, D, page):
    """2^24 keys, all in one page that the table names again and again: O is the page's own, LSE
    larger by the logarithm of the number of copies."""
    b = ref.make([new], [page], H=8, H_kv=1, D=D, page=page, seed=68, poison=False)
    c = f4.Cache(b, 68)
    q = ref.rows(b, 8, 69)
    copies = (1 << 24) // page
    table = b.table[:, :1].expand(1, copies).contiguous()
    o, lse = torch.empty_like(q), torch.empty((new, 8), device="cuda")
    bsa.forward_paged_fp4(q, *c.arrays(), table, b.q_start, torch.tensor([1 << 24], dtype=torch.int32, device="cuda"), o, lse,
                          causal=False, max_new=max_new)
    status_ok()
    O, L, A, R = ref.attend(b, q, causal=False)
    W = f4.visible(b)  # (of one copy: all sums are relative to the number of copies)
    # f4.check_attention's bound, and the long sums.  A thread block has some 2^24 / 128 / 148 = 886 key tiles.
    # The denominator: at most 8 additions in a row to a tile, of every second one at most (row tiles of 16), or 9 of
    # each (prompts): below 8192 additions, to partial sums that average half the whole: 2^-12.
    # The numerator: at most 8 products of 16 keys to a tile, each rounded, or cut, by a step 2^-23 at
    # most of the partial sum: 7088 / 2 2^-23 < 2^-11.
    d = (D + 16) * 2.0 ** -24 * (R + 1)
    bound = 2.0 ** -8 * 1.01 * O.abs() + (2.0 ** -11 * 1.01 + 2.0 ** -11 + 2.0 ** -12 + 2 * d[..., None]) * A + 2.0 ** -25 * W
    assert ((o.double() - O).abs() <= bound).all()
    assert ((lse.double() - L - math.log(copies)).abs() <= 2.0 ** -12 + d + 8 * 2.0 ** -24 * (1 + L.abs() + 17)).all()


def test_the_smallest_and_largest_gains():
    """Gains from the smallest normal number to 2^125, with values of their sizes and zeros among them: append and read."""
    b = ref.make([300, 1], [300, 200], H=4, H_kv=4, D=64, page=32, seed=74, poison=False)
    c = f4.Cache(b, 74)
    c.k_gain = torch.tensor([2.0 ** -126, 1e-20, 3e20, 2.0 ** 125], device="cuda")
    c.v_gain = c.k_gain.flip(0).contiguous()
    q, k, v = ref.rows(b, 4, 75), ref.rows(b, 4, 76), ref.rows(b, 4, 77)
    k, v = ((x.double() * g.double()[:, None]).to(torch.bfloat16) for x, g in ((k, c.k_gain), (v, c.v_gain)))
    k[:, :, 3], v[5] = 0, 0
    before = c.clone()
    q_out, _ = run_append(b, c, q, k, v, means=False)
    status_ok()
    check_append(b, c, q, k, v, before, q_out, None)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    bsa.paged_read_fp4(*c.arrays(), *b.arrays(), ko, vo, **c.gains())
    status_ok()
    for h in range(4):
        for out, cache in ((ko, b.k_cache), (vo, b.v_cache)):
            want = b.keys(0, h, cache)
            # half a step, of the smallest numbers 2^-134
            assert ((out[:300, h].double() - want).abs() <= 2.0 ** -8 * 1.01 * want.abs() + 2.0 ** -134).all()


def test_a_page_may_be_there_twice():
    """Two sequences, and two places of one, share pages."""
    b = ref.make([3, 40], [500, 500], H=8, H_kv=2, D=128, page=64, seed=70, poison=False)
    b.table[1] = b.table[0]
    b.table[:, 5] = b.table[:, 2]
    c = f4.Cache(b, 70)
    q = ref.rows(b, 8, 71)
    o, lse = run_forward(b, c, q)
    status_ok()
    f4.check_attention(b, q, o, lse)
    back = torch.empty((b.tokens, 2, 128), dtype=torch.bfloat16, device="cuda")
    bsa.paged_read_fp4(*c.arrays(), *b.arrays(), back)
    status_ok()
    assert torch.equal(back[:3], back[40:])


# ------------------------------------------------------------------ queries that are not finite

def test_infinite_queries_against_keys_of_one_sign():
    """Scores of -infinity only: a row without a key; of +infinity: NaN.  No other row changes."""
    b = ref.make([70, 1], [500, 300], H=8, H_kv=2, D=128, page=64, seed=72)
    c = f4.Cache(b, 72)
    c.k &= 0x77
    c.k |= 0x11  # (no zero, no negative level)
    raw = c.k_scale.view(torch.uint8)
    raw.copy_(torch.where(raw == 0, torch.full_like(raw, 0x20), raw))
    c.refresh()
    q = ref.rows(b, 8, 73)
    o0, lse0 = run_forward(b, c, q)
    for t, h in ((11, 3), (69, 0), (70, 7)):
        q[t, h, 17] = -float("inf")
        q[t, h - 1 if h else 1, 5] = float("inf")
    o, lse = run_forward(b, c, q)
    status_ok()
    off = torch.isinf(q).any(-1)
    assert torch.equal(bits(o)[~off], bits(o0)[~off]) and torch.equal(lse[~off], lse0[~off])
    none, nan = torch.isneginf(q).any(-1), torch.isposinf(q).any(-1)
    assert (o[none] == 0).all() and torch.isneginf(lse[none]).all()
    assert torch.isnan(o[nan].float()).all() and torch.isnan(lse[nan]).all()


# ------------------------------------------------------------------ scratch that the binding brings

def test_scratch_of_a_call_goes_back_when_it_returns():
    """On the current stream, on another one, in a capture, and when the call is refused."""
    b = ref.make([1, 40], [900, 300], H=8, H_kv=2, D=128, page=64, seed=78)
    c = f4.Cache(b, 78)
    q = ref.rows(b, 8, 79)
    want = run_forward(b, c, q)
    side = torch.cuda.Stream()
    o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bsa.forward_paged_fp4(q, *c.arrays(), *b.arrays(), o, lse)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for kw in ({}, dict(stream=side)):
        side.wait_stream(torch.cuda.current_stream())
        bsa.forward_paged_fp4(q, *c.arrays(), *b.arrays(), o, lse, **kw)
        torch.cuda.synchronize()
        assert torch.cuda.memory_allocated() == before
        assert torch.equal(bits(o), bits(want[0])) and torch.equal(lse, want[1])
        o.zero_()
    with pytest.raises(bsa.BsaError):
        bsa.forward_paged_fp4(q, *c.arrays(), *b.arrays(), o, lse, scale=float("nan"))
    assert torch.cuda.memory_allocated() == before
    # the graph's scratch is its own: what is allocated in between does not get it
    held = [torch.full((1 << 22,), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(8)]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(o), bits(want[0])) and torch.equal(lse, want[1])
    assert all(bool((x == 0x7f).all()) for x in held)
    status_ok()


# ------------------------------------------------------------------ lists of few and of many tokens

@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,K,D,page", [(14, 2, 64, 16), (32, 8, 128, 64), (3, 3, 128, 128), (128, 1, 64, 32), (40, 2, 128, 16), (16, 1, 64, 128)])
def test_lists_of_few_and_of_many_tokens(H, K, D, page, causal):
    """Sequences on either side of where tokens' lists are taken together, one whose lists are empty, one
    alone, and what the host is told."""
    for new, length in (([1, 8, 9, 0, 200, 2, 17], [900, 1500, 700, 50, 1300, 2, 4000]), ([150], [2500]), ([3], [600]), ([0], [70])):
        b = ref.make(new, length, H=H, H_kv=K, D=D, page=page, seed=90, first=1, pad_tokens=40)
        c = f4.Cache(b, 90, gains=True)
        q = ref.rows(b, H, 91)
        sel, cnt, want = lists_for(b, np.random.default_rng(92), 6, empty=0.15)
        if len(new) > 1:
            t = b.q_start[2].item()  # a sequence of empty lists
            cnt[t:t + 9] = 0
            for x in range(t, t + 9):
                want[x] = [[] for _ in want[x]]
        for max_new in (0, 1, max(new), 10 ** 6):
            o, lse = run_forward(b, c, q, sel=sel, sel_cnt=cnt, causal=causal, max_new=max_new)
            status_ok()
            f4.check_attention(b, q, o, lse, sel=want, causal=causal)
            assert untouched(b, o, lse)


def test_lists_of_a_query_that_is_not_finite():
    """It changes no other row, whether they list the same blocks or others."""
    b = ref.make([70, 3], [1500, 600], H=8, H_kv=2, D=128, page=64, seed=94)
    c = f4.Cache(b, 94)
    q = ref.rows(b, 8, 95)
    sel, cnt, want = lists_for(b, np.random.default_rng(96), 4)
    o0, lse0 = run_forward(b, c, q, sel=sel, sel_cnt=cnt)
    f4.check_attention(b, q, o0, lse0, sel=want)
    q[11, 3, 7], q[40, 0, 0], q[71, 5, 1] = float("nan"), float("inf"), float("nan")
    o, lse = run_forward(b, c, q, sel=sel, sel_cnt=cnt)
    status_ok()
    same = torch.ones(b.tokens, 8, dtype=torch.bool, device="cuda")
    same[11, 3] = same[40, 0] = same[71, 5] = False
    assert torch.equal(bits(o)[same], bits(o0)[same]) and torch.equal(lse[same], lse0[same])
    assert torch.isnan(o[11, 3].float()).all() and torch.isnan(o[71, 5].float()).all()


def test_one_sequence_captured_and_replayed_with_fewer_tokens():
    """A graph for up to 40 tokens of one sequence, with lists and without, replayed with 40, 3 and none."""
    b = ref.make([40], [600], H=8, H_kv=2, D=128, page=64, seed=97)
    c = f4.Cache(b, 97)
    q = ref.rows(b, 8, 98)
    sel, cnt, want = lists_for(b, np.random.default_rng(99), 4)
    o, lse = torch.empty_like(q), torch.empty((40, 8), device="cuda")
    o2, lse2 = torch.empty_like(q), torch.empty((40, 8), device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        bsa.forward_paged_fp4(q, *c.arrays(), *b.arrays(), o, lse)
        bsa.forward_paged_fp4(q, *c.arrays(), *b.arrays(), o2, lse2, sel=sel, sel_cnt=cnt)
    for n in (40, 3, 0, 40):
        b.q_start.copy_(torch.tensor([0, n], dtype=torch.int32))
        b.new = [n]
        for x in (o, o2, lse, lse2):
            x.fill_(7.0)
        graph.replay()
        status_ok()
        if n:
            f4.check_attention(b, q, o, lse)
            f4.check_attention(b, q, o2, lse2, sel=want)
        for x in (o, o2, lse, lse2):
            assert (x[n:] == 7.0).all()
