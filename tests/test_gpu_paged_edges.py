"""Paged cache: scores of any magnitude, thread blocks with several runs of
work, long waits, and first calls from several threads, against fp64 (bounds
as in paged_ref)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import long_context_mask_gb300 as bsa
import paged_ref as ref
from gpu_util import status_ok
from test_gpu_paged import bits, check_select, lists_for, mean_keys, run_forward, run_select

pytestmark = pytest.mark.gpu
BOUNDS, TIMEOUT = 6, 5


# ------------------------------------------------------------------ selection

@pytest.mark.parametrize("kind", ["equal", "steps", "close", "shuffled"])
@pytest.mark.parametrize("q_exp,m_exp", [(0, -76), (0, -80), (-80, 0), (-50, -50), (0, -100), (-90, 60), (70, 70)])
def test_close_and_equal_scores_of_any_magnitude(kind, q_exp, m_exp):
    """Powers of two change no order: the lists are those of the unscaled scores.
    shuffled: the same values in another order against a query of equal ones, so
    that the exact scores are equal and their fp32 sums are not."""
    b = ref.make([30], [128 * 400 + 7], H=4, H_kv=2, D=128, page=128, seed=54, poison=False)
    q, km = ref.rows(b, 4, 55), mean_keys(b, 56)
    at = b.table[0].long()
    if kind == "steps":
        for j in range(400):
            km[at[j]] = km[at[j % 9]]
    else:
        km[:] = km[0]
    if kind == "shuffled":
        q[:] = q[..., :1].clone()
        g = torch.Generator().manual_seed(59)
        for j in range(400):
            km[at[j]] = km[at[j]][:, torch.randperm(128, generator=g).cuda()]
    if kind == "close":
        q[..., 5] = 2.0 ** -22
        for j in range(400):
            km[at[j], :, 5] = 1.0 + (j * 37 % 101) / 128
    kw = dict(topk=16, sink_blocks=1, local_blocks=1)
    want = ref.select(b, q, km, *kw.values())
    q, km = q * 2.0 ** q_exp, km * 2.0 ** m_exp
    assert q.isfinite().all() and km.isfinite().all()
    sel, cnt = run_select(b, q, km, **kw)
    status_ok()
    for t in range(30):
        for h in range(2):
            assert sel[t, h].tolist() == want[t][h] and int(cnt[t, h]) == 18, (t, h)


# ------------------------------------------------------------------ first calls

FIRST_CALLS = """
import sys, threading
sys.path[:0] = [{root!r}, {tests!r}]
import torch, paged_ref as ref, long_context_mask_gb300 as bsa
n = 8
bs = [ref.make([1, 40], [900, 300], H=8, H_kv=2, D=64 + 64 * (x % 2), page=64, seed=x, poison=False) for x in range(n)]
qs = [ref.rows(b, 8, 1) for b in bs]
outs = [(torch.empty_like(q), torch.empty((41, 8), device="cuda"), torch.empty((41, 2, 6), dtype=torch.int32, device="cuda"),
         torch.empty((41, 2), dtype=torch.int32, device="cuda")) for q in qs]
kms = [torch.randn((b.n_pages, 2, b.D), device="cuda").to(torch.bfloat16) for b in bs]
streams = [torch.cuda.Stream() for _ in bs]
failed, together = [], threading.Barrier(n)
torch.cuda.synchronize()
bsa.load_library()

def go(x):
    b, q, (o, lse, sel, cnt) = bs[x], qs[x], outs[x]
    try:
        with torch.cuda.stream(streams[x]):
            together.wait()
            bsa.select_paged(q, kms[x], *b.arrays(), sel, cnt, page_size=64, topk=4)
            bsa.forward_paged(q, b.k_cache, b.v_cache, *b.arrays(), o, lse)
    except Exception as e:
        failed.append(e)

threads = [threading.Thread(target=go, args=(x,)) for x in range(n)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not failed, failed
assert bsa.device_status() == 0
for b, q, km, (o, lse, sel, cnt) in zip(bs, qs, kms, outs):
    ref.check_attention(b, q, o, lse)
    want = ref.select(b, q, km, 4, 1, 1)
    assert all(sel[t, h, :len(want[t][h])].tolist() == want[t][h] for t in range(41) for h in range(2))
"""


def test_first_calls_from_several_threads_at_once():
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALLS.format(root=os.path.dirname(tests), tests=tests)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=240)
    assert r.returncode == 0, r.stderr[-2000:]


# ------------------------------------------------------------------ long waits

def wait_selftest(kind):
    ns = torch.zeros(2, dtype=torch.int64, device="cuda")
    bsa.selftest_paged_wait(kind, ns)
    return bsa.device_status(), (ns.double() * 1e-6).tolist()


def test_a_wait_for_what_never_comes_ends():
    status_ok()
    st, ms = wait_selftest(bsa.PAGED_WAIT_NOTHING)
    assert st == TIMEOUT and -1000 < ms[0] <= -2
    status_ok()


def test_a_wait_for_what_goes_on_goes_on():
    """Progress is noted all the time, between the waiting warp's looks at clock and note too."""
    for _ in range(3):
        st, ms = wait_selftest(bsa.PAGED_WAIT_BUSY)
        assert st == 0 and 50 <= ms[0] < 1000


@pytest.mark.parametrize("before", [0, BOUNDS])
def test_a_time_out_is_told_whatever_was_to_be_told_before(before):
    """It ends the block's other waits, and takes the place of a code that means less."""
    status_ok()
    if before:
        b = ref.make([1], [40], H=1, H_kv=1, D=64, page=32, seed=1, poison=False)
        b.kv_len.fill_(-1)
        run_forward(b, ref.rows(b, 1, 2))                 # (BOUNDS: nothing is read through a bad length)
    st, ms = wait_selftest(bsa.PAGED_WAIT_TWO)
    assert st == TIMEOUT
    assert -500 < ms[0] <= -2 and -500 < ms[1] <= -2
    status_ok()


@pytest.mark.parametrize("behind", [1, 1000])
def test_short_sequences_behind_rows_that_take_long(behind):
    """Each thread block's run is a sequence of 2^19 keys, whose rows are computed from their own
    keys for more than a second, and two short ones: whoever waits for those rows has not lost its
    time.  behind 1: all scores of the run are there early, and their issuer waits for the last product."""
    n, L, S = 128, 1 << 19, min(152, torch.cuda.get_device_properties(0).multi_processor_count)
    dev = "cuda"
    k = torch.zeros((L // 128, 1, 128, 64), dtype=torch.bfloat16, device=dev)
    v = torch.ones_like(k)
    v[0, 0, 0, 0] = float("inf")       # every long row's O is not finite,
    v[-1, 0, -1, 1] = float("nan")     # and this one all but the last do not see
    table = torch.full((3 * S, L // 128), -1, dtype=torch.int32, device=dev)
    table[::3] = torch.arange(L // 128, dtype=torch.int32, device=dev)
    pages = (behind + 127) // 128
    table[1::3, :pages] = table[2::3, :pages] = torch.arange(1, 1 + pages, dtype=torch.int32, device=dev)
    new = torch.tensor([n, 1, 1], dtype=torch.int32).repeat(S)
    start = torch.cat([torch.zeros(1, dtype=torch.int32), new.cumsum(0).to(torch.int32)]).to(dev)
    length = torch.tensor([L, behind, behind], dtype=torch.int32, device=dev).repeat(S)
    q = torch.randn((S * (n + 2), 1, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(dev)
    o, lse = torch.empty_like(q), torch.empty((S * (n + 2), 1), device=dev)
    bsa.forward_paged(q, k, v, table, start, length, o, lse)
    status_ok()
    want = torch.ones((S, n + 2, 64), device=dev)
    want[:, :n, 0] = float("inf")
    want[:, n - 1, 1] = float("nan")
    got = o.view(S, n + 2, 64).float()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
    fin = want.isfinite()
    assert ((got - want)[fin].abs() <= 2.0 ** -7).all()
    keys = torch.cat([torch.arange(L - n + 1, L + 1), torch.full((2,), behind)]).double().to(dev)
    # a sum of ones in fp32, at most 2^19: exact; a logarithm and a product
    assert ((lse.view(S, n + 2).double() - keys.log()).abs() <= 8 * 2.0 ** -24 * (1 + keys.log())).all()


# ------------------------------------------------------------------ several runs a thread block

def runs_per_block(b, window=0, sinks=0, causal=True, sel=None):
    """How many runs of work a thread block of the attention takes: a batch whose key tiles are
    read more than twice and hold more than 64 MB is gone through in up to four phases."""
    tpt, grid = 128 // (b.H // b.H_kv), min(152, torch.cuda.get_device_properties(0).multi_processor_count)
    starts = b.q_start.tolist()
    tiles = pairs = cache = 0
    for s, (n, length) in enumerate(zip(b.new, b.length)):
        cache += (length + 127) // 128 * b.H_kv if n else 0
        for t in range(0, n, tpt):
            pos, last = length - n + t, length - n + min(t + tpt, n) - 1
            tiles += b.H_kv
            if sel is not None:
                toks = range(starts[s] + t, starts[s] + min(t + tpt, n))
                pairs += sum(max(1, len({x for i in toks for x in sel[i][h] if 128 * x <= length - n + i - starts[s]}))
                             for h in range(b.H_kv))
                continue
            hi = last // 128 + 1 if causal else (length + 127) // 128
            lo = min(max(pos - window + 1, 0) // 128, hi) if window else 0
            pairs += b.H_kv * (hi - lo + (min((min(sinks, last + 1) + 127) // 128, lo) if window else 0))
    units, size = pairs + 4 * tiles, cache * 128 * b.D * 4
    if size <= 64 << 20 or pairs <= 2 * cache:
        return 1
    return min(4, -(-size // (64 << 20)), max(units // (16 * grid), 1))


def check_heads(b, q, o, lse, kv_heads, sel=None, **kw):
    """Some key/value heads against fp64."""
    G = b.H // b.H_kv
    for h in kv_heads:
        one = ref.Batch(b.new, b.length, G, 1, b.D, b.page, "cuda", table=b.table, q_start=b.q_start, kv_len=b.kv_len,
                        k_cache=b.k_cache[:, h:h + 1], v_cache=b.v_cache[:, h:h + 1], n_pages=b.n_pages, tokens=b.tokens)
        x = slice(h * G, (h + 1) * G)
        ref.check_attention(one, q[:, x], o[:, x], lse[:, x], sel=None if sel is None else [[t[h]] for t in sel], **kw)


LARGE = {
    # many chunks over caches of their own, some sequences without a new token
    "batch": (4, dict(new=[89, 0, 90, 1, 70] * 15, length=[989, 300, 1000, 900, 1100] * 15, H=40, H_kv=8, D=128, page=32), {}),
    "chunk": (3, dict(new=[1000], length=[36007], H=32, H_kv=8, D=128, page=128), {}),
    "two": (2, dict(new=[400, 500], length=[12000, 9100], H=32, H_kv=8, D=128, page=16), {}),
    "window": (3, dict(new=[2000] * 6, length=[3001] * 6, H=64, H_kv=16, D=128, page=64), dict(window=1000, sinks=130)),
    "all": (2, dict(new=[300, 200], length=[80000, 60001], H=14, H_kv=2, D=64, page=128), dict(causal=False)),
    "lists": (2, dict(new=[128, 40, 128, 128, 128], length=[40000, 40001, 39000, 41000, 128 * 300], H=14, H_kv=2, D=64, page=16),
              "lists"),
}


@pytest.mark.parametrize("name", LARGE)
def test_several_runs_to_a_thread_block(name):
    """Batches whose key tiles are read by many query tiles and do not stay in L2."""
    runs, shape, kw = LARGE[name]
    b = ref.make(**shape, seed=130, poison=False)
    q, sel = ref.rows(b, b.H, 131), None
    if kw == "lists":
        s, c, sel = lists_for(b, np.random.default_rng(132), 100)
        kw = dict(sel=s, sel_cnt=c)
        assert runs_per_block(b, sel=sel) == runs
    else:
        assert runs_per_block(b, **kw) == runs
    o, lse = run_forward(b, q, **kw)
    status_ok()
    check_heads(b, q, o, lse, sorted({0, b.H_kv // 2, b.H_kv - 1}), sel,
                **{k: v for k, v in kw.items() if k in ("causal", "window", "sinks")})
    # every head: the same rows in a batch of one head (one run to a block, other cuts), within both bounds
    o2, lse2 = run_forward(b, q, **kw)
    assert torch.equal(bits(o), bits(o2)) and torch.equal(lse, lse2)
    G = b.H // b.H_kv
    for h in range(b.H_kv):
        x = slice(h * G, (h + 1) * G)
        oh, lh = torch.empty_like(o[:, x].contiguous()), torch.empty((b.tokens, G), device="cuda")
        k1 = dict(kw)
        if sel is not None:
            k1.update(sel=kw["sel"][:, h:h + 1].contiguous(), sel_cnt=kw["sel_cnt"][:, h:h + 1].contiguous())
        bsa.forward_paged(q[:, x].contiguous(), b.k_cache[:, h:h + 1].contiguous(), b.v_cache[:, h:h + 1].contiguous(),
                          *b.arrays(), oh, lh, **k1)
        # both sides within check_attention's bounds: weights rounded to bf16 (A is at most the
        # largest |v|, below 8), O itself, and in fp32 d = (D + 16) 2^-24 (R + 1) < 2^-12, R < 27
        far = 2 * 1.01 * 2.0 ** -8 * (b.v_cache.abs().max().float() + oh.float().abs()) + 2.0 ** -7
        assert ((o[:, x].float() - oh.float()).abs() <= far).all()
        fin = torch.isfinite(lh)
        assert torch.equal(torch.isfinite(lse[:, x]), fin) and ((lse[:, x] - lh).abs()[fin] <= 2.0 ** -10).all()
    status_ok()


# ------------------------------------------------------------------ values that are not finite and seen

def elapsed(f, n=5):
    f()
    times = []
    for _ in range(n):
        a, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        e.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(e))
    return sorted(times)[n // 2]


@pytest.mark.parametrize("kw", [{}, dict(window=1500, sinks=100), "lists"])
def test_a_value_that_all_rows_see_costs_no_time(kw):
    """Rows next to hidden values that are not finite are computed key by key, which takes some
    hundred times as long; one bad value in the far past, which every row sees, is not such a case."""
    S = 16  # (enough for whole rows in a thread block's run)
    b = ref.make([250] * S, [4250 + 64 * s for s in range(S)], H=8, H_kv=2, D=128, page=64, seed=140, poison=False)
    q = ref.rows(b, 8, 141)
    if kw == "lists":
        sel, cnt, _ = lists_for(b, np.random.default_rng(142), 12)
        sel[..., 0] = 0
        kw = dict(sel=sel.clamp(min=0), sel_cnt=cnt.clamp(min=1))
    clean = elapsed(lambda: run_forward(b, q, **kw))
    o0, lse0 = run_forward(b, q, **kw)
    pos = 7 if kw else 3000
    b.v_cache[b.table[:, pos // 64].long(), :, pos % 64, 5] = float("nan")
    b.v_cache[b.table[:, pos // 64].long(), :, pos % 64, 9] = float("inf")
    took = elapsed(lambda: run_forward(b, q, **kw))
    o, lse = run_forward(b, q, **kw)
    status_ok()
    assert torch.isnan(o[:, :, 5]).all() and torch.isinf(o[:, :, 9]).all()
    rest = torch.ones(128, dtype=torch.bool, device="cuda")
    rest[5] = rest[9] = False
    assert torch.equal(bits(o)[..., rest], bits(o0)[..., rest]) and torch.equal(lse, lse0)
    assert took < 5 * clean + 0.1, (took, clean)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("place", [70, 127, 1079, 1080, 1081, 1150, 1199, 1381, 1400, 1499])
@pytest.mark.parametrize("H,K,D,page", [(4, 2, 128, 32), (14, 2, 64, 128)])
def test_one_bad_value_at_an_edge_of_what_rows_see(H, K, D, page, place, causal):
    """Behind the sinks, before and within the windows' first keys, behind the rows' own positions:
    each alone, so that each edge is looked at for itself."""
    window, sinks = 300, 70
    b = ref.make([120, 33], [1500, 700], H=H, H_kv=K, D=D, page=page, seed=150, poison=False)
    q = ref.rows(b, H, 151)
    kw = dict(causal=causal, window=window, sinks=sinks)
    o0, lse0 = run_forward(b, q, **kw)
    good = b.v_cache.clone()
    b.v_cache[b.table[0, place // page], :, place % page, 3] = float("nan")
    o, lse = run_forward(b, q, **kw)
    status_ok()
    p = torch.arange(1380, 1500, device="cuda")
    sees = ((place <= p) | (not causal)) & ((place > p - window) | (place < sinks))
    hit = torch.cat([sees, torch.zeros(33, dtype=torch.bool, device="cuda")])
    assert torch.isnan(o[hit][:, :, 3]).all() and torch.isfinite(o[~hit].float()).all()
    b.v_cache = good
    o[hit] = o0[hit]
    ref.check_attention(b, q, o, lse, **kw)
