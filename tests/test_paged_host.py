"""The paged cache calls' host checks: sizes and pointers through the C ABI,
shapes, strides, types and devices through the binding (no GPU)."""
import ctypes

import pytest
import torch

import long_context_mask_gb300 as bsa
from long_context_mask_gb300 import build as bsa_build
from long_context_mask_gb300.binding import PagedBatch

FAKE = 0x10000  # never dereferenced: the calls below fail validation first
ODD = 0x10002
OK, INVALID, UNSUPPORTED = 0, 1, 2
CUDA_STEP = "expected a CUDA tensor"


@pytest.fixture(scope="module")
def lib():
    bsa_build.build()
    return bsa.load_library()


def batch(**kw):
    a = dict(page_table=FAKE, q_start=FAKE, kv_len=FAKE, seqs=3, tokens=10, max_pages=8, page_size=32, n_pages=40)
    a.update(kw)
    return PagedBatch(*a.values())


def append(lib, b=None, **kw):
    a = dict(q=FAKE, qs=1024, k=FAKE, ks=512, v=FAKE, vs=512, H=8, H_kv=4, D=128, rope=FAKE, rope_len=64, rot=128,
             inter=0, qn=FAKE, kn=FAKE, eps=1e-6, qo=FAKE, qos=1024, kc=FAKE, vc=FAKE, km=FAKE, stream=None)
    a.update(kw)
    b = batch() if b is None else b
    return lib.bsa_paged_append(ctypes.byref(b), *a.values())


def forward(lib, b=None, **kw):
    a = dict(q=FAKE, qs=1024, kc=FAKE, vc=FAKE, H=8, H_kv=4, D=128, causal=1, window=0, sinks=0, sel=None, cnt=None,
             width=0, scale=0.0, ws=FAKE, nbytes=1 << 40, o=FAKE, lse=FAKE, stream=None)
    a.update(kw)
    b = batch() if b is None else b
    return lib.bsa_forward_paged(ctypes.byref(b), *a.values())


def select(lib, b=None, **kw):
    a = dict(q=FAKE, qs=1024, km=FAKE, H=8, H_kv=4, D=128, topk=4, sink=1, local=1, ws=FAKE, nbytes=1 << 40, sel=FAKE,
             cnt=FAKE, width=6, stream=None)
    a.update(kw)
    b = batch() if b is None else b
    return lib.bsa_select_paged(ctypes.byref(b), *a.values())


@pytest.mark.parametrize("call", [append, forward, select])
def test_sizes_that_every_call_rejects(lib, call):
    assert call(lib, D=96) == UNSUPPORTED
    assert call(lib, batch(page_size=24)) == UNSUPPORTED
    assert call(lib, batch(page_size=256)) == UNSUPPORTED
    assert call(lib, H=9) == INVALID                                  # H_kv does not divide H
    assert call(lib, H_kv=0) == INVALID
    assert call(lib, H=2, H_kv=4) == INVALID
    assert call(lib, H=129, H_kv=1) == INVALID                        # more than 128 heads to a tile row
    assert call(lib, H=70000, H_kv=70000) == INVALID
    assert call(lib, batch(seqs=-1)) == INVALID
    assert call(lib, batch(seqs=16385)) == INVALID
    assert call(lib, batch(tokens=-1)) == INVALID
    assert call(lib, batch(tokens=(1 << 24) + 1)) == INVALID
    assert call(lib, batch(tokens=1 << 24), H=128, H_kv=128) == INVALID   # tokens * H
    assert call(lib, batch(max_pages=0)) == INVALID
    assert call(lib, batch(max_pages=(1 << 19) + 1)) in (INVALID, UNSUPPORTED)
    assert call(lib, batch(n_pages=0)) == INVALID
    assert call(lib, batch(n_pages=1 << 24)) == INVALID               # slots of the cache in 32 bits
    for gone in ("page_table", "q_start", "kv_len"):
        assert call(lib, batch(**{gone: None})) == INVALID
        assert call(lib, batch(**{gone: ODD})) == INVALID
    assert call(lib, q=ODD) == INVALID
    assert call(lib, qs=1020) == INVALID                              # not a multiple of 8
    assert call(lib, qs=1016) == INVALID                              # shorter than a token


@pytest.mark.parametrize("call", [append, forward, select])
def test_nothing_to_do_is_fine(lib, call):
    assert call(lib, batch(seqs=0)) == OK
    assert call(lib, batch(tokens=0, page_table=None, q_start=None, kv_len=None)) == OK


@pytest.mark.parametrize("call", [append, forward, select])
def test_null_batch(lib, call):
    fn = {append: lib.bsa_paged_append, forward: lib.bsa_forward_paged, select: lib.bsa_select_paged}[call]
    args = {append: [FAKE, 1024, FAKE, 512, FAKE, 512, 8, 4, 128, None, 0, 0, 0, None, None, 0.0, FAKE, 1024, FAKE, FAKE, None, None],
            forward: [FAKE, 1024, FAKE, FAKE, 8, 4, 128, 1, 0, 0, None, None, 0, 0.0, FAKE, 1 << 40, FAKE, FAKE, None],
            select: [FAKE, 1024, FAKE, 8, 4, 128, 4, 1, 1, FAKE, 1 << 40, FAKE, FAKE, 6, None]}[call]
    assert fn(None, *args) == INVALID


def test_append_rejects(lib):
    for bad in (dict(rope_len=0), dict(rot=0), dict(rot=24), dict(rot=144), dict(rope=ODD), dict(inter=2),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(qn=ODD), dict(kn=ODD),
                dict(k=None), dict(v=None), dict(k=ODD), dict(ks=504), dict(vs=500), dict(qo=None), dict(qo=ODD),
                dict(qos=1000), dict(qos=2048), dict(kc=None), dict(vc=None), dict(kc=ODD), dict(vc=ODD), dict(km=ODD)):
        assert append(lib, **bad) == INVALID, bad


def test_forward_rejects(lib):
    nan, inf = float("nan"), float("inf")
    for bad in (dict(causal=2), dict(window=-1), dict(sinks=-1), dict(scale=nan), dict(scale=inf),
                dict(sel=FAKE, width=4), dict(sel=FAKE, cnt=FAKE, width=0), dict(width=4),
                dict(sel=FAKE, cnt=FAKE, width=4, window=64), dict(sel=ODD, cnt=FAKE, width=4),
                dict(sel=FAKE, cnt=ODD, width=4), dict(kc=None), dict(vc=None), dict(o=None), dict(lse=None),
                dict(ws=None), dict(ws=ODD), dict(o=ODD), dict(lse=ODD), dict(kc=ODD), dict(vc=ODD)):
        assert forward(lib, **bad) == INVALID, bad
    need = lib.bsa_forward_paged_workspace_size(ctypes.byref(batch()), 8, 4, 128, 0)
    assert need > 0 and forward(lib, nbytes=need - 1) == INVALID
    more = lib.bsa_forward_paged_workspace_size(ctypes.byref(batch()), 8, 4, 128, 6)
    assert more > need and forward(lib, sel=FAKE, cnt=FAKE, width=6, nbytes=more - 1) == INVALID
    assert lib.bsa_forward_paged_workspace_size(ctypes.byref(batch()), 9, 4, 128, 0) == 0
    assert lib.bsa_forward_paged_workspace_size(None, 8, 4, 128, 0) == 0


def test_select_rejects(lib):
    for bad in (dict(topk=-1), dict(sink=-1), dict(local=0), dict(width=5), dict(width=0), dict(topk=2 ** 31 - 1),
                dict(km=None), dict(km=ODD), dict(sel=None), dict(cnt=None), dict(sel=ODD), dict(cnt=ODD)):
        assert select(lib, **bad) == INVALID, bad
    assert select(lib, batch(max_pages=32769)) == UNSUPPORTED          # more than 2^20 positions
    need = lib.bsa_select_paged_workspace_size(ctypes.byref(batch()), 8, 4, 128)
    if need:
        assert select(lib, nbytes=need - 1) == INVALID


# ------------------------------------------------------------------ the binding

def accepted(fn, *a, **kw):
    with pytest.raises(ValueError, match=CUDA_STEP):
        fn(*a, **kw)


def rejected(fn, *a, **kw):
    with pytest.raises((ValueError, TypeError)) as e:
        fn(*a, **kw)
    assert CUDA_STEP not in str(e.value)


def bf16(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def f32(*s):
    return torch.zeros(s)


T, H, K, D, P, PAGES, S = 10, 8, 4, 128, 32, 40, 3


def paged():
    return dict(k_cache=bf16(PAGES, K, P, D), v_cache=bf16(PAGES, K, P, D), page_table=i32(S, 8), q_start=i32(S + 1),
                kv_len=i32(S))


def call_append(**kw):
    a = dict(k=bf16(T, K, D), v=bf16(T, K, D), **paged(), q=bf16(T, H, D), q_out=bf16(T, H, D), rope=f32(64, 128))
    a.update(kw)
    bsa.paged_append(a.pop("k"), a.pop("v"), a.pop("k_cache"), a.pop("v_cache"), a.pop("page_table"),
                     a.pop("q_start"), a.pop("kv_len"), **a)


def call_forward(**kw):
    a = dict(q=bf16(T, H, D), **paged(), o=bf16(T, H, D), lse=f32(T, H))
    a.update(kw)
    bsa.forward_paged(a.pop("q"), a.pop("k_cache"), a.pop("v_cache"), a.pop("page_table"), a.pop("q_start"),
                      a.pop("kv_len"), a.pop("o"), a.pop("lse"), **a)


def call_select(**kw):
    a = dict(q=bf16(T, H, D), k_mean=bf16(PAGES, K, D), page_table=i32(S, 8), q_start=i32(S + 1), kv_len=i32(S),
             sel=i32(T, K, 6), sel_cnt=i32(T, K), page_size=P, topk=4)
    a.update(kw)
    bsa.select_paged(a.pop("q"), a.pop("k_mean"), a.pop("page_table"), a.pop("q_start"), a.pop("kv_len"),
                     a.pop("sel"), a.pop("sel_cnt"), **a)


@pytest.mark.parametrize("kw", [{}, dict(q=None, q_out=None), dict(rope=None), dict(q_norm=bf16(D), k_norm=bf16(D)),
                                dict(k_mean=bf16(PAGES, K, D)), dict(q=bf16(T, H + 2 * K, D)[:, :H]),
                                dict(k=bf16(T, H + 2 * K, D)[:, H:H + K])])
def test_append_takes_the_documented_calls(lib, kw):
    accepted(call_append, **kw)


@pytest.mark.parametrize("kw", [
    dict(k=f32(T, K, D)), dict(k=bf16(T, K + 1, D)), dict(v=bf16(T + 1, K, D)), dict(q_out=None), dict(q=bf16(T + 1, H, D)),
    dict(q_out=bf16(T, H, D // 2)), dict(k=bf16(T, K, 2 * D)[..., ::2]), dict(k=bf16(K, T, D).transpose(0, 1)),
    dict(rope=torch.zeros((64, 128), dtype=torch.float64)), dict(rope=f32(64)), dict(q_norm=bf16(D - 1)),
    dict(k_norm=f32(D)), dict(k_mean=bf16(PAGES, K, D - 1)), dict(k_mean=f32(PAGES, K, D)),
    dict(v_cache=bf16(PAGES, K, P, D // 2)), dict(k_cache=f32(PAGES, K, P, D)), dict(page_table=i32(8)),
    dict(page_table=torch.zeros((S, 8), dtype=torch.int64)), dict(q_start=i32(S)), dict(kv_len=i32(S - 1)),
    dict(kv_len=torch.zeros(S, dtype=torch.int32, device="meta"))])
def test_append_refuses(lib, kw):
    rejected(call_append, **kw)


@pytest.mark.parametrize("kw", [{}, dict(sel=i32(T, K, 6), sel_cnt=i32(T, K)), dict(q=bf16(T, H + 2, D)[:, :H]),
                                dict(causal=False, window=64, sinks=4)])
def test_forward_takes_the_documented_calls(lib, kw):
    accepted(call_forward, **kw)


@pytest.mark.parametrize("kw", [
    dict(q=f32(T, H, D)), dict(q=bf16(H, D)), dict(o=f32(T, H, D)), dict(o=bf16(T, H, D // 2)), dict(lse=f32(T, H - 1)),
    dict(sel=i32(T, K, 6)), dict(sel_cnt=i32(T, K)), dict(sel=i32(T - 1, K, 6), sel_cnt=i32(T, K)),
    dict(sel=i32(T, H, 6), sel_cnt=i32(T, H)), dict(sel=i32(T, K, 6), sel_cnt=i32(T, K - 1)),
    dict(sel=torch.zeros((T, K, 6), dtype=torch.int64), sel_cnt=i32(T, K)), dict(q_start=i32(S)),
    dict(workspace=torch.zeros(16, dtype=torch.uint8, device="meta"))])
def test_forward_refuses(lib, kw):
    rejected(call_forward, **kw)


@pytest.mark.parametrize("kw", [{}, dict(q=bf16(T, H + 2, D)[:, :H]), dict(sel=i32(T + 4, K, 9))])
def test_select_takes_the_documented_calls(lib, kw):
    accepted(call_select, **kw)


@pytest.mark.parametrize("kw", [
    dict(q=f32(T, H, D)), dict(q=bf16(T, H, D // 2)), dict(k_mean=f32(PAGES, K, D)), dict(k_mean=bf16(PAGES, K * D)),
    dict(sel=i32(T, H, 6)), dict(sel=i32(T, K * 6)), dict(sel_cnt=i32(T, K - 1)), dict(kv_len=i32(S - 1))])
def test_select_refuses(lib, kw):
    rejected(call_select, **kw)


def test_lists_of_any_use_fit(lib):
    """Lists are at most 2^20 entries wide."""
    assert forward(lib, sel=FAKE, cnt=FAKE, width=(1 << 20) + 1) == INVALID
    assert lib.bsa_forward_paged_workspace_size(ctypes.byref(batch()), 8, 4, 128, (1 << 20) + 1) == 0
    assert lib.bsa_forward_paged_workspace_size(ctypes.byref(batch()), 8, 4, 128, 1 << 20) > 0


@pytest.mark.parametrize("call", [append, forward, select])
def test_heads_fit_the_launches(lib, call):
    """A launch has a thread block for each group of heads along one axis, of at most 65535."""
    assert call(lib, batch(tokens=0), H=16384, H_kv=16384) == OK
    assert call(lib, batch(tokens=0), H=16385, H_kv=16385) == INVALID


# ------------------------------------------------------------------ other ranks, numbers that do not fit

@pytest.mark.parametrize("kw", [dict(q=bf16(T)), dict(q=bf16(T * H * D)), dict(q=bf16(T, H * D)), dict(q_out=bf16(T)),
                                dict(k=bf16(T)), dict(k=torch.zeros((), dtype=torch.bfloat16)), dict(v=bf16(T * K, D))])
def test_append_refuses_other_ranks(lib, kw):
    rejected(call_append, **kw)


@pytest.mark.parametrize("call,kw", [
    (call_forward, dict(window=1 << 32)), (call_forward, dict(window=(1 << 32) + 575, sinks=64)),
    (call_forward, dict(window=64, sinks=1 << 31)), (call_forward, dict(sinks=-(1 << 32))),
    (call_select, dict(topk=(1 << 32) + 4)), (call_select, dict(sink_blocks=1 << 32)),
    (call_select, dict(local_blocks=(1 << 32) + 1)), (call_select, dict(page_size=(1 << 32) + P))])
def test_numbers_beyond_32_bits_are_not_cut(lib, call, kw):
    """(cut to 32 bits they would be another window, another number of blocks)"""
    rejected(call, **kw)


def test_workspace_sizes_of_numbers_beyond_32_bits(lib):
    sizes = dict(seqs=S, tokens=T, max_pages=8, page_size=P, H=H, H_kv=K, D=D)
    assert bsa.forward_paged_workspace_size(**sizes) > 0 and bsa.select_paged_workspace_size(**sizes) > 0
    for name in sizes:
        for fn in (bsa.forward_paged_workspace_size, bsa.select_paged_workspace_size):
            with pytest.raises(ValueError):
                fn(**{**sizes, name: sizes[name] + (1 << 32)})
    with pytest.raises(ValueError):
        bsa.forward_paged_workspace_size(**sizes, sel_width=1 << 32)
