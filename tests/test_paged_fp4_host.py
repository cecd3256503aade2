"""Host checks of the calls on a cache in 4 bits: sizes and pointers through the
C ABI, shapes, strides, types and devices through the binding (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import long_context_mask_gb300 as bsa
from long_context_mask_gb300.binding import Fp4Cache
from test_paged_host import (FAKE, INVALID, ODD, OK, UNSUPPORTED, accepted, batch, bf16, f32, i32, lib, rejected)  # noqa: F401

SIXTEEN = 0x10010


def cache(**kw):
    a = dict(k=FAKE, k_scale=FAKE, v=FAKE, v_scale=SIXTEEN, k_gain=None, v_gain=None)
    a.update(kw)
    return Fp4Cache(*a.values())


def append(lib, b=None, c=None, **kw):
    a = dict(q=FAKE, qs=1024, k=FAKE, ks=512, v=FAKE, vs=512, H=8, H_kv=4, D=128, rope=FAKE, rope_len=64, rot=128,
             inter=0, qn=FAKE, kn=FAKE, eps=1e-6, qo=FAKE, qos=1024)
    km = kw.pop("km", FAKE)
    a.update(kw)
    b, c = batch() if b is None else b, cache() if c is None else c
    return lib.bsa_paged_append_fp4(ctypes.byref(b), *a.values(), ctypes.byref(c), km, None)


def read(lib, b=None, c=None, **kw):
    a = dict(H_kv=4, D=128)
    o = dict(ko=FAKE, ks=512, vo=FAKE, vs=512)
    for x in kw:
        (a if x in a else o)[x] = kw[x]
    b, c = batch() if b is None else b, cache() if c is None else c
    return lib.bsa_paged_read_fp4(ctypes.byref(b), *a.values(), ctypes.byref(c), *o.values(), None)


def forward(lib, b=None, c=None, **kw):
    a = dict(H=8, H_kv=4, D=128, causal=1, window=0, sinks=0, sel=None, cnt=None, width=0, scale=0.0, max_new=0, ws=FAKE,
             nbytes=1 << 50, o=FAKE, lse=FAKE)
    q, qs = kw.pop("q", FAKE), kw.pop("qs", 1024)
    a.update(kw)
    b, c = batch() if b is None else b, cache() if c is None else c
    return lib.bsa_forward_paged_fp4(ctypes.byref(b), q, qs, ctypes.byref(c), *a.values(), None)


@pytest.mark.parametrize("call", [append, forward, read])
def test_sizes_that_every_call_rejects(lib, call):
    assert call(lib, D=96) == UNSUPPORTED
    assert call(lib, batch(page_size=24)) == UNSUPPORTED
    assert call(lib, H_kv=0) == INVALID
    assert call(lib, H_kv=16385, **({} if call is read else dict(H=16385))) == INVALID
    for kw in (dict(seqs=-1), dict(seqs=16385), dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(max_pages=0),
               dict(n_pages=0), dict(n_pages=1 << 24)):
        assert call(lib, batch(**kw)) == INVALID
    for gone in ("page_table", "q_start", "kv_len"):
        assert call(lib, batch(**{gone: None})) == INVALID
        assert call(lib, batch(**{gone: ODD})) == INVALID
    for part in ("k", "k_scale", "v", "v_scale"):
        assert call(lib, c=cache(**{part: None})) == INVALID
        assert call(lib, c=cache(**{part: ODD})) == INVALID
    for part in ("k_gain", "v_gain"):
        assert call(lib, c=cache(**{part: ODD})) == INVALID
    if call is not read:
        assert call(lib, H=9) == INVALID
        assert call(lib, H=129, H_kv=1) == INVALID
        assert call(lib, q=ODD) == INVALID and call(lib, qs=1020) == INVALID and call(lib, qs=1016) == INVALID


@pytest.mark.parametrize("call", [append, forward, read])
def test_nothing_to_do_is_fine(lib, call):
    assert call(lib, batch(seqs=0)) == OK
    assert call(lib, batch(tokens=0, page_table=None, q_start=None, kv_len=None)) == OK


def test_null_structs(lib):
    b, c = batch(), cache()
    rb, rc = ctypes.byref(b), ctypes.byref(c)
    front = [FAKE, 1024, FAKE, 512, FAKE, 512, 8, 4, 128, None, 0, 0, 0, None, None, 0.0, FAKE, 1024]
    assert lib.bsa_paged_append_fp4(None, *front, rc, None, None) == INVALID
    assert lib.bsa_paged_append_fp4(rb, *front, None, None, None) == INVALID
    assert lib.bsa_paged_read_fp4(None, 4, 128, rc, FAKE, 512, FAKE, 512, None) == INVALID
    assert lib.bsa_paged_read_fp4(rb, 4, 128, None, FAKE, 512, FAKE, 512, None) == INVALID
    back = [8, 4, 128, 1, 0, 0, None, None, 0, 0.0, 0, FAKE, 1 << 50, FAKE, FAKE, None]
    assert lib.bsa_forward_paged_fp4(None, FAKE, 1024, rc, *back) == INVALID
    assert lib.bsa_forward_paged_fp4(rb, FAKE, 1024, None, *back) == INVALID


def test_append_rejects(lib):
    for bad in (dict(rope_len=0), dict(rot=0), dict(rot=24), dict(rot=144), dict(rope=ODD), dict(inter=2),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(qn=ODD), dict(kn=ODD),
                dict(k=None), dict(v=None), dict(k=ODD), dict(ks=504), dict(vs=500), dict(qo=None), dict(qo=ODD),
                dict(qos=1000), dict(qos=2048), dict(km=ODD)):
        assert append(lib, **bad) == INVALID, bad


def test_read_rejects(lib):
    for bad in (dict(ko=ODD), dict(vo=ODD), dict(ks=504), dict(vs=516), dict(ko=None, vo=None)):
        assert read(lib, **bad) == INVALID, bad


def test_forward_rejects(lib):
    nan, inf = float("nan"), float("inf")
    for bad in (dict(causal=2), dict(window=-1), dict(sinks=-1), dict(scale=nan), dict(scale=inf), dict(max_new=-1),
                dict(sel=FAKE, width=4), dict(sel=FAKE, cnt=FAKE, width=0), dict(width=4),
                dict(sel=FAKE, cnt=FAKE, width=4, window=64), dict(sel=ODD, cnt=FAKE, width=4),
                dict(sel=FAKE, cnt=ODD, width=4), dict(sel=FAKE, cnt=FAKE, width=(1 << 20) + 1), dict(o=None),
                dict(lse=None), dict(ws=None), dict(ws=ODD), dict(o=ODD), dict(lse=ODD)):
        assert forward(lib, **bad) == INVALID, bad
    size = lib.bsa_forward_paged_fp4_workspace_size
    need = size(ctypes.byref(batch()), 8, 4, 128, 0)
    assert need > 0 and forward(lib, nbytes=need - 1) == INVALID
    more = size(ctypes.byref(batch()), 8, 4, 128, 6)
    assert more > need and forward(lib, sel=FAKE, cnt=FAKE, width=6, nbytes=more - 1) == INVALID
    assert size(ctypes.byref(batch()), 9, 4, 128, 0) == 0 and size(None, 8, 4, 128, 0) == 0
    assert size(ctypes.byref(batch()), 8, 4, 128, (1 << 20) + 1) == 0
    # lists of (tokens + sequences) * H_kv tiles are counted in 32 bits
    many = batch(seqs=16384, tokens=131000, n_pages=16)
    assert size(ctypes.byref(many), 16384, 16384, 64, 0) > 0 and size(ctypes.byref(many), 16384, 16384, 64, 1) == 0
    assert forward(lib, many, H=16384, H_kv=16384, D=64, qs=16384 * 64, sel=FAKE, cnt=FAKE, width=1) == INVALID


# ------------------------------------------------------------------ the binding

T, H, K, D, P, PAGES, S = 10, 8, 4, 128, 32, 40, 3


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def e4m3(*s):
    return u8(*s).view(torch.float8_e4m3fn)


def paged():
    return dict(k_cache=u8(PAGES, K, P, D // 2), k_scale=e4m3(PAGES, K, P, D // 16), v_cache=u8(PAGES, K, P, D // 2),
                v_scale=e4m3(PAGES, K, P, D // 16), page_table=i32(S, 8), q_start=i32(S + 1), kv_len=i32(S))


def call_append(**kw):
    a = dict(k=bf16(T, K, D), v=bf16(T, K, D), **paged(), q=bf16(T, H, D), q_out=bf16(T, H, D), rope=f32(64, 128))
    a.update(kw)
    bsa.paged_append_fp4(*[a.pop(x) for x in ("k", "v", *paged())], **a)


def call_read(**kw):
    a = dict(**paged(), k_out=bf16(T, K, D), v_out=bf16(T, K, D))
    a.update(kw)
    bsa.paged_read_fp4(*[a.pop(x) for x in paged()], **a)


def call_forward(**kw):
    a = dict(q=bf16(T, H, D), **paged(), o=bf16(T, H, D), lse=f32(T, H))
    a.update(kw)
    bsa.forward_paged_fp4(*[a.pop(x) for x in ("q", *paged(), "o", "lse")], **a)


CACHE_ERRORS = [
    dict(k_cache=bf16(PAGES, K, P, D)), dict(k_cache=u8(PAGES, K, P, D)), dict(v_cache=u8(PAGES, K, P)),
    dict(k_scale=u8(PAGES, K, P, D // 16)), dict(v_scale=e4m3(PAGES, K, P, D // 8)), dict(v_scale=e4m3(PAGES, K, P)),
    dict(v_scale=torch.zeros((PAGES, K, P, D // 16), dtype=torch.uint8).view(torch.float8_e5m2)),
    dict(k_gain=f32(K - 1)), dict(v_gain=bf16(K)), dict(k_cache=u8(PAGES, K, P, D)[..., ::2]),
    dict(k_gain=torch.zeros(K, device="meta")), dict(page_table=i32(8)), dict(q_start=i32(S)), dict(kv_len=i32(S - 1)),
    dict(page_table=torch.zeros((S, 8), dtype=torch.int64))]


@pytest.mark.parametrize("call", [call_append, call_read, call_forward])
@pytest.mark.parametrize("kw", CACHE_ERRORS)
def test_other_caches_are_refused(lib, call, kw):
    rejected(call, **kw)


@pytest.mark.parametrize("call", [call_append, call_read, call_forward])
def test_documented_caches_are_taken(lib, call):
    accepted(call)
    accepted(call, k_gain=f32(K), v_gain=f32(K + 1))
    accepted(call, v_gain=f32(K))


@pytest.mark.parametrize("kw", [dict(q=None, q_out=None), dict(rope=None), dict(q_norm=bf16(D), k_norm=bf16(D)),
                                dict(k_mean=bf16(PAGES, K, D)), dict(q=bf16(T, H + 2 * K, D)[:, :H]),
                                dict(k=bf16(T, H + 2 * K, D)[:, H:H + K])])
def test_append_takes_the_documented_calls(lib, kw):
    accepted(call_append, **kw)


@pytest.mark.parametrize("kw", [
    dict(k=f32(T, K, D)), dict(k=bf16(T, K + 1, D)), dict(v=bf16(T + 1, K, D)), dict(q_out=None), dict(q=bf16(T + 1, H, D)),
    dict(q_out=bf16(T, H, D // 2)), dict(rope=f32(64)), dict(q_norm=bf16(D - 1)), dict(k_norm=f32(D)),
    dict(k_mean=bf16(PAGES, K, D - 1)), dict(k_mean=f32(PAGES, K, D)), dict(k=bf16(T)), dict(q=bf16(T))])
def test_append_refuses(lib, kw):
    rejected(call_append, **kw)


@pytest.mark.parametrize("kw", [dict(k_out=None), dict(v_out=None), dict(k_out=bf16(T, K + 2, D)[:, 1:1 + K])])
def test_read_takes_the_documented_calls(lib, kw):
    accepted(call_read, **kw)


@pytest.mark.parametrize("kw", [dict(k_out=None, v_out=None), dict(k_out=f32(T, K, D)), dict(v_out=bf16(T + 1, K, D)),
                                dict(k_out=bf16(T, K * D)), dict(v_out=bf16(T, K, 2 * D)[..., ::2]), dict(k_out=bf16(T, H, D))])
def test_read_refuses(lib, kw):
    rejected(call_read, **kw)


@pytest.mark.parametrize("kw", [dict(sel=i32(T, K, 6), sel_cnt=i32(T, K)), dict(q=bf16(T, H + 2, D)[:, :H]),
                                dict(causal=False, window=64, sinks=4), dict(max_new=1)])
def test_forward_takes_the_documented_calls(lib, kw):
    accepted(call_forward, **kw)


@pytest.mark.parametrize("kw", [
    dict(q=f32(T, H, D)), dict(q=bf16(H, D)), dict(o=f32(T, H, D)), dict(o=bf16(T, H, D // 2)), dict(lse=f32(T, H - 1)),
    dict(sel=i32(T, K, 6)), dict(sel_cnt=i32(T, K)), dict(sel=i32(T - 1, K, 6), sel_cnt=i32(T, K)),
    dict(sel=i32(T, H, 6), sel_cnt=i32(T, H)), dict(workspace=torch.zeros(16, dtype=torch.uint8, device="meta")),
    dict(window=1 << 32), dict(window=64, sinks=1 << 31), dict(max_new=1 << 32), dict(max_new=(1 << 32) + 1)])
def test_forward_refuses(lib, kw):
    rejected(call_forward, **kw)


def test_workspace_sizes_of_numbers_beyond_32_bits(lib):
    sizes = dict(seqs=S, tokens=T, max_pages=8, page_size=P, H=H, H_kv=K, D=D)
    assert bsa.forward_paged_fp4_workspace_size(**sizes) > 0
    for name in sizes:
        with pytest.raises(ValueError):
            bsa.forward_paged_fp4_workspace_size(**{**sizes, name: sizes[name] + (1 << 32)})


# ------------------------------------------------------------------ quotients

def quotient(x, y):
    """The library's x / y: fp32 steps, each rounded once (a fused product and sum included)."""
    f32 = np.float32
    recip = f32(1) / y
    q = x * recip
    rest = f32(x.astype(np.longdouble) - q.astype(np.longdouble) * y.astype(np.longdouble))
    return f32(q.astype(np.longdouble) + rest.astype(np.longdouble) * recip.astype(np.longdouble))


def test_quotients_by_scales_are_rounded_quotients():
    """By every scale, by 6 and by gains of any kind, for numbers of any kind a row may hold: the
    division's result, bit by bit (so that halves between levels are met exactly)."""
    rng = np.random.default_rng(1)
    scales = [m / 8 * 2.0 ** -6 for m in range(1, 8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    gains = np.exp(rng.uniform(-20, 20, 300))
    edges = np.array([0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6])
    for y in np.concatenate([scales, [6.0], gains]).astype(np.float32):
        at = (edges * np.float64(y)).astype(np.float32)
        near = np.concatenate([at, np.nextafter(at, np.float32(0)), np.nextafter(at, np.float32(1e30))])
        x = np.concatenate([near, (rng.normal(size=2000) * y).astype(np.float32),
                            (rng.normal(size=500) * np.exp(rng.uniform(-30, 30, 500))).astype(np.float32)])
        yy = np.full_like(x, y)
        assert np.array_equal(quotient(x, yy), x / yy), y
