"""A paged cache in 4 bits and its 64-bit reference (test infrastructure).

Follows the definitions in include/bsa.h, in fp64, and shares no code with the
library; batches and attention are paged_ref's."""
from __future__ import annotations

import torch

import paged_ref as ref

LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def e4m3(byte):
    """Values of e4m3 bytes, as a scale counts them: NaN and negative ones are 0."""
    b = byte.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    x = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m / 8 * 2.0 ** -6)
    return torch.where((b >= 127), torch.zeros_like(x), x)


def nibbles(codes):
    c = codes.to(torch.int64)
    return torch.stack([c & 15, c >> 4], -1).flatten(-2)


def levels(n):
    t = torch.tensor(LEVELS + [-x for x in LEVELS], dtype=torch.float64, device=n.device)
    return t[n]


def held(codes, scale, gain=None):
    """What codes [..., D / 2] and scales [..., D / 16] stand for, fp64; gain broadcasts against [...]."""
    s = scale.view(torch.uint8) if scale.dtype != torch.uint8 else scale
    x = (levels(nibbles(codes)).unflatten(-1, (-1, 16)) * e4m3(s)[..., None]).flatten(-2)
    return x if gain is None else x * gain.double()[..., None]


class Cache:
    """Codes, scales and gains beside a paged_ref batch b; b.k_cache and b.v_cache become what they stand for."""

    def __init__(self, b, seed=0, gains=False, dirty=True):
        """Random codes under scales around 1/6 (values of some 0 .. 1.5); dirty: every slot
        that holds no token has random bytes, scales that are NaN, negative and huge among them."""
        g = torch.Generator().manual_seed(1000 + seed)
        shape = (b.n_pages, b.H_kv, b.page)
        self.b, self.dev = b, b.device
        self.k_gain = (0.5 + torch.rand(b.H_kv, generator=g)).to(b.device) if gains else None
        self.v_gain = (0.5 + torch.rand(b.H_kv, generator=g)).to(b.device) if gains else None
        live = torch.zeros(shape[0], shape[2], dtype=torch.bool)
        for s, n in enumerate(b.length):
            for p in range((n + b.page - 1) // b.page):
                live[b.table[s, p].cpu().long(), :min(b.page, n - p * b.page)] = True
        for name in ("k", "v"):
            codes = torch.randint(0, 256, (*shape, b.D // 2), generator=g, dtype=torch.uint8)
            good = (0.25 * torch.rand((*shape, b.D // 16), generator=g)).to(torch.float8_e4m3fn).view(torch.uint8)
            if dirty:
                junk = torch.randint(0, 256, good.shape, generator=g, dtype=torch.uint8)
                junk = torch.where(torch.rand(good.shape, generator=g) < 0.3, torch.full_like(junk, 0x7f), junk)
                good = torch.where(live[:, None, :, None], good, junk)
            setattr(self, name, codes.to(b.device))
            setattr(self, name + "_scale", good.to(b.device).view(torch.float8_e4m3fn))
        self.refresh()

    def arrays(self):
        return self.k, self.k_scale, self.v, self.v_scale

    def gains(self):
        return dict(k_gain=self.k_gain, v_gain=self.v_gain)

    def clone(self):
        return [x.clone() for x in self.arrays()]

    def refresh(self):
        b = self.b
        for name in ("k", "v"):
            gain = getattr(self, name + "_gain")
            setattr(b, name + "_cache", held(getattr(self, name), getattr(self, name + "_scale"),
                                             None if gain is None else gain[:, None]))
        return self


def check_attention(b, q, o, lse, tokens=None, **kw):
    """o and lse against the reference, element by element.

    Errors: a score is a sum of D exact products in fp32, off by at most D 2^-24 R, its
    scaled value and exponential by a few 2^-24 of |s| <= R and of itself: d = (D + 16) 2^-24
    (R + 1) relative for each p_j, and twice that after the division by their sum.  (What a query
    loses in fp16 lies 2^39 below its row's largest value.)  Each p_j is rounded to fp16
    against an earlier maximum of its row: 2^-11 of itself and, below fp16's normal
    numbers, 2^-25 where the sum is at least 1.  O is rounded to bf16 (2^-8)."""
    O, L, A, R = ref.attend(b, q, **kw)
    W = visible(b, **kw)
    t = slice(b.q_start[0].item(), b.q_start[-1].item()) if tokens is None else tokens
    O, L, A, R, W = O[t], L[t], A[t], R[t], W[t]
    d = (b.D + 16) * 2.0 ** -24 * (R + 1)
    bound = 2.0 ** -8 * O.abs() * 1.01 + (2.0 ** -11 * 1.01 + 2 * d[..., None]) * A + 2.0 ** -25 * W + 1e-30
    err = (o[t].double() - O).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"O: {int(bad.sum())} values off, worst {float((err / bound).nan_to_num(1e9).max()):.2f} of the bound, first at {bad.nonzero()[0].tolist()}"
    fin = torch.isfinite(L)
    assert torch.equal(torch.isneginf(lse[t]), torch.isneginf(L)), "LSE: -inf rows differ"
    le = (lse[t].double() - L).abs()[fin]
    lb = (d + 8 * 2.0 ** -24 * (1 + L.abs()))[fin]
    assert (le <= lb).all(), f"LSE off by {float(le.max())}"


def visible(b, causal=True, window=0, sinks=0, sel=None, scale=None):
    """Sum of |v| over a sequence's keys, [tokens, H, D]: at least what any row sees."""
    W = torch.zeros((b.tokens, b.H, b.D), dtype=torch.float64, device=b.device)
    starts = b.q_start.tolist()
    for s, (n, length) in enumerate(zip(b.new, b.length)):
        for h in range(b.H_kv if n and length else 0):
            G = b.H // b.H_kv
            W[starts[s]:starts[s] + n, h * G:(h + 1) * G] = b.keys(s, h, b.v_cache).abs().sum(0)
    return W


def check_quantised(x, err, codes, scale, gain=None):
    """codes [..., D / 2] and scales [..., D / 16] as bytes of rows x [..., D] (fp64) that the
    library knows to within err: each scale is one of the nearest to max |x / gain| / 6
    and each code one of the nearest levels to x / gain / scale, nearest as far as err, and
    the quotients' fp32 roundings, tell."""
    g = torch.ones((), dtype=torch.float64, device=x.device) if gain is None else gain.double()[..., None]
    t, e = (x / g).unflatten(-1, (-1, 16)), (err / g + 2.0 ** -24 * (x / g).abs()).unflatten(-1, (-1, 16))
    s = e4m3(scale)
    assert (scale < 127).all()
    want, off = t.abs().amax(-1) / 6, e.amax(-1) / 6
    off = off + 2.0 ** -24 * want
    grid = e4m3(torch.arange(127, device=x.device))
    near = (grid - want.clamp(max=448.0)[..., None]).abs().amin(-1)
    assert ((s - want.clamp(max=448.0)).abs() <= near + 2 * off).all(), "scales"
    one = torch.where(s > 0, s, torch.ones_like(s))[..., None]
    y, ey = t / one, e / one + 2.0 ** -24 * (t / one).abs()
    n = nibbles(codes).unflatten(-1, (-1, 16))
    got = levels(n)
    y = y.clamp(-6, 6)
    grid = levels(torch.arange(16, device=x.device))
    near = (grid - y[..., None]).abs().amin(-1)
    ok = (got - y).abs() <= near + 2 * ey
    assert torch.where(s[..., None] > 0, ok, n & 7 == 0).all(), "codes"


def random_rows(b, heads, seed, spread=True):
    """bf16 rows whose groups have sizes of many magnitudes."""
    x = ref.rows(b, heads, seed).float()
    if spread:
        g = torch.Generator().manual_seed(seed + 77)
        e = torch.randint(-8, 6, (*x.shape[:2], b.D // 16, 1), generator=g).float().exp2().to(x.device)
        x = (x.unflatten(-1, (-1, 16)) * e).flatten(-2)
    return x.to(torch.bfloat16)

