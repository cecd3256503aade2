"""Ragged batches over a paged cache and their 64-bit reference (test infrastructure).

Everything here follows the definitions in include/bsa.h, one sequence at a
time in fp64, and shares no code with the library."""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

BLOCK = 128


@dataclass
class Batch:
    """Sequences with `new` tokens each, `length` tokens in the cache with them."""
    new: list
    length: list
    H: int
    H_kv: int
    D: int
    page: int
    device: str
    table: torch.Tensor = None
    q_start: torch.Tensor = None
    kv_len: torch.Tensor = None
    k_cache: torch.Tensor = None
    v_cache: torch.Tensor = None
    n_pages: int = 0
    tokens: int = 0

    def arrays(self):
        return self.table, self.q_start, self.kv_len

    def pages_of(self, s):
        return self.table[s, :(self.length[s] + self.page - 1) // self.page].long()

    def keys(self, s, h, cache=None):
        """Rows 0 .. length - 1 of one sequence and key/value head, fp64."""
        c = self.k_cache if cache is None else cache
        return c[self.pages_of(s), h].reshape(-1, self.D)[:self.length[s]].double()


def make(new, length, H=4, H_kv=2, D=128, page=16, seed=0, device="cuda", spare=2, pad_tokens=0, first=0,
         max_pages=None, poison=True):
    """A batch with its pages in random order.  poison: every slot that holds no
    token of a sequence is NaN (the others N(0, 1)), and so is every table entry
    behind a sequence's last page out of range."""
    g = torch.Generator().manual_seed(seed)
    need = [(n + page - 1) // page for n in length]
    n_pages = sum(need) + spare
    order = torch.randperm(n_pages, generator=g)
    width = max(max(need), 1) if max_pages is None else max_pages
    table = torch.full((len(new), width), -7, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    starts = [first]
    for n in new:
        starts.append(starts[-1] + n)
    b = Batch(list(new), list(length), H, H_kv, D, page, device, n_pages=n_pages, tokens=starts[-1] + pad_tokens)
    b.table = table.to(device)
    b.q_start = torch.tensor(starts, dtype=torch.int32, device=device)
    b.kv_len = torch.tensor(length, dtype=torch.int32, device=device)
    fill = torch.full if poison else (lambda shape, _v, dtype: torch.zeros(shape, dtype=dtype))
    caches = []
    for _ in range(2):
        c = fill((n_pages, H_kv, page, D), float("nan"), dtype=torch.bfloat16)
        for s, n in enumerate(length):
            for p in range(need[s]):
                rows = min(page, n - p * page)
                c[table[s, p], :, :rows] = torch.randn((H_kv, rows, D), generator=g).to(torch.bfloat16)
        caches.append(c.to(device))
    b.k_cache, b.v_cache = caches
    return b


def rows(b, heads, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((b.tokens, heads, b.D), generator=g).to(torch.bfloat16).to(b.device)


def rope_table(n, rot, theta=10000.0, device="cuda"):
    a = torch.arange(n, dtype=torch.float64)[:, None] * theta ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    return torch.cat([a.cos(), a.sin()], 1).float().to(device).contiguous()


def turned(x, pos, rope, interleaved, w, eps):
    """(norm and rotation of x [n, heads, D] at positions pos in fp64, the
    magnitude that bounds its fp32 rounding errors)."""
    x = x.double()
    if w is not None:
        x = x / ((x * x).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    size = x.abs()
    if rope is None:
        return x, size
    rot = rope.shape[1]
    cs = rope[pos].double()[:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    a = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    c = a + 1 if interleaved else a + rot // 2
    y, big = x.clone(), size.clone()
    y[..., a] = x[..., a] * cos - x[..., c] * sin
    y[..., c] = x[..., c] * cos + x[..., a] * sin
    big[..., a] = big[..., c] = size[..., a] + size[..., c]
    return y, big


def attend(b, q, causal=True, window=0, sinks=0, sel=None, scale=None):
    """fp64 (O, LSE, A, R): A = sum_j p_j |v_j| and R = max_j |q| |k_j| scale bound
    the rounding errors.  sel: [tokens][kv head] lists of blocks."""
    scale = b.D ** -0.5 if scale is None else scale
    G = b.H // b.H_kv
    O = torch.zeros((b.tokens, b.H, b.D), dtype=torch.float64, device=b.device)
    A = torch.zeros_like(O)
    L = torch.full((b.tokens, b.H), -math.inf, dtype=torch.float64, device=b.device)
    R = torch.zeros_like(L)
    starts = b.q_start.tolist()
    for s, (n, length) in enumerate(zip(b.new, b.length)):
        if n == 0 or length == 0:
            continue
        t0 = starts[s]
        pos = torch.arange(length - n, length, device=b.device)
        j = torch.arange(length, device=b.device)
        for h in range(b.H_kv):
            k, v = b.keys(s, h), b.keys(s, h, b.v_cache)
            see = j[None] <= pos[:, None] if causal else torch.ones((n, length), dtype=torch.bool, device=b.device)
            if window > 0:
                see = see & ((j[None] > pos[:, None] - window) | (j[None] < sinks))
            if sel is not None:
                keep = torch.zeros((n, (length + BLOCK - 1) // BLOCK), dtype=torch.bool, device=b.device)
                for i in range(n):
                    keep[i, [x for x in sel[t0 + i][h] if 0 <= x < keep.shape[1]]] = True
                see = see & keep[:, j // BLOCK]
            for x in range(h * G, (h + 1) * G):
                qq = q[t0:t0 + n, x].double()
                z = (qq @ k.T * scale).masked_fill(~see, -math.inf)
                m = z.amax(1, keepdim=True)
                p = torch.where(see, (z - torch.where(m == -math.inf, torch.zeros_like(m), m)).exp(), torch.zeros_like(z))
                den = p.sum(1, keepdim=True)
                p = p / torch.where(den > 0, den, torch.ones_like(den))
                O[t0:t0 + n, x], A[t0:t0 + n, x] = p @ v, p @ v.abs()
                L[t0:t0 + n, x] = (m + den.log())[:, 0]
                R[t0:t0 + n, x] = qq.norm(dim=1) * k.norm(dim=1).max() * scale
    return O, L, A, R


def check_attention(b, q, o, lse, tokens=None, **kw):
    """o and lse against the reference, element by element.

    Errors: a score is a sum of D exact products in fp32, off by at most D 2^-24
    R, its scaled value and exponential by a few 2^-24 of |s| <= R and of itself:
    d = (D + 16) 2^-24 (R + 1) relative for each p_j, and twice that after the
    division by their sum.  Each p_j is rounded to bf16 (2^-8) before the
    product with v, O once more at the end."""
    O, L, A, R = attend(b, q, **kw)
    t = slice(b.q_start[0].item(), b.q_start[-1].item()) if tokens is None else tokens
    O, L, A, R = O[t], L[t], A[t], R[t]
    d = (b.D + 16) * 2.0 ** -24 * (R + 1)
    bound = 2.0 ** -8 * (A + O.abs()) * 1.01 + 2 * d[..., None] * A + 1e-30
    err = (o[t].double() - O).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"O: {int(bad.sum())} values off, worst {float((err / bound).nan_to_num(1e9).max()):.2f} of the bound, first at {bad.nonzero()[0].tolist()}"
    fin = torch.isfinite(L)
    assert torch.equal(torch.isneginf(lse[t]), torch.isneginf(L)), "LSE: -inf rows differ"
    le = (lse[t].double() - L).abs()[fin]
    lb = (d + 8 * 2.0 ** -24 * (1 + L.abs()))[fin]
    assert (le <= lb).all(), f"LSE off by {float(le.max())}"


def select(b, q, k_mean, topk, sinks, local):
    """fp64 [tokens][kv head] lists, ascending; and the counts."""
    per = BLOCK // b.page
    G = b.H // b.H_kv
    out = [[[] for _ in range(b.H_kv)] for _ in range(b.tokens)]
    starts = b.q_start.tolist()
    for s, (n, length) in enumerate(zip(b.new, b.length)):
        full = length // BLOCK
        last = b.table[s, [(j + 1) * per - 1 for j in range(full)]].long() if full else None
        for h in range(b.H_kv):
            for i in range(n):
                pos = length - n + i
                if pos < 0:
                    continue
                t, own = starts[s] + i, pos // BLOCK
                forced = [j for j in range(own + 1) if j < sinks or j > own - local]
                ranked = [j for j in range(own + 1) if j not in set(forced)]
                if len(ranked) > topk:
                    qs = q[t, h * G:(h + 1) * G].double().sum(0)
                    sc = (k_mean[last, h].double() @ qs).tolist()
                    ranked = sorted(ranked, key=lambda j: (-sc[j], j))[:topk]
                out[t][h] = sorted(forced + ranked)
    return out
