"""Cases, plain forms and exact values of the operators on a key/value cache held in 4 bits.

A row of the cache (one token and head, D values) is D / 2 bytes of codes and
D / 16 scales.  Value d stands for

    level(code_d) * scale_(d / 16) * gain

with the sixteen levels +-{0, 0.5, 1, 1.5, 2, 3, 4, 6} of a 4-bit float (sign,
two exponent bits, one of mantissa; value 2i in the low half of byte i), the
scale of its sixteen neighbours in 8 bits (e4m3) and one fp32 gain for each
key/value head (1 where there is none).

  append   rotate (and optionally normalise) the new queries and keys of a
           ragged batch, quantise keys and values and write them into the pages
           of the cache, with the mean key of each block that fills up; then
           read the new tokens back, as they are held now.
  read     the keys and values of many tokens out of the cache, as bf16.
  attend   attention of the new tokens (one for each sequence, a chunk, a whole
           prompt) over everything the cache holds for their sequence, through
           a sliding window with sinks, or over listed blocks alone.

`run` computes them in elementary torch operations in 32 bits where `own` is
false, and calls the library where it is true.
"""
import math
import random

import torch

own = False

BLOCK = 128
EPS = 1e-6
GROUP = 16
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# --------------------------------------------------------------------------- cases

def _case(name, op, **kw):
    c = dict(op=op, seqs=1, q=1, ragged=False, ctx=1024, heads=32, kv_heads=8, dim=128, page=128, gains=False)
    if op == "append":
        c.update(rot=128, interleaved=False, norms=False)
    elif op == "attend":
        c.update(window=0, sinks=0, topk=0)
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one decoding step of 32 conversations: latency
        _case("append_step_32", "append", seqs=32, ctx=2048, ragged=True, gains=True),
        # one whole prompt into an empty cache, with the per-head norms of newer models
        _case("append_prompt_8192", "append", q=8192, ctx=0, page=64, norms=True),
        # a serving step that mixes prompts' chunks: 14 heads of 64 over 2, partial rotation of
        # neighbouring pairs, small pages
        _case("append_mixed", "append", seqs=24, q=700, ragged=True, ctx=1500, heads=14, kv_heads=2, dim=64,
              page=16, rot=32, interleaved=True),
        # four long documents taken out of the cache, to be kept elsewhere
        _case("read_documents", "read", seqs=4, q=32768, ctx=0, page=64),
        # the last tokens of a few conversations, small heads and pages
        _case("read_tails", "read", seqs=6, q=150, ragged=True, ctx=900, heads=14, kv_heads=2, dim=64, page=16,
              gains=True),
        # the next token of one conversation: the smallest call
        _case("attend_one_1000", "attend", ctx=1000),
        # one decoding step of a full batch: bound by reading the cache
        _case("attend_step_64", "attend", seqs=64, ragged=True, ctx=8192),
        # the next token after a very long document: one row of work to split over the whole card
        _case("attend_one_131072", "attend", ctx=131071, page=64, gains=True),
        # chunks of many lengths over caches of many lengths, single tokens among them
        _case("attend_mixed", "attend", seqs=8, q=256, ragged=True, ctx=16384, heads=14, kv_heads=2, dim=64,
              page=16),
        # one whole prompt: bound by the matrix products
        _case("attend_prompt_8192", "attend", q=8192, ctx=0),
        # two chunks through a sliding window with sinks (575 + 64, the language-model layer of the benchmark)
        _case("attend_window", "attend", seqs=2, q=2048, ctx=6000, page=32, window=575, sinks=64),
        # one decoding step over long documents, 18 blocks of each
        _case("attend_listed_16", "attend", seqs=16, ragged=True, ctx=65536, topk=16, gains=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Batches, lengths, head layouts and page sizes over the whole range; a
    case that would cost more than the largest listed one is drawn again."""
    while True:
        op = rng.choice(["append", "append", "read", "attend", "attend", "attend"])
        heads, kv_heads = rng.choice([(32, 8), (32, 8), (8, 8), (14, 2), (16, 1), (24, 4), (12, 12), (40, 8)])
        dim = rng.choice([64, 128, 128])
        kind = rng.choice(["step", "step", "chunk", "mixed"])
        seqs = 1 if kind == "chunk" else _log(rng, 1, 96)
        q = 1 if kind == "step" else _log(rng, 2, 8192)
        ctx = _log(rng, 64, 131072) if kind != "mixed" else _log(rng, 64, 16384)
        if op == "append":
            ctx = min(ctx, 4096)
        elif op == "read":
            q, ctx = _log(rng, 1, 32768), _log(rng, 1, 8192)
        c = _case(None, op, seqs=seqs, q=q, ragged=kind != "chunk", ctx=ctx, heads=heads, kv_heads=kv_heads, dim=dim,
                  page=rng.choice([16, 32, 64, 128]), gains=rng.random() < 0.4)
        if op == "append":
            c.update(rot=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.3, norms=rng.random() < 0.5)
        elif op == "attend":
            how = rng.random()
            if how < 0.2:
                c.update(window=_log(rng, 64, 4096), sinks=rng.choice([0, 4, 64, 200]))
            elif how < 0.4:
                c.update(topk=_log(rng, 1, 48))
        pairs = seqs * heads * q * (ctx + q)          # what the plain form multiplies out
        cache = seqs * kv_heads * (ctx + q) * dim
        lists = seqs * q * kv_heads * (ctx + q) // BLOCK if op == "attend" and c["topk"] else 0
        if op == "read":
            if seqs * q <= 4 * 32768 and cache <= 8 * 8 * 32768 * 128:
                return c
        elif pairs <= 32 * 8192 * 8192 and cache <= 64 * 8 * 8192 * 128 and lists <= 1 << 25 and \
                (op != "append" or seqs * q <= 8192):
            return c


def _lens(case):
    """(new tokens, tokens in the cache after them) for each sequence, by the case alone."""
    r = random.Random("%(seqs)d %(q)d %(ctx)d" % case)
    ql, kl = [], []
    for s in range(case["seqs"]):
        n = case["q"] if not case["ragged"] or s == 0 else r.randint(1, case["q"])
        before = case["ctx"] if not case["ragged"] or s == 0 else r.randint(case["ctx"] // 2, case["ctx"])
        ql.append(n)
        kl.append(before + n)
    return ql, kl


# --------------------------------------------------------------------------- the 4-bit rows, plainly

def _levels(dev):
    up = torch.tensor(LEVELS, dtype=torch.float32, device=dev)
    return torch.cat([up, -up])


def _quantised(x):
    """Codes [..., D / 2] and scales [..., D / 16] (uint8, the e4m3 bytes) of x [..., D] fp32."""
    g = x.unflatten(-1, (-1, GROUP))
    scale = (g.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    y = torch.where(s > 0, g / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(g))
    # nearest level, halves to the even one (where that is the upper one, its edge belongs to it)
    edge = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    below = torch.nextafter(edge, torch.zeros_like(edge))
    edge = torch.where(torch.arange(7, device=x.device) % 2 == 1, below, edge)
    code = torch.bucketize(y.abs(), edge, out_int32=True).to(torch.uint8) + 8 * (y < 0).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], scale.view(torch.uint8)


def _values(codes, scales, gain=None):
    """What codes [..., D / 2] and scales [..., D / 16] (uint8) stand for, fp32; gain broadcasts against [...]."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    x = _levels(codes.device)[n] * scales.view(torch.float8_e4m3fn).float().repeat_interleave(GROUP, -1)
    return x if gain is None else x * gain[..., None]


# --------------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    ql, kl = _lens(case)
    S, T, H, K, D, P = case["seqs"], sum(ql), case["heads"], case["kv_heads"], case["dim"], case["page"]
    per_seq = (max(kl) + P - 1) // P
    need = [(n + P - 1) // P for n in kl]
    pages = sum(need) + 3
    # pages in a scattered order, as after many sequences have come and gone
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    at = torch.tensor([[sum(need[:s]) + p if p < need[s] else -1 for p in range(per_seq)] for s in range(S)], device=dev)
    table = torch.where(at >= 0, order[at.clamp(min=0)], torch.full_like(at, -1, dtype=torch.int32)).contiguous()
    starts = [0]
    for n in ql:
        starts.append(starts[-1] + n)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    st = dict(case=dict(case), table=table, q_start=torch.tensor(starts, dtype=torch.int32, device=dev),
              kv_len=torch.tensor(kl, dtype=torch.int32, device=dev), most=max(ql))
    # the host's plan of the ragged batch: each token's sequence and place, padded
    most = max(ql)
    st["seq"] = torch.repeat_interleave(torch.arange(S, device=dev), torch.tensor(ql, device=dev))
    st["place"] = torch.arange(T, device=dev) - st["q_start"].long()[st["seq"]]
    if case["op"] == "attend":
        st["pad"] = torch.tensor(starts[:-1], device=dev)[:, None] + \
            torch.minimum(torch.arange(most, device=dev), torch.tensor(ql, device=dev)[:, None] - 1)
    st["pos"] = st["kv_len"].long()[st["seq"]] - torch.tensor(ql, device=dev)[st["seq"]] + st["place"]
    if case["gains"]:
        # calibrated by head, so that the groups' scales lie in the middle of their type's range
        st["k_gain"] = 0.05 * (1 + torch.rand(K, generator=g, device=dev))
        st["v_gain"] = 0.02 * (1 + torch.rand(K, generator=g, device=dev))
    # keys have a few channels that are larger than the others
    wide = torch.ones(D, device=dev)
    wide[torch.randperm(D, generator=g, device=dev)[:D // 16]] = 3.0
    for name, shape in (("k", wide), ("v", torch.ones(D, device=dev))):
        codes = torch.empty((pages, K, P, D // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((pages, K, P, D // GROUP), dtype=torch.uint8, device=dev)
        step = max(1, (1 << 26) // (K * P * D))
        for a in range(0, pages, step):
            n = min(step, pages - a)
            x = normal(n, K, P, D) * shape
            if case["gains"]:
                x = x / st[name + "_gain"][:, None, None]
            codes[a:a + n], scales[a:a + n] = _quantised(x)
        st[name + "_cache"], st[name + "_scale"] = codes, scales.view(torch.float8_e4m3fn)
    if case["op"] != "attend":
        st["k_back"] = torch.empty((T, K, D), dtype=torch.bfloat16, device=dev)
        st["v_back"] = torch.empty((T, K, D), dtype=torch.bfloat16, device=dev)
    if case["op"] == "append":
        # one projection's output: queries, keys and values of a token side by side
        qkv = normal(T, H + 2 * K, D)
        qkv[:, H:H + K] *= wide
        qkv = qkv.to(torch.bfloat16)
        st.update(q=qkv[:, :H], k=qkv[:, H:H + K], v=qkv[:, H + K:])
        half = case["rot"] // 2
        angle = torch.arange(max(kl), device=dev, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)[None]
        st["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        if case["norms"]:
            st["q_norm"] = (1 + 0.1 * normal(D)).to(torch.bfloat16)
            st["k_norm"] = (1 + 0.1 * normal(D)).to(torch.bfloat16)
        st["k_mean"] = torch.zeros((pages, K, D), dtype=torch.bfloat16, device=dev)
        # tokens at the last place of a block
        st["last"] = torch.nonzero(st["pos"] % BLOCK == BLOCK - 1).flatten()
        st["q_out"] = torch.empty((T, H, D), dtype=torch.bfloat16, device=dev)
    elif case["op"] == "attend":
        st["q"] = normal(T, H, D).to(torch.bfloat16)
        st["o"] = torch.empty((T, H, D), dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.empty((T, H), device=dev)
        if case["topk"]:
            # what a selection gives: the first block, the token's own and the best of the others, ascending
            width = case["topk"] + 2
            blocks = (max(kl) + BLOCK - 1) // BLOCK
            block = torch.arange(blocks, device=dev)
            mine = (st["pos"] // BLOCK)[:, None, None]
            score = torch.rand((T, K, blocks), generator=g, device=dev)
            score = torch.where((block == 0) | (block == mine), torch.full_like(score, 2.0), score)
            score = torch.where(block > mine, torch.full_like(score, -1.0), score)
            top, sel = score.topk(min(width, blocks), -1)
            sel = torch.where(top >= 0, sel, torch.full_like(sel, 1 << 30)).sort(-1)[0]
            if blocks < width:
                sel = torch.cat([sel, sel.new_full((T, K, width - blocks), 1 << 30)], -1)
            st["sel_cnt"] = (sel < (1 << 30)).sum(-1).to(torch.int32)
            st["sel"] = torch.where(sel < (1 << 30), sel, torch.full_like(sel, -1)).to(torch.int32).contiguous()
    return st


# --------------------------------------------------------------------------- plain forms

def _rotated(x, w, st):
    """Norm and rotation of the heads of x [T, heads, D], in 32 bits (the norm's factor by way of 64)."""
    c = st["case"]
    x = x.float()
    if w is not None:
        x = x * (x.double().square().mean(-1, keepdim=True) + EPS).rsqrt().float() * w.float()
    rot = c["rot"]
    cs = st["rope"][st["pos"]][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([ya, yb], -1).flatten(-2) if c["interleaved"] else torch.cat([ya, yb], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _slots(st):
    """(page, row of the page) of each new token."""
    P = st["case"]["page"]
    return st["table"].long()[st["seq"], st["pos"] // P], st["pos"] % P


def _read_one(st, name, page, row):
    return st[name + "_back"].copy_(_values(st[name + "_cache"][page, :, row],
                                            st[name + "_scale"].view(torch.uint8)[page, :, row], st.get(name + "_gain")))


def _read(st):
    page, row = _slots(st)
    return dict(k=_read_one(st, "k", page, row), v=_read_one(st, "v", page, row))


def _write_one(st, name, x, page, row):
    if st["case"]["gains"]:
        x = x / st[name + "_gain"][:, None]
    codes, scales = _quantised(x)
    st[name + "_cache"][page, :, row] = codes
    st[name + "_scale"].view(torch.uint8)[page, :, row] = scales


def _append(st):
    P = st["case"]["page"]
    page, row = _slots(st)
    st["q_out"].copy_(_rotated(st["q"], st.get("q_norm"), st))
    _write_one(st, "k", _rotated(st["k"], st.get("k_norm"), st), page, row)
    _write_one(st, "v", st["v"].float(), page, row)
    last = st["last"]
    first = st["pos"][last] - (BLOCK - 1)
    pieces = torch.arange(BLOCK // P, device=last.device)
    grp = st["table"].long()[st["seq"][last][:, None], first[:, None] // P + pieces]
    gain = st["k_gain"][:, None] if st["case"]["gains"] else None
    held = _values(st["k_cache"][grp], st["k_scale"].view(torch.uint8)[grp], gain)
    st["k_mean"][page[last]] = (held.sum((1, 3)) / BLOCK).to(torch.bfloat16)
    return dict(q=st["q_out"], k_mean=st["k_mean"], **_read(st))


def _picked(st, blocks):
    """The lists as truth values [S, kv heads, tokens, blocks], of the padded batch."""
    sel = st["sel"].long()
    hit = torch.zeros((*sel.shape[:2], blocks + 1), dtype=torch.bool, device=sel.device)
    hit.scatter_(-1, torch.where(sel >= 0, sel, torch.full_like(sel, blocks)), True)
    return hit[st["pad"]][..., :blocks].permute(0, 2, 1, 3)


def _attention(st):
    """Softmax attention of the padded batch over the gathered pages, in 32 bits."""
    c = st["case"]
    S, K, D, P = c["seqs"], c["kv_heads"], c["dim"], c["page"]
    G = c["heads"] // K
    table = st["table"].long().clamp(min=0)
    L = table.shape[1] * P
    key = torch.arange(L, device=table.device)
    kl = st["kv_len"].long()

    def held(name):
        gain = st[name + "_gain"][:, None] if c["gains"] else None
        x = _values(st[name + "_cache"][table], st[name + "_scale"].view(torch.uint8)[table], gain)
        return x.permute(0, 2, 1, 3, 4).reshape(S, K, L, D)

    k = held("k")
    q = st["q"][st["pad"]].float().reshape(S, -1, K, G, D).permute(0, 2, 3, 1, 4)  # [S, K, G, tokens, D]
    pos = st["pos"][st["pad"]]                                                     # [S, tokens]
    see = key <= pos[..., None]
    if c["window"]:
        see = see & ((key > pos[..., None] - c["window"]) | (key < c["sinks"]))
    see = see[:, None]
    if c["topk"]:
        see = see & _picked(st, (L + BLOCK - 1) // BLOCK).repeat_interleave(BLOCK, -1)[..., :L]
    n = q.shape[3]
    s = (q.reshape(S, K, G * n, D) @ k.transpose(-1, -2)).reshape(S, K, G, n, L) * D ** -0.5
    del k
    s = torch.where(see[:, :, None], s, torch.full((), -math.inf, device=s.device))
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = (s - top).exp_()
    del s
    v = held("v")
    v = torch.where((key < kl[:, None])[:, None, :, None], v, torch.zeros((), device=v.device))
    den = p.sum(-1, keepdim=True)
    o = (p.reshape(S, K, G * n, L) @ v).reshape(S, K, G, n, D) / torch.where(den > 0, den, torch.ones_like(den))
    lse = (top + den.log())[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(S, n, K * G, D)[st["seq"], st["place"]]
    lse = lse.permute(0, 3, 1, 2).reshape(S, n, K * G)[st["seq"], st["place"]]
    return dict(o=o.to(torch.bfloat16), lse=lse)


# --------------------------------------------------------------------------- one pass

def _call(st):
    """The library's calls."""
    import long_context_mask_gb300 as bsa
    c = st["case"]
    cache = (st["k_cache"], st["k_scale"], st["v_cache"], st["v_scale"])
    batch = (st["table"], st["q_start"], st["kv_len"])
    gains = dict(k_gain=st.get("k_gain"), v_gain=st.get("v_gain"))
    if c["op"] == "attend":
        bsa.forward_paged_fp4(st["q"], *cache, *batch, st["o"], st["lse"], causal=True, window=c["window"],
                              sinks=c["sinks"], sel=st.get("sel"), sel_cnt=st.get("sel_cnt"), max_new=st["most"], **gains)
        return dict(o=st["o"], lse=st["lse"])
    if c["op"] == "append":
        bsa.paged_append_fp4(st["k"], st["v"], *cache, *batch, q=st["q"], q_out=st["q_out"], rope=st["rope"],
                             interleaved=c["interleaved"], q_norm=st.get("q_norm"), k_norm=st.get("k_norm"), eps=EPS,
                             k_mean=st["k_mean"], **gains)
    bsa.paged_read_fp4(*cache, *batch, st["k_back"], st["v_back"], **gains)
    back = dict(k=st["k_back"], v=st["v_back"])
    return back if c["op"] == "read" else dict(q=st["q_out"], k_mean=st["k_mean"], **back)


def run(st):
    if own:
        return _call(st)
    op = st["case"]["op"]
    return _append(st) if op == "append" else _read(st) if op == "read" else _attention(st)


# --------------------------------------------------------------------------- what a pass cannot do without

def _seen(c, pos):
    """Keys that a query at position pos attends to."""
    if not c["window"]:
        return pos + 1
    first = max(0, pos - c["window"] + 1)
    return pos + 1 - first + min(c["sinks"], first)


def work(case):
    ql, kl = _lens(case)
    T, H, K, D = sum(ql), case["heads"], case["kv_heads"], case["dim"]
    row = D // 2 + D // GROUP                                   # bytes of a key or a value
    tables = 8 * len(ql) + 4 * sum((n + case["page"] - 1) // case["page"] for n in kl) + 8 * K * bool(case["gains"])
    if case["op"] == "read":
        return dict(bytes=T * K * 2 * (row + 2 * D) + tables, flops=2 * T * K * D)
    if case["op"] == "append":
        done = sum(b // BLOCK - (b - a) // BLOCK for a, b in zip(ql, kl))
        old = sum((b - a) % BLOCK for a, b in zip(ql, kl) if b // BLOCK > (b - a) // BLOCK)  # keys of filled blocks
        moved = T * (H * 4 * D + K * 2 * (2 * D + row))         # in, and out to the cache
        back = T * K * 2 * (row + 2 * D)
        return dict(bytes=moved + back + 4 * case["rot"] * min(T, max(kl)) + tables + 2 * K * D * done + K * row * old,
                    flops=(3 * case["rot"] + 4 * D * bool(case["norms"])) * T * (H + K) + 6 * T * K * D + BLOCK * done * K * D)
    io = 4 * T * H * D + 4 * T * H + tables
    if not case["topk"]:
        pairs = sum(_seen(case, p) for a, b in zip(ql, kl) for p in range(b - a, b))
        keys = 0
        for a, b in zip(ql, kl):
            keys += b if not case["window"] else _seen(case, b - a) + a - 1
        return dict(bytes=io + 2 * K * row * min(keys, sum(kl)), flops=4 * D * H * pairs)
    pairs = picks = keys = 0
    for a, b in zip(ql, kl):
        here = 0
        for p in range(b - a, b):
            n = min(p // BLOCK + 1, case["topk"] + 2)
            here = (n - 1) * BLOCK + p % BLOCK + 1
            pairs += here
            picks += n
        keys += here  # one token's blocks at least; how many more is for the data to say
    return dict(bytes=io + 2 * K * row * keys + 4 * K * (picks + T), flops=4 * D * H * pairs)


# --------------------------------------------------------------------------- exact values

def _e4m3(byte):
    """An e4m3 byte's magnitude in 64 bits, by its bits."""
    b = byte.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    return torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m / 8 * 2.0 ** -6)


def _held(codes, scales):
    """What codes and scales stand for, in 64 bits and by their bits."""
    b = codes.to(torch.int64)
    n = torch.empty((*b.shape[:-1], 2 * b.shape[-1]), dtype=torch.int64, device=b.device)
    n[..., 0::2], n[..., 1::2] = b % 16, b // 16
    e, m = (n >> 1) & 3, (n & 1).double()
    mag = torch.where(e > 0, (1 + m / 2) * torch.exp2(e.double() - 1), m / 2)
    x = torch.where(n >= 8, -mag, mag)
    return (x.unflatten(-1, (-1, GROUP)) * _e4m3(scales)[..., None]).flatten(-2)


def _nearest(x):
    """Values of x [..., D] (64 bits) as the cache can hold them."""
    out = torch.empty_like(x)
    every = _e4m3(torch.arange(127, device=x.device))
    mid = (every[1:] + every[:-1]) / 2
    level = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    half = (level[1:] + level[:-1]) / 2

    def to_grid(a, grid, mids):
        i = torch.searchsorted(mids, a.contiguous())            # a tie goes to the lower one ...
        up = (i < mids.numel()) & (mids[i.clamp(max=mids.numel() - 1)] == a) & (i % 2 == 1)
        return grid[i + up]                                      # ... unless that is the odd one

    for d in range(0, x.shape[-1], GROUP):
        g = x[..., d:d + GROUP]
        s = to_grid(g.abs().amax(-1) / 6, every, mid)[..., None]
        y = g.abs() / torch.where(s > 0, s, torch.ones_like(s))
        out[..., d:d + GROUP] = torch.where(s > 0, to_grid(y, level, half) * s * g.sign(), torch.zeros_like(g))
    return out


def exact(case, seed):
    """The definition, sequence by sequence in 64 bits."""
    st = prepare(case, seed)
    ql, kl = _lens(case)
    H, K, D, P = case["heads"], case["kv_heads"], case["dim"], case["page"]
    G = H // K
    T = sum(ql)
    table = st["table"].tolist()
    one = torch.ones(K, dtype=torch.float64, device="cuda")
    gain = {n: st[n + "_gain"].double() if case["gains"] else one for n in ("k", "v")}

    def rows(name, s, lo, hi):
        """Rows lo .. hi - 1 of sequence s as the cache holds them [hi - lo, K, D]."""
        where = torch.arange(lo, hi, device="cuda")
        ids = torch.tensor(table[s], device="cuda")[where // P]
        x = _held(st[name + "_cache"][ids, :, where % P], st[name + "_scale"].view(torch.uint8)[ids, :, where % P])
        return x * gain[name][:, None]

    if case["op"] == "read":
        back = {n: torch.cat([rows(n, s, b - a, b) for s, (a, b) in enumerate(zip(ql, kl))]) for n in ("k", "v")}
        return dict(k=back["k"], v=back["v"])
    if case["op"] == "append":
        means = st["k_mean"].double()
        out = {n: torch.empty((T, x, D), dtype=torch.float64, device="cuda") for n, x in (("q", H), ("k", K), ("v", K))}
        rope, rot = st["rope"].double(), case["rot"]
        i0 = torch.arange(0, rot, 2, device="cuda") if case["interleaved"] else torch.arange(rot // 2, device="cuda")
        i1 = i0 + 1 if case["interleaved"] else i0 + rot // 2

        def turned(x, w, lo, hi):
            x = x.double()
            if w is not None:
                x = x / ((x * x).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
            y = x.clone()
            c, s = rope[lo:hi, None, :rot // 2], rope[lo:hi, None, rot // 2:]
            y[..., i0] = x[..., i0] * c - x[..., i1] * s
            y[..., i1] = x[..., i1] * c + x[..., i0] * s
            return y

        t = 0
        for s, (a, b) in enumerate(zip(ql, kl)):
            out["q"][t:t + a] = turned(st["q"][t:t + a], st.get("q_norm"), b - a, b)
            k = turned(st["k"][t:t + a], st.get("k_norm"), b - a, b)
            out["k"][t:t + a] = _nearest(k / gain["k"][:, None]) * gain["k"][:, None]
            out["v"][t:t + a] = _nearest(st["v"][t:t + a].double() / gain["v"][:, None]) * gain["v"][:, None]
            for blk in range((b - a) // BLOCK, b // BLOCK):
                lo, hi = blk * BLOCK, (blk + 1) * BLOCK
                keys = out["k"][t + max(lo, b - a) - (b - a):t + hi - (b - a)]
                if lo < b - a:
                    keys = torch.cat([rows("k", s, lo, b - a), keys])
                means[table[s][(hi - 1) // P]] = keys.sum(0) / BLOCK
            t += a
        return dict(q=out["q"], k_mean=means, k=out["k"], v=out["v"])
    if 4 * D * H * sum(a * b for a, b in zip(ql, kl)) > 1e13:
        return None
    o = torch.empty((T, H, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((T, H), dtype=torch.float64, device="cuda")
    t = 0
    for s, (a, b) in enumerate(zip(ql, kl)):
        pos = torch.arange(b - a, b, device="cuda")
        key = torch.arange(b, device="cuda")
        ks, vs = rows("k", s, 0, b), rows("v", s, 0, b)
        for h in range(K):
            see = key[None] <= pos[:, None]
            if case["window"]:
                see &= (key[None] > pos[:, None] - case["window"]) | (key[None] < case["sinks"])
            if case["topk"]:
                see &= (st["sel"][t:t + a, h, :, None] == (key // BLOCK)[None, None]).any(1) if a * b < 1 << 24 else \
                    torch.stack([(r[:, None] == (key // BLOCK)[None]).any(0) for r in st["sel"][t:t + a, h]])
            for x in range(h * G, (h + 1) * G):
                z = (st["q"][t:t + a, x].double() @ ks[:, h].T) / math.sqrt(D)
                z.masked_fill_(~see, -math.inf)
                lse[t:t + a, x] = torch.logsumexp(z, 1)
                o[t:t + a, x] = torch.softmax(z, 1) @ vs[:, h]
        t += a
    return dict(o=o, lse=lse)
