"""Cases, plain forms and exact values of the paged key/value cache operators.

Three operators, each reached through one public call (two for the third):

  append   rotate (and optionally normalise) the new queries and keys of a
           ragged batch and write keys and values into the pages of the cache;
           a 128-token block that fills up gets its mean key.
  attend   attention of the new tokens (one for each sequence, a chunk, a
           whole prompt) over everything the cache holds for their sequence.
  select   for each new token and key/value head, the best blocks by the score
           q . mean key, then attention over those blocks alone.

`run` computes them in elementary torch operations in 32 bits (scores that are
compared in 64) where `own` is false, and calls the library where it is true.
"""
import math
import random

import torch

own = False

BLOCK = 128
EPS = 1e-6


# --------------------------------------------------------------------------- cases

def _case(name, op, **kw):
    c = dict(op=op, seqs=1, q=1, ragged=False, ctx=1024, heads=32, kv_heads=8, dim=128, page=128)
    if op == "append":
        c.update(rot=128, interleaved=False, norms=False)
    elif op == "attend":
        c.update(window=0, sinks=0)
    else:
        c.update(topk=16, sink_blocks=1, local_blocks=1)
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one decoding step of 32 conversations: latency
        _case("append_step_32", "append", seqs=32, ctx=2048, ragged=True),
        # one whole prompt into an empty cache, with the per-head norms of newer models
        _case("append_prompt_8192", "append", q=8192, ctx=0, page=64, norms=True),
        # a serving step that mixes prompts' chunks: 14 heads of 64 over 2, partial rotation of
        # neighbouring pairs, small pages
        _case("append_mixed", "append", seqs=24, q=700, ragged=True, ctx=1500, heads=14, kv_heads=2, dim=64,
              page=16, rot=32, interleaved=True),
        # the next token of one conversation: the smallest call
        _case("attend_one_1000", "attend", ctx=1000),
        # one decoding step of a full batch: bound by reading the cache
        _case("attend_step_64", "attend", seqs=64, ragged=True, ctx=8192),
        # the next token after a very long document: one row of work to split over the whole card
        _case("attend_one_131072", "attend", ctx=131071, page=64),
        # chunks of many lengths over caches of many lengths, single tokens among them
        _case("attend_mixed", "attend", seqs=8, q=256, ragged=True, ctx=16384, heads=14, kv_heads=2, dim=64,
              page=16),
        # one whole prompt: bound by the matrix products
        _case("attend_prompt_8192", "attend", q=8192, ctx=0),
        # two chunks through a sliding window with sinks (575 + 64, the language-model layer of the benchmark)
        _case("attend_window", "attend", seqs=2, q=2048, ctx=6000, page=32, window=575, sinks=64),
        # one decoding step over long documents, 18 blocks of each
        _case("select_step_16", "select", seqs=16, ragged=True, ctx=65536),
        # a chunk of a very long document
        _case("select_chunk_1024", "select", q=1024, ctx=64512),
        # short chunks, odd sizes
        _case("select_mixed", "select", seqs=5, q=40, ragged=True, ctx=6000, heads=14, kv_heads=2, dim=64, page=32,
              topk=7, sink_blocks=2, local_blocks=3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Batches, lengths, head layouts and page sizes over the whole range; a
    case that would cost more than the largest listed one is drawn again."""
    while True:
        op = rng.choice(["append", "attend", "attend", "select"])
        heads, kv_heads = rng.choice([(32, 8), (32, 8), (8, 8), (14, 2), (16, 1), (24, 4), (12, 12), (40, 8)])
        dim = rng.choice([64, 128, 128])
        kind = rng.choice(["step", "step", "chunk", "mixed"])
        seqs = 1 if kind == "chunk" else _log(rng, 1, 96)
        q = 1 if kind == "step" else _log(rng, 2, 8192 if op != "select" else 1500)
        ctx = _log(rng, 64, 131072) if kind != "mixed" else _log(rng, 64, 16384)
        if op == "append":
            ctx = min(ctx, 4096)
        c = _case(None, op, seqs=seqs, q=q, ragged=kind != "chunk", ctx=ctx, heads=heads, kv_heads=kv_heads, dim=dim,
                  page=rng.choice([16, 32, 64, 128]))
        if op == "append":
            c.update(rot=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.3, norms=rng.random() < 0.5)
        elif op == "attend":
            if rng.random() < 0.25:
                c.update(window=_log(rng, 64, 4096), sinks=rng.choice([0, 4, 64, 200]))
        else:
            c.update(topk=_log(rng, 1, 48), sink_blocks=rng.choice([0, 1, 2]), local_blocks=rng.choice([1, 2, 4]))
        pairs = seqs * heads * q * (ctx + q)          # what the plain form multiplies out
        cache = seqs * kv_heads * (ctx + q) * dim
        if pairs <= 32 * 8192 * 8192 and cache <= 16 * 8 * 65536 * 128 and (op != "append" or seqs * q <= 8192):
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
              kv_len=torch.tensor(kl, dtype=torch.int32, device=dev))
    # the host's plan of the ragged batch: each token's sequence and place, padded
    most = max(ql)
    st["seq"] = torch.tensor([s for s in range(S) for _ in range(ql[s])], device=dev)
    st["place"] = torch.tensor([i for s in range(S) for i in range(ql[s])], device=dev)
    st["pad"] = torch.tensor([[starts[s] + min(i, ql[s] - 1) for i in range(most)] for s in range(S)], device=dev)
    st["pos"] = st["kv_len"].long()[st["seq"]] - torch.tensor(ql, device=dev)[st["seq"]] + st["place"]
    k_cache = torch.empty((pages, K, P, D), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    v_cache = torch.empty((pages, K, P, D), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    st.update(k_cache=k_cache, v_cache=v_cache)
    if case["op"] == "append":
        # one projection's output: queries, keys and values of a token side by side
        qkv = normal(T, H + 2 * K, D).to(torch.bfloat16)
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
        return st
    q = normal(T, H, D)
    if case["op"] == "select":
        # keys of a block share a direction and so do the queries of 64 neighbouring tokens: some
        # blocks matter more than others, and for neighbours they are much the same ones
        per = BLOCK // P
        blocks = (per_seq + per - 1) // per
        shift = normal(S, blocks, K, D) * 0.7
        owner = torch.zeros((pages, K, D), device=dev)
        page_of = table.long()
        shifts = shift.repeat_interleave(per, 1)[:, :per_seq]
        live = page_of >= 0
        owner[page_of[live]] = shifts[live]
        k_cache += owner[:, :, None].to(torch.bfloat16)
        turn = normal((T + 63) // 64 + 1, H, D)
        q = q + turn[torch.arange(T, device=dev) // 64]
        # mean key of every full block, kept at the page that holds the block's last token
        mean = torch.zeros((pages, K, D), dtype=torch.bfloat16, device=dev)
        full = per_seq // per
        if full:
            grp = page_of[:, :full * per].reshape(S, full, per)
            ok = grp[..., -1] >= 0
            last = grp[..., -1][ok]
            sums = torch.zeros((last.numel(), K, D), device=dev)
            for p in range(per):
                sums += k_cache[grp[..., p][ok]].float().sum(2)
            mean[last] = (sums / BLOCK).to(torch.bfloat16)
        st["k_mean"] = mean
        width = case["topk"] + case["sink_blocks"] + case["local_blocks"]
        st["sel"] = torch.empty((T, K, width), dtype=torch.int32, device=dev)
        st["sel_cnt"] = torch.empty((T, K), dtype=torch.int32, device=dev)
    st["q"] = q.to(torch.bfloat16)
    st["o"] = torch.empty((T, H, D), dtype=torch.bfloat16, device=dev)
    st["lse"] = torch.empty((T, H), device=dev)
    return st


# --------------------------------------------------------------------------- plain forms

def _rotated(x, w, st):
    """Norm and rotation of the heads of x [T, heads, D], in 32 bits."""
    c = st["case"]
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    rot = c["rot"]
    cs = st["rope"][st["pos"]][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([ya, yb], -1).flatten(-2) if c["interleaved"] else torch.cat([ya, yb], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _append(st):
    c = st["case"]
    P = c["page"]
    page = st["table"].long()[st["seq"], st["pos"] // P]
    st["q_out"].copy_(_rotated(st["q"], st.get("q_norm"), st))
    st["k_cache"][page, :, st["pos"] % P] = _rotated(st["k"], st.get("k_norm"), st).to(torch.bfloat16)
    st["v_cache"][page, :, st["pos"] % P] = st["v"]
    last = st["last"]
    first = st["pos"][last] - (BLOCK - 1)
    pieces = torch.arange(BLOCK // P, device=last.device)
    grp = st["table"].long()[st["seq"][last][:, None], first[:, None] // P + pieces]
    st["k_mean"][page[last]] = (st["k_cache"][grp].float().sum((1, 3)) / BLOCK).to(torch.bfloat16)
    return dict(q=st["q_out"], k_cache=st["k_cache"], v_cache=st["v_cache"], k_mean=st["k_mean"])


def _attention(st, picked=None):
    """Softmax attention of the padded batch over the gathered pages, in 32 bits.
    picked: truth values [S, kv heads, tokens, blocks], or None for all blocks."""
    c = st["case"]
    S, K, D, P = c["seqs"], c["kv_heads"], c["dim"], c["page"]
    G = c["heads"] // K
    table = st["table"].long().clamp(min=0)
    L = table.shape[1] * P
    key = torch.arange(L, device=table.device)
    kl = st["kv_len"].long()
    k = st["k_cache"][table].permute(0, 2, 1, 3, 4).reshape(S, K, L, D).float()
    v = st["v_cache"][table].permute(0, 2, 1, 3, 4).reshape(S, K, L, D).float()
    v = torch.where((key < kl[:, None])[:, None, :, None], v, torch.zeros((), device=v.device))
    q = st["q"][st["pad"]].float().reshape(S, -1, K, G, D).permute(0, 2, 3, 1, 4)  # [S, K, G, tokens, D]
    pos = st["pos"][st["pad"]]                                                     # [S, tokens]
    see = key <= pos[..., None]
    if c.get("window"):
        see = see & ((key > pos[..., None] - c["window"]) | (key < c["sinks"]))
    see = see[:, None]
    if picked is not None:
        see = see & picked.repeat_interleave(BLOCK, -1)[..., :L]
    n = q.shape[3]
    s = (q.reshape(S, K, G * n, D) @ k.transpose(-1, -2)).reshape(S, K, G, n, L) * D ** -0.5
    s = torch.where(see[:, :, None], s, torch.full((), -math.inf, device=s.device))
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = (s - top).exp_()
    del s
    den = p.sum(-1, keepdim=True)
    o = (p.reshape(S, K, G * n, L) @ v).reshape(S, K, G, n, D) / torch.where(den > 0, den, torch.ones_like(den))
    lse = (top + den.log())[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(S, n, K * G, D)[st["seq"], st["place"]]
    lse = lse.permute(0, 3, 1, 2).reshape(S, n, K * G)[st["seq"], st["place"]]
    return o.to(torch.bfloat16), lse


def _selection(st):
    """Blocks of each token and key/value head: (truth values [S, kv heads, tokens, blocks], list, counts).
    Scores in 64 bits: they are compared with one another."""
    c = st["case"]
    S, K, D, P = c["seqs"], c["kv_heads"], c["dim"], c["page"]
    G = c["heads"] // K
    per = BLOCK // P
    table = st["table"].long()
    blocks = (table.shape[1] + per - 1) // per
    block = torch.arange(blocks, device=table.device)
    last = table[:, (block * per + per - 1).clamp(max=table.shape[1] - 1)].clamp(min=0)
    mean = st["k_mean"][last].double()                                             # [S, blocks, K, D]
    q = st["q"][st["pad"]].double().reshape(S, -1, K, G, D).sum(3)                 # [S, tokens, K, D]
    score = q.transpose(1, 2) @ mean.permute(0, 2, 3, 1)                           # [S, K, tokens, blocks]
    mine = (st["pos"][st["pad"]] // BLOCK)[:, None, :, None]
    forced = (block <= mine) & ((block < c["sink_blocks"]) | (block > mine - c["local_blocks"]))
    open_ = (block < mine) & ~forced
    score = torch.where(open_, score, torch.full((), -math.inf, device=score.device, dtype=score.dtype))
    by = torch.sort(score, dim=-1, descending=True, stable=True)[1]
    rank = torch.empty_like(by).scatter_(-1, by, block.expand_as(by).contiguous())
    picked = forced | (open_ & (rank < c["topk"]))
    width = c["topk"] + c["sink_blocks"] + c["local_blocks"]
    lists = torch.where(picked, block, torch.full_like(block, 1 << 30)).sort(-1)[0][..., :width]
    if lists.shape[-1] < width:
        lists = torch.cat([lists, lists.new_full((*lists.shape[:-1], width - lists.shape[-1]), 1 << 30)], -1)
    lists = torch.where(lists < (1 << 30), lists, torch.full_like(lists, -1)).to(torch.int32)
    own_tokens = lambda x: x.transpose(1, 2)[st["seq"], st["place"]]  # noqa: E731
    return picked, own_tokens(lists), own_tokens(picked.sum(-1).to(torch.int32))


# --------------------------------------------------------------------------- one pass

def _call(st):
    """The library's calls."""
    import long_context_mask_gb300 as bsa
    c = st["case"]
    batch = (st["table"], st["q_start"], st["kv_len"])
    if c["op"] == "append":
        bsa.paged_append(st["k"], st["v"], st["k_cache"], st["v_cache"], *batch, q=st["q"], q_out=st["q_out"],
                         rope=st["rope"], interleaved=c["interleaved"], q_norm=st.get("q_norm"),
                         k_norm=st.get("k_norm"), eps=EPS, k_mean=st["k_mean"])
        return dict(q=st["q_out"], k_cache=st["k_cache"], v_cache=st["v_cache"], k_mean=st["k_mean"])
    if c["op"] == "attend":
        bsa.forward_paged(st["q"], st["k_cache"], st["v_cache"], *batch, st["o"], st["lse"], causal=True,
                          window=c["window"], sinks=c["sinks"])
        return dict(o=st["o"], lse=st["lse"])
    bsa.select_paged(st["q"], st["k_mean"], *batch, st["sel"], st["sel_cnt"], page_size=c["page"], topk=c["topk"],
                     sink_blocks=c["sink_blocks"], local_blocks=c["local_blocks"])
    bsa.forward_paged(st["q"], st["k_cache"], st["v_cache"], *batch, st["o"], st["lse"], causal=True, sel=st["sel"],
                      sel_cnt=st["sel_cnt"])
    return dict(o=st["o"], lse=st["lse"], sel=st["sel"], sel_cnt=st["sel_cnt"])


def run(st):
    if own:
        return _call(st)
    op = st["case"]["op"]
    if op == "append":
        return _append(st)
    if op == "attend":
        o, lse = _attention(st)
        return dict(o=o, lse=lse)
    picked, lists, counts = _selection(st)
    o, lse = _attention(st, picked)
    return dict(o=o, lse=lse, sel=lists, sel_cnt=counts)


# --------------------------------------------------------------------------- what a pass cannot do without

def _seen(c, pos, kv_len):
    """Keys that a query at position pos attends to."""
    if not c.get("window"):
        return pos + 1
    first = max(0, pos - c["window"] + 1)
    return pos + 1 - first + min(c["sinks"], first)


def work(case):
    ql, kl = _lens(case)
    T, H, K, D = sum(ql), case["heads"], case["kv_heads"], case["dim"]
    tables = 8 * len(ql) + 4 * sum((n + case["page"] - 1) // case["page"] for n in kl)
    if case["op"] == "append":
        done = sum(b // BLOCK - (b - a) // BLOCK for a, b in zip(ql, kl))
        old = sum((b - a) % BLOCK for a, b in zip(ql, kl) if b // BLOCK > (b - a) // BLOCK)  # keys of filled blocks
        rows = T * (H + 2 * K) * D
        return dict(bytes=4 * rows + 4 * case["rot"] * min(T, max(kl)) + tables + 2 * K * D * (done + old),
                    flops=(3 * case["rot"] + 4 * D * bool(case["norms"])) * T * (H + K) + BLOCK * done * K * D)
    io = 4 * T * H * D + 4 * T * H + tables
    if case["op"] == "attend":
        pairs = sum(_seen(case, p, b) for a, b in zip(ql, kl) for p in range(b - a, b))
        keys = 0
        for a, b in zip(ql, kl):
            keys += b if not case["window"] else _seen(case, b - a, b) + a - 1
        return dict(bytes=io + 4 * K * D * min(keys, sum(kl)), flops=4 * D * H * pairs)
    pairs = picks = keys = means = 0
    for a, b in zip(ql, kl):
        here = 0
        for p in range(b - a, b):
            mine = p // BLOCK
            forced = min(mine + 1, case["sink_blocks"] + case["local_blocks"])
            n = forced + min(case["topk"], mine + 1 - forced)
            here = (n - 1) * BLOCK + p % BLOCK + 1
            pairs += here
            picks += n
            means += mine
        keys += here  # one token's blocks at least; how many more is for the data to say
    return dict(bytes=io + 4 * K * D * keys + 2 * K * D * sum(b // BLOCK for b in kl) + 4 * K * (picks + T),
                flops=4 * D * H * pairs + 2 * D * K * means)


# --------------------------------------------------------------------------- exact values

def exact(case, seed):
    """The definition, sequence by sequence in 64 bits."""
    st = prepare(case, seed)
    ql, kl = _lens(case)
    H, K, D, P = case["heads"], case["kv_heads"], case["dim"], case["page"]
    G = H // K
    table = st["table"].tolist()
    if case["op"] == "append":
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        rounded = st["k_cache"].double()
        means = st["k_mean"].double()
        q_out = torch.empty(st["q"].shape, dtype=torch.float64, device=kc.device)
        rope, rot = st["rope"].double(), case["rot"]
        one = torch.arange(0, rot, 2, device=kc.device) if case["interleaved"] else torch.arange(rot // 2, device=kc.device)
        two = one + 1 if case["interleaved"] else one + rot // 2

        def turned(x, w, lo, hi):
            x = x.double()
            if w is not None:
                x = x / ((x * x).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
            y = x.clone()
            c, s = rope[lo:hi, None, :rot // 2], rope[lo:hi, None, rot // 2:]
            y[..., one] = x[..., one] * c - x[..., two] * s
            y[..., two] = x[..., two] * c + x[..., one] * s
            return y

        t = 0
        for s, (a, b) in enumerate(zip(ql, kl)):
            q_out[t:t + a] = turned(st["q"][t:t + a], st.get("q_norm"), b - a, b)
            k = turned(st["k"][t:t + a], st.get("k_norm"), b - a, b)
            at = b - a
            while at < b:
                stop = min(b, (at // P + 1) * P)
                page, i = table[s][at // P], at - (b - a)
                kc[page, :, at % P:at % P + stop - at] = k[i:i + stop - at].transpose(0, 1)
                rounded[page, :, at % P:at % P + stop - at] = k[i:i + stop - at].transpose(0, 1).float().bfloat16().double()
                vc[page, :, at % P:at % P + stop - at] = st["v"][t + i:t + i + stop - at].transpose(0, 1).double()
                at = stop
            for blk in range((b - a) // BLOCK, b // BLOCK):
                which = [table[s][(blk * BLOCK + p) // P] for p in range(0, BLOCK, P)]
                means[which[-1]] = rounded[which].sum((0, 2)) / BLOCK
            t += a
        return dict(q=q_out, k_cache=kc, v_cache=vc, k_mean=means)
    T = sum(ql)
    o = torch.empty((T, H, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((T, H), dtype=torch.float64, device="cuda")
    t = 0
    for s, (a, b) in enumerate(zip(ql, kl)):
        which = torch.tensor(table[s][:(b + P - 1) // P], device="cuda")
        pos = torch.arange(b - a, b, device="cuda")
        key = torch.arange(b, device="cuda")
        for h in range(K):
            k = st["k_cache"][which, h].reshape(-1, D)[:b].double()
            v = st["v_cache"][which, h].reshape(-1, D)[:b].double()
            see = key[None] <= pos[:, None]
            if case.get("window"):
                see &= (key[None] > pos[:, None] - case["window"]) | (key[None] < case["sinks"])
            if case["op"] == "select":
                n_blocks = (b + BLOCK - 1) // BLOCK
                ends = torch.tensor([table[s][((j + 1) * BLOCK - 1) // P] if (j + 1) * BLOCK <= b else 0
                                     for j in range(n_blocks)], device="cuda")
                qs = st["q"][t:t + a, h * G:(h + 1) * G].double().sum(1)
                score = qs @ st["k_mean"][ends, h].double().T
                j = torch.arange(n_blocks, device="cuda")[None]
                mine = pos[:, None] // BLOCK
                keep = (j <= mine) & ((j < case["sink_blocks"]) | (j > mine - case["local_blocks"]))
                may = (j < mine) & ~keep
                score = score.masked_fill(~may, -math.inf)
                n = min(case["topk"], n_blocks)
                order = torch.argsort(score, dim=1, descending=True, stable=True)[:, :n]
                best = torch.zeros_like(may).scatter_(1, order, True)
                see &= (keep | (best & may))[:, key // BLOCK]
            for x in range(h * G, (h + 1) * G):
                z = (st["q"][t:t + a, x].double() @ k.T) / math.sqrt(D)
                z.masked_fill_(~see, -math.inf)
                lse[t:t + a, x] = torch.logsumexp(z, 1)
                o[t:t + a, x] = torch.softmax(z, 1) @ v
        t += a
    return dict(o=o, lse=lse) if case["op"] == "attend" else dict(o=o, lse=lse, sel=None, sel_cnt=None)
