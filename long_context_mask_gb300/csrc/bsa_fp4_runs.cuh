// Work of the attention over a cache in 4 bits, for both of its kernels: row tiles, the cut of all
// work into equal runs, a run's row tiles one by one, and the join of rows that a cut splits.
//
// Rows are the new tokens of a sequence times the G query heads of a key/value head, token by token;
// a row tile is `wide` of them (with lists: of one token or of tpt whole ones), a key tile 128 positions.  All (key/value
// head, sequence, row tile, key tile) units are laid out in that order and cut into equal runs, one for
// each thread block; no host knowledge of the lengths is needed.  A row tile that a cut splits leaves
// its parts (O, maximum, sum, all fp32) in the workspace, and the join adds them in key order, so
// that a call's result does not depend on timing.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "bsa_fp4_ptx.cuh"
#include "bsa_internal.h"
#include "bsa_paged.cuh"
#include "bsa_rows.cuh"

namespace bsa {

constexpr float kFp4Ln2 = 0.6931471805599453f;
constexpr int kFp4PromptWide = 128;  // rows of a large row tile
// A row's maximum while it has seen no score above -infinity.  (Finite: -infinity less it is -infinity, a weight of 0, not
// NaN; any other score passes it by more than a maximum may be passed.)
constexpr float kFp4NoKey = -FLT_MAX;
// log2 of the weight that a score has when it becomes its row's maximum.  Weights are fp16 numbers, which lose bits below
// 2^-14 and end at 2^-25 and 2^16: a start at 2^6 leaves 31 bits below a row's largest weight, for rows whose first key
// takes nearly all of it, and 10 for scores to grow before the next maximum is taken.  (Prompt of 8192, scores of 1.2, 2.4, 3.7, 4.9
// nats about their mean: with 2^0 456, 457, 457, 468 us, 2^4 456, 456, 468, 536, 2^6 456, 458, 494, 620.  8192 even weights beside
// one 17 nats above them, whose value is 0: what they leave in O is off by 44 %, by 4.5 % at most, by 1.1 % at most.)
constexpr float kFp4Start = 6.0f;

struct Fp4Params {
    CUtensorMap map_k, map_ks, map_v, map_vs;  // codes and scales of short pages: a row a page and head
    PagedBatch b;
    const uint8_t *k, *k_scale, *v, *v_scale;
    const float *k_gain, *v_gain;
    const __nv_bfloat16* q;
    int64_t q_stride;
    int32_t H, H_kv, group;
    int32_t causal, window, sinks;
    int32_t least, most;  // sequences with so many rows are this kernel's
    float scale_log2;
    __nv_bfloat16* o;
    float* lse;
    // lists: of tile f = kvh * nt_cap + i, the i-th tpt tokens of the kernel's sequences; who: words words of token bits for each entry
    const int32_t *list, *list_cnt;
    const uint32_t* who;
    int32_t nt_cap, cap, words, tpt;
    // parts of split tiles
    float* part_o;    // [runs, 2, wide, D]
    float2* part_ml;  // [runs, 2, wide] maximum (log2) and sum
    int4* joins;      // [runs] parts (0: none), first packed row (token * group + head), rows, kvh
};

// Key tiles that the tokens at positions pos0 .. pos0 + ntok - 1 see some key
// of: the sink tiles 0 .. ns - 1 and lo .. lo + (n - ns) - 1.
__device__ __forceinline__ int32_t fp4_key_tiles(const Fp4Params& P, int32_t pos0, int32_t ntok, int32_t kl, int32_t& lo,
                                                 int32_t& ns) {
    const int32_t hi = P.causal ? min(kl, pos0 + ntok) : kl;  // keys 0 .. hi - 1
    lo = ns = 0;
    if (hi <= 0) return 0;
    const int32_t hi_t = (hi + 127) >> 7;
    if (P.window > 0) {
        lo = min(max(pos0 - P.window + 1, 0) >> 7, hi_t);
        ns = min((min(P.sinks, hi) + 127) >> 7, lo);
    }
    return hi_t - lo + ns;
}

// a / b; nearly every dividend fits 32 bits, whose division is much shorter.
__device__ __forceinline__ int64_t fp4_divide(int64_t a, int64_t b) {
    return (a >> 32) == 0 && (b >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// A thread block's run.
struct Fp4Run {
    int64_t share;          // units of a run; the first `extra` runs have one more
    int32_t extra, nt;      // row tiles of one key/value head
    __device__ __forceinline__ int64_t start(int32_t x) const { return share * x + min(x, extra); }
    // the run that holds unit u
    __device__ __forceinline__ int32_t of(int64_t u) const {
        const int64_t longer = (share + 1) * extra;  // units of the longer runs
        return (int32_t)(u < longer ? fp4_divide(u, share + 1) : extra + fp4_divide(u - longer, share));
    }
};
// Its first unit, and what all threads have to know of it (shared memory).
struct Fp4Start {
    int32_t kvh, s, t, i, x0;  // head, sequence, row tile of the sequence and of the head, unit within the row tile
    PagedSeq q;
    Fp4Run run;
    int32_t any;               // 0: this thread block has no run
    int64_t part[20];          // of the prefix sums
};

// Exclusive prefix sum over the first kScan threads of the block, which alone call it.
template <int kScan>
__device__ __forceinline__ int64_t fp4_prefix(int64_t x, int64_t* part, int64_t& total) {
    constexpr int warps = kScan / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t incl = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    auto meet = [] { asm volatile("bar.sync 1, %0;" ::"n"(kScan) : "memory"); };
    meet();  // an earlier call's readers are done with part
    if (lane == 31) part[warp] = incl;
    meet();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < warps; ++w) {
        const int64_t v = part[w];
        before += w < warp ? v : 0;
        all += v;
    }
    total = all;
    return before + incl - x;
}

// kCost: a row tile of n key tiles counts n + kCost in a run, the constant for its start and its end.
template <int kWide, int kCost, bool kLists>
struct Fp4Work {
    const Fp4Params& P;

    __device__ __forceinline__ int32_t per_token() const { return (P.group + kWide - 1) / kWide; }
    // with lists: tokens of a tile (of the narrow row tiles, one)
    __device__ __forceinline__ int32_t tpt() const { return kWide < kFp4PromptWide ? 1 : P.tpt; }
    __device__ __forceinline__ int32_t tiles(int32_t nq) const {
        const int32_t rows = nq * P.group;
        if (rows < P.least || rows > P.most) return 0;
        if constexpr (kLists) return (nq + tpt() - 1) / tpt() * per_token();
        return (rows + kWide - 1) / kWide;
    }
    // rows of row tile t: `n` from row0 on (token * group + head)
    __device__ __forceinline__ void rows(int32_t t, int32_t nq, int32_t& row0, int32_t& n) const {
        if constexpr (kLists) {
            const int32_t per = per_token(), x = t / per, h = (t - x * per) * kWide;
            row0 = x * tpt() * P.group + h;
            n = min(min(kWide, tpt() * P.group - h), nq * P.group - row0);
        } else {
            row0 = t * kWide;
            n = min(kWide, nq * P.group - row0);
        }
    }
    __device__ __forceinline__ int64_t list_of(int32_t kvh, int32_t i) const {  // (row tile i of the head)
        return (int64_t)kvh * P.nt_cap + i / per_token();
    }
    // key tiles of row tile i of the head, tile t of its sequence of nq new tokens and kl keys
    __device__ __forceinline__ int32_t keys(int32_t kvh, int32_t i, int32_t t, int32_t nq, int32_t kl, int32_t& lo,
                                            int32_t& ns) const {
        if constexpr (kLists) {
            lo = ns = 0;
            return P.list_cnt[list_of(kvh, i)];
        } else {
            int32_t row0, n;
            rows(t, nq, row0, n);
            const int32_t first = row0 / P.group, last = (row0 + n - 1) / P.group;
            return fp4_key_tiles(P, kl - nq + first, last - first + 1, kl, lo, ns);
        }
    }
    static __device__ __forceinline__ int32_t units(int32_t n) { return max(n, 1) + kCost; }
    // a cut x units into a row tile leaves so many of its key tiles on the left
    static __device__ __forceinline__ int32_t cut_at(int32_t x) { return max(x - kCost, 0); }

    // This thread block's run and its first unit, by the first kScan threads of the block (which alone
    // call it; the others would only wait for one another).  scratch: 3 seqs words of shared memory.  The
    // caller puts a __syncthreads() between this and what uses `start` or writes to scratch.
    template <int kScan>
    __device__ __forceinline__ void find(int32_t* scratch, Fp4Start& start) const {
        // of sequence s: the row tiles of the sequences before it, its new tokens and its length
        int32_t *cum = scratch, *seq_nq = cum + P.b.seqs, *seq_kl = seq_nq + P.b.seqs;
        int32_t nt;
        {
            const int32_t per = (P.b.seqs + kScan - 1) / kScan;
            const int32_t a = min((int32_t)threadIdx.x * per, P.b.seqs), e = min(a + per, P.b.seqs);
            int64_t mine = 0, all;
            for (int32_t s = a; s < e; ++s) {
                PagedSeq q;
                if (!paged_seq(P.b, s, q) && blockIdx.x == 0) raise_status(P.b.status, BSA_ERR_BOUNDS);
                seq_nq[s] = q.nq;
                seq_kl[s] = q.kl;
                mine += tiles(q.nq);
            }
            int64_t at = fp4_prefix<kScan>(mine, start.part, all);
            for (int32_t s = a; s < e; ++s) {
                cum[s] = (int32_t)min(at, (int64_t)INT32_MAX);
                at += tiles(seq_nq[s]);
            }
            // (beyond this: only with starts that decrease, reported above)
            const int64_t most = kLists ? (int64_t)P.nt_cap * per_token() : (int64_t)P.b.tokens * P.group / kWide + P.b.seqs;
            nt = (int32_t)min(all, most);
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kScan) : "memory");
        const int64_t rows = kLists ? (int64_t)nt * P.H_kv : nt;  // tiles whose counts differ
        const int64_t per_row = fp4_divide(rows + kScan - 1, kScan);
        const int64_t f0 = min((int64_t)threadIdx.x * per_row, rows), f1 = min(f0 + per_row, rows);
        // walks this thread's tiles: visit(kvh, i, s, t, units)
        auto walk = [&](auto&& visit) {
            if (f0 >= f1) return;
            int32_t kvh = kLists ? (int32_t)fp4_divide(f0, nt) : 0, i = (int32_t)(f0 - (int64_t)kvh * nt), s = 0;
            auto seek = [&]() {
                int32_t lo = 0, hi = P.b.seqs;  // the last s with cum[s] <= i
                while (hi - lo > 1) {
                    const int32_t mid = (lo + hi) >> 1;
                    if (cum[mid] <= i) lo = mid;
                    else hi = mid;
                }
                s = lo;
            };
            seek();
            for (int64_t f = f0; f < f1; ++f) {
                const int32_t t = i - cum[s];
                int32_t lo, ns;
                if (visit(kvh, i, s, t, units(keys(kvh, i, t, seq_nq[s], seq_kl[s], lo, ns)))) return;
                ++i;
                if (i == nt) {
                    i = 0;
                    ++kvh;
                    if (f + 1 < f1) seek();
                } else if (s + 1 < P.b.seqs && cum[s + 1] <= i) {
                    seek();
                }
            }
        };
        int64_t mine = 0, total;
        int4 only = make_int4(0, 0, 0, 0);  // (a thread with one tile need not walk again)
        walk([&](int32_t kvh, int32_t i, int32_t s, int32_t t, int32_t n) {
            mine += n;
            only = make_int4(kvh, s, t, i);
            return false;
        });
        const int64_t before = fp4_prefix<kScan>(mine, start.part, total);
        const int64_t all = kLists ? total : total * P.H_kv;
        const int32_t blocks = (int32_t)min((int64_t)gridDim.x, all);
        const bool any = (int32_t)blockIdx.x < blocks;
        if (threadIdx.x == 0) start.any = any;
        if (!any) return;
        Fp4Run run;
        run.share = fp4_divide(all, blocks);
        run.extra = (int32_t)(all - run.share * blocks);
        run.nt = nt;
        if (threadIdx.x == 0) start.run = run;
        const int64_t u0 = run.start(blockIdx.x), head = kLists ? 0 : fp4_divide(u0, total), x = kLists ? u0 : u0 - head * total;
        if (x >= before && x < before + mine) {
            auto begin = [&](int32_t kvh, int32_t s, int32_t t, int32_t i, int64_t at) {
                start.kvh = kLists ? kvh : (int32_t)head;
                start.s = s;
                start.t = t;
                start.i = i;
                start.x0 = (int32_t)(x - at);
                start.q.nq = seq_nq[s];
                start.q.kl = seq_kl[s];
                start.q.q0 = P.b.q_start[s];
            };
            if (f1 - f0 == 1) {
                begin(only.x, only.y, only.z, only.w, before);
            } else {
                int64_t at = before;
                walk([&](int32_t kvh, int32_t i, int32_t s, int32_t t, int32_t n) {
                    if (x < at + n) {
                        begin(kvh, s, t, i, at);
                        return true;
                    }
                    at += n;
                    return false;
                });
            }
        }
    }
};

// Codes (or scales) of pages, a lane each, to shared memory; every thread of the warp calls it.  Lane l has
// page l % N of its tile (cache row `row`, -1: none; `first`: of the tile's first page; live: the tile is there),
// dst its place, row_bytes a row's bytes.  Long pages come by a bulk copy each.  Short ones come four to a
// copy, a page behind the sequence's end as the tile's first: every copy keeps the issuing warp some 100
// cycles (64 tokens over caches up to 8192, 32 + 8 heads of 128, in pages of 16: 153 us with a copy a page, 110 so, and
// 101 in pages of 128).
constexpr int32_t kFp4LongPage = 64;
__device__ __forceinline__ void fp4_load_pages(const uint8_t* src, const CUtensorMap* map, int32_t page, int32_t row_bytes, bool live,
                                               int32_t row, int32_t first, uint32_t dst, uint32_t bar) {
    if (page >= kFp4LongPage) {
        if (row >= 0) bulk_load(dst, src + (int64_t)row * row_bytes, page * row_bytes, bar);
        return;
    }
    const int32_t y = (row >= 0 ? row : max(first, 0)) >> (__ffs(page) - 1);  // (a multiple of the page)
    const int32_t y1 = __shfl_down_sync(0xffffffffu, y, 1), y2 = __shfl_down_sync(0xffffffffu, y, 2), y3 = __shfl_down_sync(0xffffffffu, y, 3);
    if (live && (threadIdx.x & 3) == 0) tma_gather4(dst, map, 0, y, y1, y2, y3, bar);
}
// What a tile's first lane has to expect of that, pages_there of the tile's being there.
__device__ __forceinline__ uint32_t fp4_page_bytes(int32_t page, int32_t pages_there, int32_t row_bytes) {
    return (uint32_t)((page < kFp4LongPage ? 128 / page : pages_there) * page * row_bytes);
}

// A row tile's part in a run, as a kernel's loading warp tells the others.
struct Fp4Segment {
    int32_t n;              // key tiles (0: no key at all; -1: no more segments)
    int32_t kvh, q0;        // head; the sequence's first packed token
    int32_t row0, nrows;    // rows (token of the sequence * group + head)
    int32_t pos_of0, kl;    // position of the sequence's first new token, keys in the cache
    int32_t part;           // -1: the whole row tile is here; else its part slot: 2 block + 0 or 1
    int32_t seq, tile;      // the sequence; the row tile's number within the head
    int32_t j0, lo, ns;     // key tile j (j0 .. j0 + n - 1) is j < ns ? j : lo + j - ns (without lists)
};

// The run's row tiles one by one.
template <int kWide, int kCost, bool kLists>
struct Fp4Walk {
    Fp4Work<kWide, kCost, kLists> work;
    Fp4Run run;
    int64_t u, u_end;
    int32_t kvh, s, t, i, x0, w;
    PagedSeq q;
    bool last;  // the run ends within the row tile

    __device__ __forceinline__ Fp4Walk(const Fp4Params& P, const Fp4Start& a)
        : work{P}, run(a.run), u(a.run.start(blockIdx.x)), u_end(a.run.start(blockIdx.x + 1)), kvh(a.kvh), s(a.s), t(a.t), i(a.i), x0(a.x0),
          q(a.q) {}
    // the row tile at hand; false: no more in this run
    __device__ __forceinline__ bool open(Fp4Segment& sg) {
        if (u >= u_end) return false;
        const int32_t n = work.keys(kvh, i, t, q.nq, q.kl, sg.lo, sg.ns), n_eff = max(n, 1);
        const int64_t left = u_end - u;
        w = work.units(n);
        last = left < w - x0;
        sg.j0 = work.cut_at(x0);
        const int32_t j1 = min(last ? work.cut_at(x0 + (int32_t)left) : n_eff, n);
        if (last && j1 <= sg.j0) return false;  // (nothing of it: only where the run ends)
        sg.n = j1 - sg.j0;
        sg.kvh = kvh;
        sg.q0 = q.q0;
        sg.seq = s;
        sg.tile = i;
        work.rows(t, q.nq, sg.row0, sg.nrows);
        sg.pos_of0 = q.kl - q.nq;
        sg.kl = q.kl;
        sg.part = sg.j0 == 0 && !(last && j1 < n_eff) ? -1 : 2 * (int32_t)blockIdx.x + (sg.j0 == 0 ? 1 : 0);
        return true;
    }
    // (by one thread) a split row tile that begins here is noted for the join: its last part is in the run of its last unit
    __device__ __forceinline__ void note(const Fp4Segment& sg) const {
        if (last && sg.j0 == 0)
            work.P.joins[blockIdx.x] = make_int4(run.of(u + (w - x0) - 1) - (int32_t)blockIdx.x + 1,
                                                 q.q0 * work.P.group + sg.row0, sg.nrows, kvh);
    }
    __device__ __forceinline__ void advance() {
        const PagedBatch& b = work.P.b;
        u += w - x0;
        x0 = 0;
        if (u >= u_end) return;
        ++t;
        if (++i == run.nt) {  // the next head
            i = t = s = 0;
            ++kvh;
            paged_seq(b, 0, q);
        }
        while (t >= work.tiles(q.nq) && s + 1 < b.seqs) {
            t = 0;
            paged_seq(b, ++s, q);
        }
    }
};

// Joins the parts of split row tiles: O = sum_c 2^(m_c - M) O_c / l with M the largest m_c
// and l = sum_c 2^(m_c - M) l_c.  Thread block (c, y) takes kRows rows of the tile that begins in
// the attention's block c: its slot 1, then slot 0 of the blocks after it.  A row's kGroups groups of
// D / 4 lanes add parts g, g + kGroups, .., four loads under way at a time; the groups' sums are
// added in order.
constexpr int kFp4JoinThreads = 256;
template <int D, int kWide, int kRows>
__global__ void __launch_bounds__(kFp4JoinThreads) k_fp4_join(const __grid_constant__ Fp4Params P) {
    constexpr int kLanes = D / 4, kAll = kFp4JoinThreads / kLanes, kGroups = kAll / kRows;
    __shared__ float4 so[kAll][kLanes];
    __shared__ float2 ml[kAll];
    launch_dependents();
    wait_primary();
    const int c = threadIdx.x % kLanes, all = threadIdx.x / kLanes, group = all % kGroups;
    const int32_t row = blockIdx.y * kRows + all / kGroups, run = blockIdx.x;
    const int4 jn = P.joins[run];
    if (jn.x == 0 || (int32_t)(blockIdx.y * kRows) >= jn.z) return;
    auto part = [&](int32_t x) -> int64_t { return (((int64_t)run + x) * 2 + (x == 0 ? 1 : 0)) * kWide + row; };
    float M = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int32_t x0 = group; x0 < (row < jn.z ? jn.x : 0); x0 += 4 * kGroups) {
        float2 y[4];
        float4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int32_t x = x0 + u * kGroups;
            y[u] = x < jn.x ? P.part_ml[part(x)] : make_float2(-INFINITY, 0.0f);
            v[u] = x < jn.x ? *reinterpret_cast<const float4*>(P.part_o + part(x) * D + 4 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (y[u].y == 0.0f) continue;  // no visible key in this part
            const float M_new = fmaxf(M, y[u].x);
            const float keep = M == -INFINITY ? 1.0f : ex2(M - M_new), f = ex2(y[u].x - M_new);  // (l and o are 0 still)
            M = M_new;
            l = fmaf(f, y[u].y, l * keep);
            o[0] = fmaf(f, v[u].x, o[0] * keep);
            o[1] = fmaf(f, v[u].y, o[1] * keep);
            o[2] = fmaf(f, v[u].z, o[2] * keep);
            o[3] = fmaf(f, v[u].w, o[3] * keep);
        }
    }
    if constexpr (kGroups > 1) {
        so[all][c] = make_float4(o[0], o[1], o[2], o[3]);
        if (c == 0) ml[all] = make_float2(M, l);
        __syncthreads();
        if (group != 0) return;
        M = -INFINITY;
        l = o[0] = o[1] = o[2] = o[3] = 0.0f;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) M = fmaxf(M, ml[all + g].x);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const float2 y = ml[all + g];
            if (y.y == 0.0f) continue;
            const float f = ex2(y.x - M);
            const float4 v = so[all + g][c];
            l = fmaf(f, y.y, l);
            o[0] = fmaf(f, v.x, o[0]);
            o[1] = fmaf(f, v.y, o[1]);
            o[2] = fmaf(f, v.z, o[2]);
            o[3] = fmaf(f, v.w, o[3]);
        }
    }
    if (row >= jn.z) return;
    // (the gain after the quotient: the smallest gain over a long sum is no normal number)
    const float inv = l == 0.0f ? 0.0f : 1.0f / l, vg = P.v_gain != nullptr ? P.v_gain[jn.w] : 1.0f;
    const int32_t x = jn.y + row, tok = x / P.group;
    const int64_t at = (int64_t)tok * P.H + jn.w * P.group + (x - tok * P.group);
    *reinterpret_cast<uint2*>(P.o + at * D + 4 * c) =
        make_uint2(pack_bf16(o[0] * inv * vg, o[1] * inv * vg), pack_bf16(o[2] * inv * vg, o[3] * inv * vg));
    if (c == 0) P.lse[at] = l == 0.0f ? -INFINITY : (M + log2f(l)) * kFp4Ln2;
}

// bsa_fp4_prompt.cu: the sequences with P.least .. P.most rows, on the tensor core's large tiles.  first: the call's
// first kernel.
bsa_status launch_fp4_prompt(const Fp4Params& P, int32_t D, bool first, cudaStream_t stream);

}  // namespace bsa
