// Attention of new tokens over a paged key/value cache held in 4 bits.
//
// What it computes is what bsa_paged_attn.cu computes (token i of a sequence at position
// p, query head h, the keys j that causality, a window with sinks or a list of blocks leave):
//     s_j = scale q . k_j,   LSE = ln sum_j exp(s_j),   O = sum_j exp(s_j - LSE) v_j
// with k_j and v_j as bsa_fp4.cuh reads them.
//
// Rows.  The new tokens of a sequence and the G query heads of a key/value head are rows,
// token by token; a row tile is 8 NT of them (with lists: of one token).  A key tile is 128
// positions, 16 for each of the thread block's eight warps.  Few rows want the keys as the
// long side of the products: with mma m16n8k16, S^T = K Q^T has 16 keys by 8 rows,
// O^T = V^T P^T has 16 values of D by 8 rows.  Codes go from memory to registers and become
// fp16 operands there, with no shared memory between:
//   K    lane (r, c) = (lane / 4, lane % 4) loads D / 4 values of keys r and r + 8.  The order
//        of the D values in the sum is free, so a byte's two values are one operand register.
//   V^T  lane (r, c) loads D / 8 values of keys 2c, 2c + 1, 2c + 8, 2c + 9.  An operand register
//        holds two keys' values at one place: their nibbles are brought together in a byte
//        before it is converted.
//   P^T  comes out of S^T's accumulators by two 8 x 8 transposes (movmatrix).
// Levels times scales are exact in fp16.  Queries are multiplied by the power of two that
// brings their row's largest value to 2^14, and rounded to fp16 (what a bf16 value loses
// lies 2^39 below the row's largest).  Weights are rounded to fp16: they are kept below
// 2^11 by raising the row's maximum when a score passes it by 2^10.
//
// Split.  All (key/value head, sequence, row tile, key tile) units are laid out in that order
// and cut into equal runs, one for each thread block.  A row tile's part in a run is joined
// over the eight warps in shared memory; a tile that a cut splits leaves its parts in the workspace
// for k_fp4_join, which adds them in key order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "bsa_device_setup.h"
#include "bsa_fp4.cuh"
#include "bsa_internal.h"
#include "bsa_paged.cuh"
#include "bsa_rows.cuh"

namespace bsa {
namespace {

constexpr int32_t kMaxWindow = 1 << 26;  // (positions lie within 2^24 of zero)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kRuns = 2 * kPagedBlocks;
constexpr int kMaxNT = 2;
constexpr float kRaise = 10.0f;  // log2 of how far a weight may pass its row's maximum

enum { kPlain = 0, kWindow = 1, kListed = 2 };

struct Fp4Params {
    PagedBatch b;
    const uint8_t *k, *k_scale, *v, *v_scale;
    const float *k_gain, *v_gain;
    const __nv_bfloat16* q;
    int64_t q_stride;
    int32_t H, H_kv, group;
    int32_t causal, window, sinks;
    float scale_log2;
    __nv_bfloat16* o;
    float* lse;
    // lists: of token tile f = kvh * nt_cap + token of the batch (in sequence order)
    const int32_t *list, *list_cnt;
    int32_t nt_cap, cap;
    // parts of split tiles
    float* part_o;    // [runs, 2, 8 NT, D]
    float2* part_ml;  // [runs, 2, 8 NT] maximum (log2) and sum
    int4* joins;      // [runs] parts (0: none), first packed row (token * group + head), rows, kvh
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t bits(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

// Key tiles that the tokens at positions pos0 .. pos0 + ntok - 1 see some key
// of: the sink tiles 0 .. ns - 1 and lo .. lo + (n - ns) - 1.
__device__ __forceinline__ int32_t key_tiles(const Fp4Params& P, int32_t pos0, int32_t ntok, int32_t kl, int32_t& lo,
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

// A row tile of n key tiles counts n + kRowCost in a run, the constant for its start and end.
constexpr int32_t kRowCost = 2;
__device__ __forceinline__ int32_t row_units(int32_t n) { return max(n, 1) + kRowCost; }
__device__ __forceinline__ int32_t cut_at(int32_t x) { return max(x - kRowCost, 0); }

// Row tile t of a sequence: its rows are `rows` from row0 on (token * group + head).
template <bool kLists>
struct Tiles {
    int32_t group, wide;  // rows of a tile, at most
    __device__ __forceinline__ int32_t per_token() const { return (group + wide - 1) / wide; }
    __device__ __forceinline__ int32_t count(int32_t nq) const {
        return kLists ? nq * per_token() : (int32_t)(((int64_t)nq * group + wide - 1) / wide);
    }
    __device__ __forceinline__ void rows(int32_t t, int32_t nq, int32_t& row0, int32_t& n) const {
        if constexpr (kLists) {
            const int32_t per = per_token(), tok = t / per, h = (t - tok * per) * wide;
            row0 = tok * group + h;
            n = min(wide, group - h);
        } else {
            row0 = t * wide;
            n = min(wide, nq * group - row0);
        }
    }
};

template <int D, int NT, int kMode>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) k_fp4_rows(const __grid_constant__ Fp4Params P) {
    constexpr bool kLists = kMode == kListed;
    constexpr int R = 8 * NT;
    constexpr int kSteps = D / 16;          // products of S^T for 16 keys; of O^T as well
    constexpr int kKW = D / 32;             // words of a K row that a lane loads
    constexpr int kVW = D / 64;             // words of a V row that a lane loads
    constexpr int kRowO = D + 4;            // a row of O in shared memory, padded
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int64_t prefix[33];
    __shared__ int32_t start[5];            // this run's first unit: kvh, sequence, row tile, unit within it, tile of the head
    __shared__ float2 ml[kWarps][R];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, c = lane & 3;
    launch_dependents();
    wait_primary();
    if (threadIdx.x == 0) P.joins[blockIdx.x] = make_int4(0, 0, 0, 0);

    // ---------------------------------------------------------------- this block's run
    const Tiles<kLists> tiles{P.group, R};
    int32_t* cum = reinterpret_cast<int32_t*>(smem);  // row tiles of the sequences before
    int32_t nt;
    {
        const int32_t per = (P.b.seqs + kThreads - 1) / kThreads;
        const int32_t a = min((int32_t)threadIdx.x * per, P.b.seqs), e = min(a + per, P.b.seqs);
        int64_t mine = 0, all;
        for (int32_t s = a; s < e; ++s) {
            PagedSeq q;
            if (!paged_seq(P.b, s, q) && blockIdx.x == 0) raise_status(P.b.status, BSA_ERR_BOUNDS);
            cum[s] = tiles.count(q.nq);
            mine += cum[s];
        }
        int64_t at = block_prefix<kThreads>(mine, prefix, all);
        for (int32_t s = a; s < e; ++s) {
            const int32_t n = cum[s];
            cum[s] = (int32_t)min(at, (int64_t)INT32_MAX);
            at += n;
        }
        // (beyond this: only with starts that decrease, reported above)
        const int64_t most = kLists ? (int64_t)P.nt_cap * tiles.per_token() : (int64_t)P.b.tokens * P.group / R + P.b.seqs;
        nt = (int32_t)min(all, most);
    }
    __syncthreads();
    auto list_of = [&](int32_t kvh, int32_t i) -> int64_t {  // (row tile i of the head)
        return (int64_t)kvh * P.nt_cap + i / tiles.per_token();
    };
    auto tile_count = [&](int32_t kvh, int32_t i, int32_t t, const PagedSeq& q, int32_t& lo, int32_t& ns) -> int32_t {
        if constexpr (kLists) {
            lo = ns = 0;
            return P.list_cnt[list_of(kvh, i)];
        } else {
            int32_t row0, n;
            tiles.rows(t, q.nq, row0, n);
            const int32_t first = row0 / P.group, last = (row0 + n - 1) / P.group;
            return key_tiles(P, q.kl - q.nq + first, last - first + 1, q.kl, lo, ns);
        }
    };
    const int64_t rows = kLists ? (int64_t)nt * P.H_kv : nt;  // tiles whose counts differ
    const int64_t per_row = (rows + kThreads - 1) / kThreads;
    const int64_t f0 = min((int64_t)threadIdx.x * per_row, rows), f1 = min(f0 + per_row, rows);
    // walks this thread's tiles: visit(kvh, i, s, t, units)
    auto walk = [&](auto&& visit) {
        if (f0 >= f1) return;
        int32_t kvh = kLists ? (int32_t)(f0 / nt) : 0, i = (int32_t)(f0 - (int64_t)kvh * nt), s = 0;
        PagedSeq q;
        auto find = [&]() {
            int32_t lo = 0, hi = P.b.seqs;  // the last s with cum[s] <= i
            while (hi - lo > 1) {
                const int32_t mid = (lo + hi) >> 1;
                if (cum[mid] <= i) lo = mid;
                else hi = mid;
            }
            s = lo;
            paged_seq(P.b, s, q);
        };
        find();
        for (int64_t f = f0; f < f1; ++f) {
            const int32_t t = i - cum[s];
            int32_t lo, ns;
            if (visit(kvh, i, s, t, row_units(tile_count(kvh, i, t, q, lo, ns)))) return;
            ++i;
            if (i == nt) {
                i = 0;
                ++kvh;
                if (f + 1 < f1) find();
            } else if (s + 1 < P.b.seqs && cum[s + 1] <= i) {
                find();
            }
        }
    };
    int64_t mine = 0, total;
    walk([&](int32_t, int32_t, int32_t, int32_t, int32_t n) {
        mine += n;
        return false;
    });
    const int64_t before = block_prefix<kThreads>(mine, prefix, total);
    const int64_t units = kLists ? total : total * P.H_kv;
    const int32_t blocks = (int32_t)min((int64_t)gridDim.x, units);
    if ((int32_t)blockIdx.x >= blocks) return;
    const int64_t share = units / blocks;  // equal runs, the first `extra` of them one unit longer
    const int32_t extra = (int32_t)(units - share * blocks);
    auto run_start = [&](int32_t x) -> int64_t { return share * x + min(x, extra); };
    {
        const int64_t u0 = run_start(blockIdx.x), head = kLists ? 0 : u0 / total, x = kLists ? u0 : u0 - head * total;
        if (x >= before && x < before + mine) {
            int64_t at = before;
            walk([&](int32_t kvh, int32_t i, int32_t s, int32_t t, int32_t n) {
                if (x < at + n) {
                    start[0] = kLists ? kvh : (int32_t)head;
                    start[1] = s;
                    start[2] = t;
                    start[3] = (int32_t)(x - at);
                    start[4] = i;
                    return true;
                }
                at += n;
                return false;
            });
        }
    }
    __syncthreads();

    // ---------------------------------------------------------------- the run's row tiles
    float* const so = reinterpret_cast<float*>(smem);  // [warp][row][kRowO] (cum makes room)
    int32_t kvh = start[0], s = start[1], t = start[2], x0 = start[3], i = start[4];
    const int64_t u_end = run_start(blockIdx.x + 1);
    int64_t u = run_start(blockIdx.x);
    PagedSeq q;
    paged_seq(P.b, s, q);
    while (u < u_end) {
        int32_t lo_t, ns;
        const int32_t n_row = tile_count(kvh, i, t, q, lo_t, ns);
        const int32_t n_eff = max(n_row, 1), w = row_units(n_row);
        const int64_t left = u_end - u;
        const bool last = left < w - x0;  // the run ends within this row tile
        const int32_t j0 = cut_at(x0), j1 = min(last ? cut_at(x0 + (int32_t)left) : n_eff, n_row);
        const bool whole = j0 == 0 && !(last && j1 < n_eff);
        if (last && j1 <= j0) break;      // (nothing of it: only where the run ends)
        int32_t row0, nrows;
        tiles.rows(t, q.nq, row0, nrows);
        const int32_t tok0 = row0 / P.group;
        const int32_t pos_of0 = q.kl - q.nq;
        const float kg = P.k_gain != nullptr ? P.k_gain[kvh] : 1.0f;

        // queries: lane (r, c) has D / 4 values of rows r, r + 8, ..
        uint32_t qf[NT][kSteps][2];
        float fac[NT][2];               // of the rows of this lane's columns 2 c, 2 c + 1
        int32_t hi[NT][2], lo[NT][2], sk[NT][2];
        auto end = [&](int32_t p) -> int32_t { return P.causal ? min(q.kl, p + 1) : q.kl; };
#pragma unroll
        for (int b = 0; b < NT; ++b) {
            const int32_t row = row0 + min(8 * b + r, nrows - 1);  // (rows beyond the tile's: any; they are not stored)
            const int32_t tok = row / P.group, head = row - tok * P.group;
            const uint4* src = reinterpret_cast<const uint4*>(P.q + ((int64_t)q.q0 + tok) * P.q_stride +
                                                              (int64_t)(kvh * P.group + head) * D + c * (D / 4));
            uint4 raw[D / 32];
#pragma unroll
            for (int y = 0; y < D / 32; ++y) raw[y] = src[y];
            const uint32_t* wd = reinterpret_cast<const uint32_t*>(raw);
            uint32_t top = 0u;  // the largest exponent field of a finite value
#pragma unroll
            for (int y = 0; y < D / 8; ++y) {
                const uint32_t e0 = wd[y] >> 7 & 0xffu, e1 = wd[y] >> 23 & 0xffu;
                top = max(top, max(e0 == 0xffu ? 0u : e0, e1 == 0xffu ? 0u : e1));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int32_t e = max((int32_t)top - 127, -100) - 14;
            const float up = __int_as_float((127 - e) << 23);
#pragma unroll
            for (int y = 0; y < D / 8; ++y) {
                const float a = __uint_as_float(wd[y] << 16) * up, d = __uint_as_float(wd[y] & 0xffff0000u) * up;
                qf[b][y >> 1][y & 1] = bits(__floats2half2_rn(a, d));
            }
            const float down = __int_as_float((127 + e) << 23) * kg * P.scale_log2;
            fac[b][0] = __shfl_sync(0xffffffffu, down, 8 * c);
            fac[b][1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int32_t p = pos_of0 + (row0 + min(8 * b + 2 * c + y, nrows - 1)) / P.group;
                hi[b][y] = end(p);
                if constexpr (kMode == kWindow) {
                    lo[b][y] = p - P.window + 1;
                    sk[b][y] = min(P.sinks, hi[b][y]);
                }
            }
        }
        const int32_t p_first = pos_of0 + tok0, p_last = pos_of0 + (row0 + nrows - 1) / P.group;
        const int32_t all_hi = end(p_first), all_lo = p_last - P.window + 1, all_sk = min(P.sinks, all_hi);

        // ---- this warp's 16 keys of the key tiles j0 .. j1 - 1
        const int32_t* table = P.b.table + (int64_t)s * P.b.max_pages;
        const int32_t* list = kLists ? P.list + list_of(kvh, i) * P.cap : nullptr;
        auto key_tile = [&](int32_t j) -> int32_t {
            if constexpr (kLists) return list[j];
            else return j < ns ? j : lo_t + j - ns;
        };
        // lane l of a window of tiles: first key of tile w0 + l's sixteen, and its row in the cache (-1: none)
        int32_t key_cur, row_cur, key_nxt, row_nxt;
        const int32_t in_page = (warp * 16) % P.b.page;
        auto look = [&](int32_t w0, int32_t& key, int32_t& row) {
            key = 0;
            row = -1;
            const int32_t j = w0 + lane;
            if (j >= j1) return;
            key = key_tile(j) * 128 + warp * 16;
            if (key >= q.kl) return;
            int32_t id = table[key / P.b.page];
            if (id < 0 || id >= P.b.n_pages) {
                raise_status(P.b.status, BSA_ERR_BOUNDS);
                id = 0;  // (this row's result is unspecified)
            }
            row = (id * P.H_kv + kvh) * P.b.page + in_page;
        };
        struct Raw {
            uint32_t k[2][kKW];
            uint32_t ks[2];   // scales of the lane's groups, one or two bytes
            uint32_t v[4][kVW];
            uint32_t vs[4];
        };
        auto load = [&](int32_t row, Raw& x) {
            if (row < 0) return;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int64_t at = row + r + 8 * y;
                const uint8_t* src = P.k + at * (D / 2) + c * (D / 8);
                const uint8_t* ss = P.k_scale + at * (D / 16);
                if constexpr (D == 128) {
                    *reinterpret_cast<uint4*>(x.k[y]) = *reinterpret_cast<const uint4*>(src);
                    x.ks[y] = *reinterpret_cast<const uint16_t*>(ss + 2 * c);
                } else {
                    *reinterpret_cast<uint2*>(x.k[y]) = *reinterpret_cast<const uint2*>(src);
                    x.ks[y] = ss[c];
                }
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int64_t at = row + 2 * c + (y & 1) + 8 * (y >> 1);
                const uint8_t* src = P.v + at * (D / 2) + r * (D / 16);
                if constexpr (D == 128) *reinterpret_cast<uint2*>(x.v[y]) = *reinterpret_cast<const uint2*>(src);
                else x.v[y][0] = *reinterpret_cast<const uint32_t*>(src);
                x.vs[y] = P.v_scale[at * (D / 16) + (D == 128 ? r : r >> 1)];
            }
        };
        float acc[NT][kSteps][4] = {};
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                m[b][y] = -INFINITY;
                l[b][y] = 0.0f;
            }
        int32_t w0 = j0;
        look(j0, key_cur, row_cur);
        look(j0 + 32, key_nxt, row_nxt);
        Raw nxt;
        int32_t row_next = __shfl_sync(0xffffffffu, row_cur, 0), key_next = __shfl_sync(0xffffffffu, key_cur, 0);
        load(row_next, nxt);
        for (int32_t j = j0; j < j1; ++j) {
            const Raw x = nxt;
            const int32_t row = row_next, kb = key_next;
            if (j + 1 - w0 == 32) {
                w0 += 32;
                key_cur = key_nxt;
                row_cur = row_nxt;
                look(w0 + 32, key_nxt, row_nxt);
            }
            row_next = __shfl_sync(0xffffffffu, row_cur, (j + 1 - w0) & 31);
            key_next = __shfl_sync(0xffffffffu, key_cur, (j + 1 - w0) & 31);
            if (j + 1 < j1) load(row_next, nxt);
            if (row < 0) continue;
            // S^T = K Q^T
            float sc[NT][4] = {};
            {
                __half2 s2[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) s2[y] = fp4_scales(x.ks[y]);
#pragma unroll
                for (int wd = 0; wd < kKW; ++wd) {
                    __half2 a[4], d[4];
                    fp4_levels(x.k[0][wd], a);
                    fp4_levels(x.k[1][wd], d);
                    const __half2 sa = D == 128 && wd >= kKW / 2 ? __high2half2(s2[0]) : __low2half2(s2[0]);
                    const __half2 sd = D == 128 && wd >= kKW / 2 ? __high2half2(s2[1]) : __low2half2(s2[1]);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t op[4] = {bits(__hmul2(a[2 * y], sa)), bits(__hmul2(d[2 * y], sd)),
                                                bits(__hmul2(a[2 * y + 1], sa)), bits(__hmul2(d[2 * y + 1], sd))};
#pragma unroll
                        for (int b = 0; b < NT; ++b) mma16816(sc[b], op, qf[b][2 * wd + y][0], qf[b][2 * wd + y][1]);
                    }
                }
            }
            bool seen = kb + 16 <= all_hi;
            if constexpr (kMode == kWindow) seen = (seen && kb >= all_lo) || kb + 16 <= all_sk;
            bool over = false;
#pragma unroll
            for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    sc[b][y] *= fac[b][y & 1];
                    if (!seen) {
                        const int32_t key = kb + r + 8 * (y >> 1);
                        bool vis = key < hi[b][y & 1];
                        if constexpr (kMode == kWindow) vis = (vis && key >= lo[b][y & 1]) || key < sk[b][y & 1];
                        if (!vis) sc[b][y] = -INFINITY;
                    }
                    over |= !(sc[b][y] <= m[b][y & 1] + kRaise);
                }
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int b = 0; b < NT; ++b)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float top = fmaxf(sc[b][y], sc[b][y + 2]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        // (row by row: what one row holds does not show in another's last bits)
                        const float m_new = top > m[b][y] + kRaise ? top : m[b][y];
                        const float keep = m[b][y] == -INFINITY ? 1.0f : ex2(m[b][y] - m_new);  // (l and O are 0 still)
                        m[b][y] = m_new;
                        l[b][y] *= keep;
#pragma unroll
                        for (int z = 0; z < kSteps; ++z) {
                            acc[b][z][y] *= keep;
                            acc[b][z][y + 2] *= keep;
                        }
                    }
            }
            uint32_t pt[NT][2];
#pragma unroll
            for (int b = 0; b < NT; ++b) {
                float p[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float base = m[b][y & 1] == -INFINITY ? 0.0f : m[b][y & 1];
                    p[y] = ex2(sc[b][y] - base);
                    l[b][y & 1] += p[y];
                }
                pt[b][0] = transpose8(bits(__floats2half2_rn(p[0], p[1])));
                pt[b][1] = transpose8(bits(__floats2half2_rn(p[2], p[3])));
            }
            // O^T += V^T P^T
            {
                const __half2 sa = fp4_scales(x.vs[0] | x.vs[1] << 8), sd = fp4_scales(x.vs[2] | x.vs[3] << 8);
                constexpr uint32_t kLow = 0x0f0f0f0fu;
#pragma unroll
                for (int wd = 0; wd < kVW; ++wd) {
                    __half2 a[4], b0[4], d[4], e[4];
                    const uint32_t v0 = x.v[0][wd], v1 = x.v[1][wd], v2 = x.v[2][wd], v3 = x.v[3][wd];
                    fp4_levels((v0 & kLow) | (v1 << 4 & ~kLow), a);
                    fp4_levels((v0 >> 4 & kLow) | (v1 & ~kLow), b0);
                    fp4_levels((v2 & kLow) | (v3 << 4 & ~kLow), d);
                    fp4_levels((v2 >> 4 & kLow) | (v3 & ~kLow), e);
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint32_t op[4] = {bits(__hmul2(a[y], sa)), bits(__hmul2(b0[y], sa)), bits(__hmul2(d[y], sd)),
                                                bits(__hmul2(e[y], sd))};
#pragma unroll
                        for (int b = 0; b < NT; ++b) mma16816(acc[b][4 * wd + y], op, pt[b][0], pt[b][1]);
                    }
                }
            }
        }

        // ---- the eight warps' parts
        __syncthreads();  // the part before (and cum) has been read
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[b][y] += __shfl_xor_sync(0xffffffffu, l[b][y], d);
                const int row = 8 * b + 2 * c + y;
                if (row < nrows) {
                    if (r == 0) ml[warp][row] = make_float2(m[b][y], l[b][y]);
                    float* to = so + (warp * R + row) * kRowO + r * (D / 8);
#pragma unroll
                    for (int z = 0; z < kSteps; z += 2)
                        *reinterpret_cast<float4*>(to + 2 * z) =
                            make_float4(acc[b][z][y], acc[b][z][y + 2], acc[b][z + 1][y], acc[b][z + 1][y + 2]);
                }
            }
        __syncthreads();
        {
            constexpr int kLanes = D / 4;
            const int col = threadIdx.x % kLanes;
            const int32_t slot = 2 * blockIdx.x + (j0 == 0 ? 1 : 0);
            for (int32_t row = threadIdx.x / kLanes; row < nrows; row += kThreads / kLanes) {
                float M = -INFINITY, sum = 0.0f, out[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int x = 0; x < kWarps; ++x) M = fmaxf(M, ml[x][row].x);
#pragma unroll
                for (int x = 0; x < kWarps; ++x) {
                    const float2 y = ml[x][row];
                    if (y.x == -INFINITY && y.y == 0.0f) continue;  // no visible key
                    const float f = ex2(y.x - M);
                    sum = fmaf(f, y.y, sum);
                    const float4 v = *reinterpret_cast<const float4*>(so + (x * R + row) * kRowO + 4 * col);
                    out[0] = fmaf(f, v.x, out[0]);
                    out[1] = fmaf(f, v.y, out[1]);
                    out[2] = fmaf(f, v.z, out[2]);
                    out[3] = fmaf(f, v.w, out[3]);
                }
                if (whole) {
                    const float inv = (sum == 0.0f ? 0.0f : 1.0f / sum) * (P.v_gain != nullptr ? P.v_gain[kvh] : 1.0f);
                    const int32_t x = row0 + row, tok = x / P.group;
                    const int64_t at = ((int64_t)q.q0 + tok) * P.H + kvh * P.group + (x - tok * P.group);
                    *reinterpret_cast<uint2*>(P.o + at * D + 4 * col) =
                        make_uint2(pack_bf16(out[0] * inv, out[1] * inv), pack_bf16(out[2] * inv, out[3] * inv));
                    if (col == 0) P.lse[at] = sum == 0.0f ? -INFINITY : (M + log2f(sum)) * kLn2;
                } else {
                    const int64_t at = (int64_t)slot * R + row;
                    *reinterpret_cast<float4*>(P.part_o + at * D + 4 * col) = make_float4(out[0], out[1], out[2], out[3]);
                    if (col == 0) P.part_ml[at] = make_float2(M, sum);
                }
            }
        }
        if (threadIdx.x == 0 && last && j0 == 0) {
            // a split row tile begins here; its last part is in the run of its last unit
            const int64_t stop = u + (w - x0);
            const int64_t longer = (share + 1) * extra;  // units of the longer runs
            const int64_t z = stop <= longer ? (stop - 1) / (share + 1) : extra + (stop - 1 - longer) / share;
            P.joins[blockIdx.x] = make_int4((int32_t)(z - blockIdx.x + 1), q.q0 * P.group + row0, nrows, kvh);
        }
        // on to the next row tile
        u += w - x0;
        x0 = 0;
        if (u < u_end) {
            ++t;
            if (++i == nt) {  // the next head
                i = t = s = 0;
                ++kvh;
                paged_seq(P.b, 0, q);
            }
            while (t >= tiles.count(q.nq) && s + 1 < P.b.seqs) {
                t = 0;
                paged_seq(P.b, ++s, q);
            }
        }
    }
}

// Joins the parts of split row tiles: O = sum_c 2^(m_c - M) O_c / l with M the largest m_c
// and l = sum_c 2^(m_c - M) l_c, parts in key order.  Thread block (c, y) takes kJoinThreads /
// (D / 4) rows of the tile that begins in k_fp4_rows' block c: its slot 1, then slot 0 of the blocks after it.
constexpr int kJoinThreads = 256;
template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads) k_fp4_join(const __grid_constant__ Fp4Params P) {
    launch_dependents();
    wait_primary();
    constexpr int kLanes = D / 4, R = 8 * NT;
    const int c = threadIdx.x % kLanes;
    const int32_t row = blockIdx.y * (kJoinThreads / kLanes) + threadIdx.x / kLanes;
    const int32_t run = blockIdx.x;
    const int4 jn = P.joins[run];
    if (jn.x == 0 || row >= jn.z) return;
    const uint32_t peers = kLanes == 32 ? 0xffffffffu : 0xffffu << (threadIdx.x & 16);  // this row's lanes
    auto part = [&](int32_t x) -> int64_t { return (((int64_t)run + x) * 2 + (x == 0 ? 1 : 0)) * R + row; };
    float M = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    // kLanes parts at a time, each thread the maximum and sum of one: all loads at once
    for (int32_t x0 = 0; x0 < jn.x; x0 += kLanes) {
        const int32_t n = min(jn.x - x0, kLanes);
        const float2 y = c < n ? P.part_ml[part(x0 + c)] : make_float2(-INFINITY, 0.0f);
        const bool none = y.x == -INFINITY && y.y == 0.0f;  // no visible key in this part
        float top = y.x;
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) top = fmaxf(top, __shfl_xor_sync(peers, top, d));
        const float M_new = fmaxf(M, top);
        const float keep = M == -INFINITY ? 1.0f : ex2(M - M_new);  // (l and o are 0 still)
        M = M_new;
        const float f = none ? 0.0f : ex2(y.x - M);
        float sum = none ? 0.0f : f * y.y;
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) sum += __shfl_xor_sync(peers, sum, d);
        l = fmaf(l, keep, sum);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] *= keep;
#pragma unroll 8
        for (int32_t x = 0; x < n; ++x) {
            const float fx = __shfl_sync(peers, f, x, kLanes);
            const bool skip = __shfl_sync(peers, (int)none, x, kLanes) != 0;
            const float4 v = *reinterpret_cast<const float4*>(P.part_o + part(x0 + x) * D + 4 * c);
            o[0] = skip ? o[0] : fmaf(fx, v.x, o[0]);
            o[1] = skip ? o[1] : fmaf(fx, v.y, o[1]);
            o[2] = skip ? o[2] : fmaf(fx, v.z, o[2]);
            o[3] = skip ? o[3] : fmaf(fx, v.w, o[3]);
        }
    }
    const float inv = (l == 0.0f ? 0.0f : 1.0f / l) * (P.v_gain != nullptr ? P.v_gain[jn.w] : 1.0f);
    const int32_t x = jn.y + row, tok = x / P.group;
    const int64_t at = (int64_t)tok * P.H + jn.w * P.group + (x - tok * P.group);
    *reinterpret_cast<uint2*>(P.o + at * D + 4 * c) =
        make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
    if (c == 0) P.lse[at] = l == 0.0f ? -INFINITY : (M + log2f(l)) * kLn2;
}

// ---------------------------------------------------------------- host side
// Workspace: joins, maxima and sums, O parts; then the tokens' lists.
struct Layout {
    size_t joins, ml, o, cnt, list, who, total;
    int32_t list_rows, cap;
};
Layout layout(const PagedForwardArgs& a) {
    Layout L{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t p = at;
        at += (bytes + 255) & ~(size_t)255;
        return p;
    };
    L.joins = take(sizeof(int4) * kRuns);
    L.ml = take(sizeof(float2) * kRuns * 2 * 8 * kMaxNT);
    L.o = take(sizeof(float) * kRuns * 2 * 8 * kMaxNT * (size_t)a.D);
    if (a.sel_width > 0) {
        const int64_t blocks = ((int64_t)a.max_pages * a.page + 127) / 128;
        L.cap = (int32_t)(blocks < a.sel_width ? blocks : a.sel_width);
        L.list_rows = a.tokens + a.seqs;
        const size_t rows = (size_t)a.H_kv * L.list_rows;
        L.cnt = take(sizeof(int32_t) * rows);
        L.list = take(sizeof(int32_t) * rows * L.cap);
        L.who = take(sizeof(uint32_t) * rows * L.cap);
    }
    L.total = at;
    return L;
}

template <int D, int NT, int kMode>
bsa_status launch_rows(const Fp4Params& P, cudaStream_t stream) {
    const size_t merge = sizeof(float) * kWarps * 8 * NT * (D + 4), cum = sizeof(int32_t) * (size_t)P.b.seqs;
    constexpr size_t most = 72 << 10;
    const size_t smem = merge > cum ? merge : cum;
    static DeviceSetup setup;
    static int sms[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return BSA_ERR_CUDA;
    const bool ready = setup.once(dev, [&] {
        return cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
               cudaFuncSetAttribute(k_fp4_rows<D, NT, kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) ==
                   cudaSuccess;
    });
    if (!ready) return BSA_ERR_CUDA;
    const int want = sms[dev] * (NT == 1 ? 2 : 1);
    const int grid = want < kRuns ? want : kRuns;
    constexpr int per_join = kJoinThreads / (D / 4);
    if (launch_chained(k_fp4_rows<D, NT, kMode>, dim3((unsigned)grid), kThreads, smem, stream, P) != cudaSuccess ||
        launch_chained(k_fp4_join<D, NT>, dim3((unsigned)grid, (8 * NT + per_join - 1) / per_join), kJoinThreads, 0, stream, P) !=
            cudaSuccess)
        return BSA_ERR_CUDA;
    return BSA_OK;
}

template <int kMode>
bsa_status launch_mode(const Fp4Params& P, int32_t D, bool wide, cudaStream_t stream) {
    if (D == 128) return wide ? launch_rows<128, 2, kMode>(P, stream) : launch_rows<128, 1, kMode>(P, stream);
    return wide ? launch_rows<64, 2, kMode>(P, stream) : launch_rows<64, 1, kMode>(P, stream);
}

}  // namespace

size_t fp4_forward_workspace(const PagedForwardArgs& a) { return layout(a).total; }

bsa_status launch_fp4_forward(const Fp4ForwardArgs& x, void* workspace, int32_t* status, cudaStream_t stream) {
    const PagedForwardArgs& a = x.f;
    const Layout L = layout(a);
    Fp4Params P;
    memset(&P, 0, sizeof(P));
    P.b = PagedBatch{a.q_start, a.kv_len, a.table, a.seqs, a.tokens, a.max_pages, a.page, a.n_pages, status};
    P.k = static_cast<const uint8_t*>(a.k_cache);
    P.v = static_cast<const uint8_t*>(a.v_cache);
    P.k_scale = static_cast<const uint8_t*>(x.k_scale);
    P.v_scale = static_cast<const uint8_t*>(x.v_scale);
    P.k_gain = x.k_gain;
    P.v_gain = x.v_gain;
    P.q = static_cast<const __nv_bfloat16*>(a.q);
    P.q_stride = a.q_stride;
    P.H = a.H;
    P.H_kv = a.H_kv;
    P.group = a.H / a.H_kv;
    P.causal = a.causal;
    P.window = a.window < kMaxWindow ? a.window : kMaxWindow;
    P.sinks = a.sinks;
    P.scale_log2 = (a.scale > 0.f ? a.scale : 1.0f / sqrtf((float)a.D)) * kLog2e;
    P.o = static_cast<__nv_bfloat16*>(a.o);
    P.lse = a.lse;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    P.joins = reinterpret_cast<int4*>(ws + L.joins);
    P.part_ml = reinterpret_cast<float2*>(ws + L.ml);
    P.part_o = reinterpret_cast<float*>(ws + L.o);
    // rows of a sequence's new tokens, at most: more than eight want the wider tile
    const int64_t most = (int64_t)(x.max_new > 0 && x.max_new < a.tokens ? x.max_new : a.tokens) * P.group;
    if (a.sel != nullptr) {
        P.nt_cap = L.list_rows;
        P.cap = L.cap;
        int32_t* cnt = reinterpret_cast<int32_t*>(ws + L.cnt);
        int32_t* list = reinterpret_cast<int32_t*>(ws + L.list);
        const bsa_status c = launch_paged_union(a, 1, L.list_rows, L.cap, 1, list, cnt, reinterpret_cast<uint32_t*>(ws + L.who),
                                                status, stream);
        if (c != BSA_OK) return c;
        P.list = list;
        P.list_cnt = cnt;
        return launch_mode<kListed>(P, a.D, P.group > 8, stream);
    }
    return a.window > 0 ? launch_mode<kWindow>(P, a.D, most > 8, stream) : launch_mode<kPlain>(P, a.D, most > 8, stream);
}

}  // namespace bsa
