// Attention of new tokens over a paged key/value cache for sm_103a
// (tcgen05 + TMEM + TMA).
//
// What it computes.  For token i of sequence s at position p, query head h
// and the keys j < kv_len[s] that the mask leaves (causal: j <= p; window:
// j > p - window or j < sinks; lists: j / 128 among the token's blocks):
//     s_j = scale q . k_j,   LSE = ln sum_j exp(s_j),   O = sum_j exp(s_j - LSE) v_j
// in one pass over the keys with the running maximum and sum of the softmax.
//
// Tiles.  The G query heads that share a key/value head are rows of one
// query tile: row r is head r % G of the tile's token r / G, 128 / G tokens
// to a tile, so a single new token reads each key once for its G heads.  A
// key tile is 128 positions: 128 / page pages, each one TMA box.  One tile
// pair costs the tensor core about 0.6 us an SM and the memory about 1.5 us
// (64 KB at a 152nd of the card's rate), so the same 128-row tile serves
// single tokens, whose time is the cache's, and prompts, whose time is the
// products'.
//
// Split.  All (key/value head, sequence, query tile, key tile) units are laid
// out in that order and cut into equal runs, one for each of at most 152
// thread blocks: long rows are split over many, short ones run several to a
// block, and no host knowledge of the lengths is needed.  Where the cache is
// read by many query tiles and is larger than L2, each block takes up to four
// runs, a quarter of the units apart: at any time all blocks work on
// neighbouring heads, whose keys and values stay in L2 (a chunk of 1024 tokens
// over 65536, 268 MB: 1.8 GB of DRAM reads with one run each).  A row that a cut
// splits leaves its parts (O, maximum, sum, all fp32) in the workspace;
// k_paged_join adds them in key order, so a call's result does not depend on
// timing.
//
// Warp roles (16 warps): 0 cuts the run into segments (one query tile's part
// of the run), tells the others through a ring of descriptors and loads the K
// tiles, 11 the V tiles (pages of 16 tokens are up to 16 copies a tile; with one
// warp for both, each copy by a lane of its own, a pair took 2,000 cycles to
// issue); 1 loads the query tiles and issues the products Q K^T, 10 the products
// P V (a warp that issues both spends as long waiting and committing as the
// tensor core has work queued: with one, a tile pair, 1,112 cycles of tensor
// work, took 1,830 cycles, of which the softmax waited 720 for scores); 2 .. 9
// are the softmax (four threads a row, see bsa_rows.cuh); 12 .. 15 normalise and
// store a segment's rows while the softmax is at the next one (it lost about
// 5,000 cycles a segment to that).
// Shared memory: the Q tile and a ring of K/V tiles.  Tensor memory: three
// score buffers and O.  Tiles are numbered through the whole run, across the
// borders of segments: Q K_g is issued as soon as its score buffer is free (P V of
// tile g - 3 has read it), so that the next segment's scores are there when the
// softmax comes to them.
//
// Rounding.  The weights exp(s - m) are rounded to bf16 for the product P V: the tensor
// core takes both operands in one type, and the values are bf16 (fp16 has not the range for
// weights up to 2^64, see softmax_rows; tf32 would have V converted and half the rate).
// Row sums add them unrounded.  O is 2.0 to 2.4e-3 (relative, in norm) from 64-bit values,
// where its own rounding to bf16 alone is 1.7e-3.
//
// What a row does not see may hold anything, NaN and infinities included.  Its
// scores are dropped by a select, and the value rows behind the end of a
// sequence are zeroed in shared memory before the product (0 times NaN is NaN).
// A value that one row of a tile sees and another does not cannot be zeroed: a
// row whose O comes out not finite, and that hides such a value in its segment
// (see bad_values), is computed again from its own keys alone (see own_keys_row).
// (One bad value that all rows see: 4000 rows over 4250 keys took 33 ms without the look
// at what they hide, 0.15 ms with it, as without the value.)
//
// Measured, 32 + 8 heads of 128: 64 tokens over 1.7 GB of keys and values 254 us
// (the copy rate); one token over 131072 90 us with the join (6.2 TB/s while it reads); a
// prompt of 8192 344 us (0.84 of the burst rate of a plain product; 387 us called in a
// loop, under the power limit), where the
// tensor core is busy 70 % of the time and the softmax hardly ever waits: 1,370
// cycles a tile pair, of which loading the scores takes 160, the exponentials of two
// warps to a scheduler 800 (512 is the least), storing 130.  Two groups of softmax
// warps on alternate tiles (392 us) and halves of a tile loaded ahead (378 us) were
// slower: what they overlap they lose to a tile's longer way.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "bsa_device_setup.h"
#include "bsa_internal.h"
#include "bsa_paged.cuh"
#include "bsa_paged_wait.cuh"
#include "bsa_rows.cuh"
#include "bsa_tma_host.h"

namespace bsa {
namespace {

// positions lie within 2^24 of zero: longer windows are no longer, and position - window stays in 32 bits
constexpr int32_t kMaxWindow = 1 << 26;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;                          // rescale O when a maximum grows by > 2^8
constexpr float kSumLimit = 18446744073709551616.0f;      // 2^64, see softmax_rows
constexpr int kSBuf = 3;                                  // TMEM score buffers
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 384;
constexpr int kProducer = 0, kMmaQK = 1, kSoftmax0 = 2, kSoftmaxWarps = 8, kMmaPV = 10, kVLoad = 11;
constexpr int kStore0 = 12, kStoreWarps = 4;
constexpr int kThreads = 32 * 16;
constexpr int kDesc = 4;                                  // segment descriptors in flight
constexpr int kConsumers = kSoftmaxWarps + kStoreWarps + 3;  // warps that read a descriptor
constexpr int kBox = 128 * 128;                           // 128 rows of 64 bf16

// kMode: which keys a row sees besides the causal and length limits.
enum { kPlain = 0, kWindow = 1, kListed = 2 };

template <int D>
struct Cfg {
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = kBox * kHalves;
    static constexpr int kStages = D == 128 ? 6 : 12;
    static constexpr int kData = kTile * (1 + kStages);
    static constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 128, 0, 0);
    static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, 0, 1);
};

// One query tile's part of the run, as the producer tells it.
struct Segment {
    int32_t n;          // key tiles (0: none, the rows are empty; -1: no more segments)
    int32_t seq;
    int32_t q0, ntok;   // first token (packed axis) and tokens of the query tile
    int32_t kvh;
    int32_t pos0, kl;   // position of the first token, keys in the cache
    int32_t j0;         // first of the tile's key tiles in this segment
    int32_t lo, ns;     // key tile of number j: j < ns ? j : lo + j - ns (without lists)
    int32_t list;       // with lists: row of the tile lists
    int32_t slot;       // -1: the whole row is here; else its part slot: 2 run + 0 or 1
};

constexpr int kPhases = kPagedRuns / kPagedBlocks;     // runs of a thread block, at most
constexpr int64_t kPhaseBytes = 64ll << 20;            // of keys and values that a run's heads may hold (half of L2)

struct Shared {
    uint64_t full[16];
    uint64_t empty[16];
    uint64_t q_full, q_empty;
    uint64_t p_full[kSBuf];   // P_g has been written (and O rescaled)
    uint64_t o_free;          // the segment's O has been read
    uint64_t ml_full, ml_empty;  // a segment's maxima and sums are in ml, have been read
    uint64_t mma_done;
    uint64_t seg_full[kDesc], seg_empty[kDesc];
    Watch watch;
    Segment seg[kDesc];
    float2 ml[128];           // of a segment's rows: maximum (log2) and sum (before: block_prefix's words)
    int32_t start[kPhases][5];  // of each run the first unit: key/value head, sequence, query tile, unit; tile within the head
    PagedSeq start_seq[kPhases];  // its sequence's entry
    uint32_t tmem_base;
};

template <int n>
struct Pages {
    static constexpr int value = n;
};

struct Params {
    CUtensorMap map_q, map_q1;  // (D, H, tokens): box 64 x G x (128 / G), 64 x G x 1
    CUtensorMap map_k, map_v;   // (64, slots, D / 64): box 64 x page x boxed halves
    PagedBatch b;
    int32_t H, H_kv, group, tpt;  // tpt: tokens of a query tile
    int32_t causal, window, sinks;
    float scale_log2;
    const __nv_bfloat16 *q, *k_cache, *v_cache;  // for own_keys_row
    int64_t q_stride;
    __nv_bfloat16* o;
    float* lse;
    // lists (null: every visible key tile): tile f = kvh * nt_cap + i
    const int32_t* list;      // [H_kv * nt_cap, cap] key tiles, ascending
    const int32_t* list_cnt;  // [H_kv * nt_cap]
    const uint32_t* list_who; // [H_kv * nt_cap, cap, words] bit t: token t of the query tile sees the key tile
    int32_t nt_cap, cap, words;
    // workspace of split rows
    float* part_o;            // [runs, 2, 128, D]
    float2* part_ml;          // [runs, 2, 128] maximum (log2) and sum
    int4* joins;              // [runs] parts (0: none), q0, ntok, kvh
};

// The first and the last of a sequence's keys from .. to - 1 whose value row is not
// finite (first > last: none).  The whole warp works on it.
struct BadKeys {
    int32_t first, last;
};
template <int D>
__device__ __noinline__ BadKeys bad_values(const Params& P, int32_t seq, int32_t kvh, int32_t from, int32_t to) {
    const int lane = threadIdx.x & 31;
    const int32_t* table = P.b.table + (int64_t)seq * P.b.max_pages;
    int32_t first = INT32_MAX, last = -1;
    for (int32_t key = max(from, 0) + lane; key < to; key += 32) {
        int32_t id = table[key / P.b.page];
        if (id < 0 || id >= P.b.n_pages) id = 0;  // (reported by the loading warps)
        const __nv_bfloat16* row = P.v_cache + (((int64_t)id * P.H_kv + kvh) * P.b.page + key % P.b.page) * D;
        bool bad = false;
#pragma unroll 4
        for (int d = 0; d < D; d += 8) {
            const uint4 x = *reinterpret_cast<const uint4*>(row + d);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)  // (all bits of an exponent are set)
                bad |= (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
        }
        if (bad) {
            first = min(first, key);
            last = key;
        }
    }
    __syncwarp();
    return {__reduce_min_sync(0xffffffffu, first), __reduce_max_sync(0xffffffffu, last)};
}

// O = sum_j 2^(s_j - m) v_j of one row over the keys of a segment that the row
// sees, read from the cache one by one; to out (fp32, unscaled) or, times inv, to
// orow.  The whole warp works on it, lane l values l D / 32 ..: slow (a row and
// key tile take some 10 us), and for rows next to values that are not finite only;
// busy tells the warps that wait meanwhile that it goes on.
template <int D, int kMode>
__device__ __noinline__ void own_keys_row(const Params& P, const Segment& sg, int32_t row_of_tile, float m, float inv, uint64_t* busy) {
    const int lane = threadIdx.x & 31;
    const int32_t tok = row_of_tile / P.group, head = row_of_tile - tok * P.group;
    constexpr int kPer = D / 32;
    const int32_t p = sg.pos0 + tok, hi = P.causal ? min(sg.kl, p + 1) : sg.kl;
    const int32_t lo = kMode == kWindow ? p - P.window + 1 : 0, sk = kMode == kWindow ? min(P.sinks, hi) : 0;
    const int32_t page = P.b.page;
    const int32_t* table = P.b.table + (int64_t)sg.seq * P.b.max_pages;
    const __nv_bfloat16* q = P.q + (int64_t)(sg.q0 + tok) * P.q_stride + (int64_t)(sg.kvh * P.group + head) * D;
    float acc[kPer] = {};
    for (int32_t j = 0; j < sg.n; ++j) {
        int32_t kt;
        bool listed = true;
        if constexpr (kMode == kListed) {
            const int64_t e = (int64_t)sg.list * P.cap + sg.j0 + j;
            kt = P.list[e];
            listed = (P.list_who[e * P.words + (tok >> 5)] >> (tok & 31)) & 1u;
        } else {
            kt = sg.j0 + j < sg.ns ? sg.j0 + j : sg.lo + sg.j0 + j - sg.ns;
        }
        if (!listed) continue;
        for (int32_t k0 = 0; k0 < 128; k0 += 32) {
            const int32_t key = kt * 128 + k0 + lane;
            const bool see = (key < hi && key >= lo) || key < sk;
            int64_t row = 0;
            float pj = 0.f;
            if (see) {
                int32_t id = table[key / page];
                if (id < 0 || id >= P.b.n_pages) id = 0;  // (reported by the loading warps)
                row = (((int64_t)id * P.H_kv + sg.kvh) * page + key % page) * D;
                float dot = 0.f;
#pragma unroll 4
                for (int d = 0; d < D; d += 8) {
                    const uint4 a4 = *reinterpret_cast<const uint4*>(q + d);
                    const uint4 b4 = *reinterpret_cast<const uint4*>(P.k_cache + row + d);
                    const __nv_bfloat162 *a2 = reinterpret_cast<const __nv_bfloat162*>(&a4),
                                         *b2 = reinterpret_cast<const __nv_bfloat162*>(&b4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 a = __bfloat1622float2(a2[i]), b = __bfloat1622float2(b2[i]);
                        dot = fmaf(a.x, b.x, fmaf(a.y, b.y, dot));
                    }
                }
                pj = exp2f(fmaf(dot, P.scale_log2, -m));
            }
            const uint32_t seen = __ballot_sync(0xffffffffu, see);
#pragma unroll 1
            for (int i0 = 0; i0 < 32; i0 += 8) {
                __nv_bfloat162 v[8][kPer / 2];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t r = __shfl_sync(0xffffffffu, row, i0 + i);
#pragma unroll
                    for (int x = 0; x < kPer / 2; ++x)
                        v[i][x] = (seen >> (i0 + i)) & 1u
                                      ? *reinterpret_cast<const __nv_bfloat162*>(P.v_cache + r + lane * kPer + 2 * x)
                                      : __nv_bfloat162{};
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float w = __shfl_sync(0xffffffffu, pj, i0 + i);
#pragma unroll
                    for (int x = 0; x < kPer / 2; ++x) {
                        const float2 f = __bfloat1622float2(v[i][x]);
                        acc[2 * x] = fmaf(w, f.x, acc[2 * x]);
                        acc[2 * x + 1] = fmaf(w, f.y, acc[2 * x + 1]);
                    }
                }
            }
        }
        if (lane == 0) *reinterpret_cast<volatile uint64_t*>(busy) = globaltimer();
        bool nan = true;  // all of them: they stay so
#pragma unroll
        for (int x = 0; x < kPer; ++x) nan &= acc[x] != acc[x];
        if (__all_sync(0xffffffffu, nan)) break;
    }
    __nv_bfloat16* orow = P.o + ((int64_t)(sg.q0 + tok) * P.H + sg.kvh * P.group + head) * D;
    float* part = P.part_o + ((int64_t)max(sg.slot, 0) * 128 + row_of_tile) * D;
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
        if (sg.slot >= 0) part[lane * kPer + x] = acc[x];
        else orow[lane * kPer + x] = __float2bfloat16_rn(acc[x] * inv);
    }
}

// The rows of a segment, a row a lane, whose O is not finite: those that hide a value
// that is not either are computed from their own keys.  The others are what they are.
// What rows of a segment hide lies at the edges of what they see: behind their own
// positions, before their windows, behind the sinks.  With lists it is what they do
// not list, too.
template <int D, int kMode>
__device__ __noinline__ void rows_again(const Params& P, const Segment& sg, int32_t row, uint32_t again, float m, float inv, uint64_t* busy) {
    const int32_t p0 = sg.pos0, tok = row / P.group, p = p0 + tok;
    bool hides = false;
    if constexpr (kMode == kListed) {
        for (int32_t j = 0; j < sg.n && (again & ~__ballot_sync(0xffffffffu, hides)) != 0u; ++j) {
            const int64_t e = (int64_t)sg.list * P.cap + sg.j0 + j;
            const int32_t kt = P.list[e];
            const int32_t last = bad_values<D>(P, sg.seq, sg.kvh, kt * 128, min(sg.kl, kt * 128 + 128)).last;
            const bool listed = tok < sg.ntok && ((P.list_who[e * P.words + (tok >> 5)] >> (tok & 31)) & 1u);
            hides |= last >= 0 && (!listed || (P.causal && last > p));
            if ((threadIdx.x & 31) == 0) *reinterpret_cast<volatile uint64_t*>(busy) = globaltimer();
        }
    } else {
        const int32_t x = sg.j0 + sg.n - 1, last = p0 + sg.ntok - 1;
        const int32_t end = min(sg.kl, ((x < sg.ns ? x : sg.lo + x - sg.ns) + 1) * 128);  // of the tiles' keys
        hides = P.causal && bad_values<D>(P, sg.seq, sg.kvh, p0 + 1, end).last > p;
        if constexpr (kMode == kWindow) {
            hides |= bad_values<D>(P, sg.seq, sg.kvh, max(sg.lo * 128, P.sinks), min(end, last - P.window + 1)).first <= p - P.window;
            const BadKeys sink = bad_values<D>(P, sg.seq, sg.kvh, P.sinks, min(sg.kl, sg.ns * 128));
            hides |= sink.first <= sink.last;
        }
    }
    __syncwarp();  // the rows' own threads have written them
    for (again &= __ballot_sync(0xffffffffu, hides); again; again &= again - 1u) {
        const int i = __ffs(again) - 1;
        const float mi = __shfl_sync(0xffffffffu, m, i), li = __shfl_sync(0xffffffffu, inv, i);
        own_keys_row<D, kMode>(P, sg, (row & ~31) + i, mi, li, busy);
    }
}

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const Watch* w, int32_t* status) {
    return __all_sync(0xffffffffu, paged_wait(bar, parity, w, status));
}

// a / b; nearly every dividend fits 32 bits, whose division is much shorter.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
    return (a >> 32) == 0 && (b >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Tile K_g (V_g) of the run is use place / stages of ring slot place % stages: K
// tiles have the even slots, V tiles the odd ones.  The empty barrier of K_g's slot
// also tells the softmax that S_g is there, V_g's tells it that O holds P_g V_g, and
// the issuer of Q K_{g+3} that the score buffer is free (one commit for all).  Its
// next completion needs the P of a later tile, for which those who wait must come
// first, and the one before it (of tile g - stages / 2, at most g - 3) is known to be
// done to who has seen S_g.
__device__ __forceinline__ uint32_t place_k(uint32_t g) { return 2u * g; }
__device__ __forceinline__ uint32_t place_v(uint32_t g) { return 2u * g + 1u; }

// Key tiles that the tokens at positions pos0 .. pos0 + ntok - 1 see some key
// of: the sink tiles 0 .. ns - 1 and lo .. lo + (n - ns) - 1.
__device__ __forceinline__ int32_t key_tiles(const Params& P, int32_t pos0, int32_t ntok, int32_t kl, int32_t& lo,
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

// The run is cut by cost: a query tile of n key tiles counts n + kRowCost, the
// constant for its start and its end.  (A causal prompt of 8192, whose blocks have
// 8 to 50 query tiles each: 394 us with 1, 369 with 2, 358 with 4, 363 with 6.)
// A cut x units into the query tile leaves cut_at(x) of its key tiles on the left.
constexpr int32_t kRowCost = 4;
__device__ __forceinline__ int32_t row_units(int32_t n) { return max(n, 1) + kRowCost; }
__device__ __forceinline__ int32_t cut_at(int32_t x) { return max(x - kRowCost, 0); }

// Which of a thread's columns 8 kk and 8 kk + 1 (kk = 0 .. 15; bit 2 kk and the
// next) are below v.
__device__ __forceinline__ uint32_t columns_below(int32_t v) {
    const int32_t n = v <= 0 ? 0 : 2 * (v >> 3) + min(v & 7, 2);
    return n >= 32 ? ~0u : (1u << n) - 1u;
}

// One key tile of the online softmax for this thread's shares of rows a and b.
// dead: the row holds no token (its scores are anything; m = 0, and it takes
// part in no decision).  A live row that has seen no key yet has m = -inf.
// As long as no row of the warp is in that state (fresh, warp-uniform) the
// exponentials are taken against the running maxima without computing the
// tile's own; only a tile whose sums leave 2^64 (or are NaN) is redone with its
// maxima.  Returns true (warp-uniform) when O must be multiplied by alpha first.
template <typename Reload>
__device__ __forceinline__ bool softmax_rows(uint32_t (&s)[64], const bool (&dead)[2], float sl2, bool& fresh,
                                             float (&m)[2], float (&l)[2], float (&alpha)[2], Reload&& reload) {
    alpha[0] = alpha[1] = 1.0f;
    float la, lb;
    if (!fresh) {
        exp_rows<0>(s, sl2, -m[0], -m[1], la, lb);
        if (!__any_sync(0xffffffffu, (!dead[0] && !(la <= kSumLimit)) || (!dead[1] && !(lb <= kSumLimit)))) {
            l[0] += la;
            l[1] += lb;
            return false;
        }
        reload();
    }
    float mt[2];
    max_rows(s, mt[0], mt[1]);
    mt[0] *= sl2;
    mt[1] *= sl2;
    const bool rescale = __any_sync(0xffffffffu, (!dead[0] && m[0] != -INFINITY && mt[0] > m[0] + kRescale) ||
                                                     (!dead[1] && m[1] != -INFINITY && mt[1] > m[1] + kRescale));
    float bias[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (!dead[i]) {
            if (m[i] == -INFINITY) {
                m[i] = mt[i];  // O and l of the row are still 0
            } else if (rescale) {
                const float m_new = fmaxf(m[i], mt[i]);
                alpha[i] = ex2(m[i] - m_new);
                l[i] *= alpha[i];
                m[i] = m_new;
            }
        }
        bias[i] = m[i] == -INFINITY ? 0.0f : -m[i];  // (no key yet: every exponential is 0)
    }
    exp_rows<0>(s, sl2, bias[0], bias[1], la, lb);
    l[0] += la;
    l[1] += lb;
    fresh = __any_sync(0xffffffffu, m[0] == -INFINITY || m[1] == -INFINITY);
    return rescale;
}

template <int D, int kMode>
__global__ void __launch_bounds__(kThreads, 1) k_paged_forward(const __grid_constant__ Params P) {
    constexpr bool kLists = kMode == kListed;
    using C = Cfg<D>;
    constexpr uint32_t S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s_q = smem_u32(smem);
    const uint32_t s_ring = s_q + C::kTile;
    Shared* sh = reinterpret_cast<Shared*>(smem + C::kData);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    int32_t* const status = P.b.status;

    if (threadIdx.x == 32 * kStore0) {
        for (uint32_t s = 0; s < S; ++s) {
            mbar_init(smem_u32(&sh->full[s]), 1);
            mbar_init(smem_u32(&sh->empty[s]), 1);
        }
        mbar_init(smem_u32(&sh->q_full), 1);
        mbar_init(smem_u32(&sh->q_empty), 1);
        for (int s = 0; s < kSBuf; ++s) mbar_init(smem_u32(&sh->p_full[s]), 32 * kSoftmaxWarps);
        mbar_init(smem_u32(&sh->o_free), 32 * kStoreWarps);
        mbar_init(smem_u32(&sh->ml_full), 32 * kSoftmaxWarps);
        mbar_init(smem_u32(&sh->ml_empty), 32 * kStoreWarps);
        mbar_init(smem_u32(&sh->mma_done), 2);
        for (int d = 0; d < kDesc; ++d) {
            mbar_init(smem_u32(&sh->seg_full[d]), 1);
            mbar_init(smem_u32(&sh->seg_empty[d]), kConsumers);
        }
        fence_mbar_init();
        prefetch_tensormap(&P.map_k);
        prefetch_tensormap(&P.map_v);
        prefetch_tensormap(&P.map_q);
        prefetch_tensormap(&P.map_q1);
    }
    launch_dependents();
    wait_primary();
    if (threadIdx.x == kThreads - 1) {  // (the first threads have the batch to read)
        // (the producer writes them again where a row is split)
#pragma unroll
        for (int p = 0; p < kPhases; ++p) P.joins[p * gridDim.x + blockIdx.x] = make_int4(0, 0, 0, 0);
        sh->watch.busy = 0;
        // a block of this launch (or an unread earlier one) timed out: abandon
        sh->watch.abort = *reinterpret_cast<const volatile int32_t*>(status) == BSA_ERR_TIMEOUT;
    }

    // ---------------------------------------------------------------- this block's run
    // of sequence s: the query tiles of the sequences before it, its new tokens and
    // its length (the data area is free here)
    int32_t* cum = reinterpret_cast<int32_t*>(smem);
    int32_t* seq_nq = cum + P.b.seqs;
    int32_t* seq_kl = seq_nq + P.b.seqs;
    int32_t nt;       // query tiles of one key/value head
    int64_t kv_tiles;  // key tiles of one key/value head's cache
    {
        const int32_t per = (P.b.seqs + kThreads - 1) / kThreads;
        const int32_t a = min((int32_t)threadIdx.x * per, P.b.seqs), e = min(a + per, P.b.seqs);
        // (both counts in one word: neither reaches 2^32)
        int64_t mine = 0, all;
        for (int32_t s = a; s < e; ++s) {
            PagedSeq q;
            if (!paged_seq(P.b, s, q) && blockIdx.x == 0) raise_status(status, BSA_ERR_BOUNDS);
            seq_nq[s] = q.nq;
            seq_kl[s] = q.kl;
            mine += (q.nq + P.tpt - 1) / P.tpt + (q.nq > 0 ? (int64_t)((q.kl + 127) >> 7) << 32 : 0);
        }
        int64_t at = block_prefix<kThreads>(mine, reinterpret_cast<int64_t*>(sh->ml), all) & 0xffffffff;
        kv_tiles = all >> 32;
        all &= 0xffffffff;
        for (int32_t s = a; s < e; ++s) {
            cum[s] = (int32_t)min(at, (int64_t)P.nt_cap);
            at += (seq_nq[s] + P.tpt - 1) / P.tpt;
        }
        nt = (int32_t)min(all, (int64_t)P.nt_cap);  // (beyond: only with starts that decrease, reported above)
    }
    __syncthreads();
    const int32_t rows = kLists ? nt * P.H_kv : nt;  // tiles whose counts differ
    const int32_t per_row = (rows + kThreads - 1) / kThreads;
    const int32_t f0 = min((int32_t)threadIdx.x * per_row, rows), f1 = min(f0 + per_row, rows);
    // walks this thread's tiles: visit(kvh, i, s, t, units), tile i of the head being query tile t of sequence s
    auto walk = [&](auto&& visit) {
        if (f0 >= f1) return;
        int32_t kvh = kLists ? f0 / nt : 0, i = f0 - kvh * nt, s = 0;
        auto find = [&]() {
            int32_t lo = 0, hi = P.b.seqs;  // the last s with cum[s] <= i
            while (hi - lo > 1) {
                const int32_t mid = (lo + hi) >> 1;
                if (cum[mid] <= i) lo = mid;
                else hi = mid;
            }
            s = lo;
        };
        find();
        for (int32_t f = f0; f < f1; ++f) {
            const int32_t t = i - cum[s];
            int32_t n;
            if constexpr (kLists) {
                n = P.list_cnt[(int64_t)kvh * P.nt_cap + i];
            } else {
                int32_t lo, ns;
                const int32_t first = t * P.tpt, nq = seq_nq[s], kl = seq_kl[s];
                n = key_tiles(P, kl - nq + first, min(P.tpt, nq - first), kl, lo, ns);
            }
            if (visit(kvh, i, s, t, row_units(n)) || f + 1 == f1) return;
            ++i;
            if (i == nt) {
                i = 0;
                ++kvh;
                find();
            } else if (s + 1 < P.b.seqs && cum[s + 1] <= i) {
                find();
            }
        }
    };
    int64_t mine = 0, total;
    int4 only = make_int4(0, 0, 0, 0);  // a thread with one tile need not walk again,
    PagedSeq only_seq{0, 0, 0};         // and has its sequence at hand when it is asked for
    walk([&](int32_t kvh, int32_t i, int32_t s, int32_t t, int32_t n) {
        mine += n;
        only = make_int4(kvh, s, t, i);
        if (f1 - f0 == 1) paged_seq(P.b, s, only_seq);
        return false;
    });
    const int64_t before = block_prefix<kThreads>(mine, reinterpret_cast<int64_t*>(sh->ml), total);
    const int64_t units = kLists ? total : total * P.H_kv;
    // runs: one for each thread block, or where key tiles are read several times and
    // do not all stay in L2, several (of 16 units at least)
    int32_t phases = 1;
    const int64_t heads_tiles = kv_tiles * P.H_kv, kv_bytes = heads_tiles * (128 * D * 4);
    if (kv_bytes > kPhaseBytes && units - (int64_t)kRowCost * nt * P.H_kv > 2 * heads_tiles)
        phases = (int32_t)min(min((int64_t)kPhases, (kv_bytes + kPhaseBytes - 1) / kPhaseBytes),
                              max(units / (16 * (int64_t)gridDim.x), (int64_t)1));
    const int32_t blocks = (int32_t)min((int64_t)gridDim.x, units);
    if ((int32_t)blockIdx.x >= blocks) return;
    const int32_t runs = blocks * phases;
    // equal runs, the first `extra` of them one unit longer
    const int64_t share = divide(units, runs);
    const int32_t extra = (int32_t)(units - share * runs);
    auto run_start = [&](int32_t r) -> int64_t { return share * r + min(r, extra); };
    for (int32_t p = 0; p < phases; ++p) {
        const int64_t u0 = run_start(p * blocks + blockIdx.x);
        const int64_t head = kLists ? 0 : divide(u0, total), r = kLists ? u0 : u0 - head * total;
        if (r >= before && r < before + mine) {
            auto begin = [&](int32_t kvh, int32_t i, int32_t s, int32_t t, int64_t at) {
                sh->start[p][0] = kLists ? kvh : (int32_t)head;
                sh->start[p][1] = s;
                sh->start[p][2] = t;
                sh->start[p][3] = (int32_t)(r - at);
                sh->start[p][4] = i;
            };
            if (f1 - f0 == 1) {
                begin(only.x, only.w, only.y, only.z, before);
                sh->start_seq[p] = only_seq;
            } else {
                int64_t at = before;
                walk([&](int32_t kvh, int32_t i, int32_t s, int32_t t, int32_t n) {
                    if (r < at + n) {
                        begin(kvh, i, s, t, at);
                        paged_seq(P.b, s, sh->start_seq[p]);
                        return true;
                    }
                    at += n;
                    return false;
                });
            }
        }
    }
    const bool abandoned = sh->watch.abort != 0;
    if (warp == kMmaQK && !abandoned) {
        __syncwarp();  // some lanes have looked for the runs' starts
        tmem_alloc(smem_u32(&sh->tmem_base), kTmemCols);
        tmem_relinquish();
    }
    // cum, written by ordinary stores, makes room for TMA loads
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (abandoned) return;
    const uint32_t tmem = sh->tmem_base;

    // Segment k, for the warps that read descriptors (null: no more); they hand
    // it back when they are through with it.
    auto next_segment = [&](uint32_t k, bool& ok) -> const Segment* {
        if (!wait_warp(smem_u32(&sh->seg_full[k % kDesc]), (k / kDesc) & 1u, &sh->watch, status)) {
            ok = false;
            return nullptr;
        }
        const Segment* sg = &sh->seg[k % kDesc];
        return sg->n >= 0 ? sg : nullptr;
    };
    auto hand_back = [&](uint32_t k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh->seg_empty[k % kDesc]));
    };

    // The K (V) tiles of a segment, whose numbers in the run begin at g.  A tile is N
    // pages, each one copy of either 64-column half, or one of both where the page
    // fills the tile; the elected lane issues them back to back.
    auto load_pages = [&](auto pages, const Segment& sg, bool is_v, uint32_t& g) -> bool {
        constexpr int N = decltype(pages)::value, page = 128 / N;
        constexpr int per_window = 32 / N;  // key tiles whose pages one 32-lane read brings
        const int32_t n = sg.n, kl = sg.kl, kvh = sg.kvh;
        const int32_t* table = P.b.table + (int64_t)sg.seq * P.b.max_pages;
        const CUtensorMap* map = is_v ? &P.map_v : &P.map_k;
        // lane l of a window: the cache row of page l % N of key tile w0 + l / N (-1: behind
        // the sequence's end)
        auto fetch = [&](int32_t w0) -> int32_t {
            const int32_t j = w0 + lane / N;
            if (j >= n) return -1;
            int32_t kt;
            if constexpr (kLists) kt = P.list[(int64_t)sg.list * P.cap + sg.j0 + j];
            else kt = sg.j0 + j < sg.ns ? sg.j0 + j : sg.lo + sg.j0 + j - sg.ns;
            const int32_t pg = kt * N + lane % N;
            if (pg * page >= kl) return -1;
            int32_t id = table[pg];
            if (id < 0 || id >= P.b.n_pages) {
                raise_status(status, BSA_ERR_BOUNDS);
                id = 0;  // keeps the pipeline in step; this row's result is unspecified
            }
            return (id * P.H_kv + kvh) * page;
        };
        int32_t w0 = 0, cur = fetch(0), nxt = fetch(per_window);
        for (int32_t j = 0; j < n; ++j, ++g) {
            if (j >= w0 + per_window) {
                w0 += per_window;
                cur = nxt;
                nxt = fetch(w0 + per_window);
            }
            int32_t row[N], held = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                row[i] = __shfl_sync(0xffffffffu, cur, (j - w0) * N + i);
                held += row[i] >= 0;
            }
            const uint32_t pos = is_v ? place_v(g) : place_k(g), slot = pos % S;
            if (!wait_warp(smem_u32(&sh->empty[slot]), ((pos / S) & 1u) ^ 1u, &sh->watch, status)) return false;
            if (elect_one()) {
                const uint32_t fb = smem_u32(&sh->full[slot]), dst = s_ring + slot * C::kTile;
                mbar_arrive_expect_tx(fb, (uint32_t)(held * page * D * 2));
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (row[i] >= 0) {
#pragma unroll
                        for (int h = 0; h < (N == 1 ? 1 : C::kHalves); ++h)
                            tma_load_3d(dst + h * kBox + i * page * 128, map, 0, row[i], h, fb);
                    }
            }
            __syncwarp();
        }
        return true;
    };
    auto load_tiles = [&](const Segment& sg, bool is_v, uint32_t& g) -> bool {
        switch (P.b.page) {
            case 128: return load_pages(Pages<1>{}, sg, is_v, g);
            case 64: return load_pages(Pages<2>{}, sg, is_v, g);
            case 32: return load_pages(Pages<4>{}, sg, is_v, g);
            default: return load_pages(Pages<8>{}, sg, is_v, g);
        }
    };

    // No product may still be running when TMEM is freed.  The issuer that is through
    // first waits for the other one's, and that one perhaps for rows that are computed
    // from their own keys.
    auto finish_products = [&](bool ok) {
        if (elect_one()) mma_commit(smem_u32(&sh->mma_done));
        __syncwarp();
        if (!ok || !wait_warp(smem_u32(&sh->mma_done), 0, &sh->watch, status)) {
            if (ok && lane == 0) set_abort(&sh->watch, status);
            paged_drain(smem_u32(&sh->mma_done), 0, status);
        }
        __syncwarp();
    };

    if (warp == kProducer) {
        // ------------------------------------------------------------ segments and K tiles
        uint32_t k = 0, g = 0;  // segments and tiles so far
        bool ok = true;
        for (int32_t p = 0; p < phases && ok; ++p) {
        const int32_t run = p * blocks + blockIdx.x;
        int32_t kvh = sh->start[p][0], s = sh->start[p][1], t = sh->start[p][2], x0 = sh->start[p][3], i = sh->start[p][4];
        int64_t u = run_start(run), left = run_start(run + 1) - u;
        PagedSeq q = sh->start_seq[p];
        while (left > 0 && ok) {
            const int32_t first = t * P.tpt, ntok = min(P.tpt, q.nq - first);
            Segment sg;
            sg.seq = s;
            sg.q0 = q.q0 + first;
            sg.ntok = ntok;
            sg.kvh = kvh;
            sg.pos0 = q.kl - q.nq + first;
            sg.kl = q.kl;
            sg.lo = sg.ns = 0;
            sg.list = 0;
            int32_t n_row;
            if constexpr (kLists) {
                sg.list = kvh * P.nt_cap + i;
                n_row = P.list_cnt[sg.list];
            } else {
                n_row = key_tiles(P, sg.pos0, ntok, q.kl, sg.lo, sg.ns);
            }
            const int32_t n_eff = max(n_row, 1), w = row_units(n_row);
            const bool last = left < w - x0;  // the run ends within this query tile
            const int32_t j0 = cut_at(x0), j1 = last ? cut_at(x0 + (int32_t)left) : n_eff;
            if (j1 <= j0) break;              // (only where it ends)
            sg.j0 = j0;
            sg.n = n_row == 0 ? 0 : j1 - j0;
            sg.slot = j0 == 0 && j1 == n_eff ? -1 : 2 * run + (j0 == 0 ? 1 : 0);
            if (!wait_warp(smem_u32(&sh->seg_empty[k % kDesc]), ((k / kDesc) & 1u) ^ 1u, &sh->watch, status)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                sh->seg[k % kDesc] = sg;
                mbar_arrive(smem_u32(&sh->seg_full[k % kDesc]));
                // the query tile is loaded when its buffer is free; on its way into L2 now
                if (k > 0)
#pragma unroll
                    for (int h = 0; h < C::kHalves; ++h)
                        tma_prefetch_3d(ntok == 1 ? &P.map_q1 : &P.map_q, h * 64, kvh * P.group, sg.q0);
            }
            __syncwarp();
            ++k;
            ok = load_tiles(sg, false, g);
            if (lane == 0 && last && j0 == 0) {
                // a split row begins here; its last part is in the run of its last unit
                const int64_t end = u + (w - x0);
                const int64_t longer = (share + 1) * extra;  // units of the longer runs
                const int64_t c = end <= longer ? divide(end - 1, share + 1) : extra + divide(end - 1 - longer, share);
                P.joins[run] = make_int4((int32_t)(c - run + 1), sg.q0, ntok, kvh);
            }
            // on to the next query tile
            left -= w - x0;
            u += w - x0;
            x0 = 0;
            if (left > 0) {
                ++t;
                if (++i == (int32_t)nt) {  // the next head
                    i = t = s = 0;
                    ++kvh;
                    paged_seq(P.b, 0, q);
                }
                while (t * P.tpt >= q.nq && s + 1 < P.b.seqs) {
                    t = 0;
                    paged_seq(P.b, ++s, q);
                }
            }
        }
        }
        if (ok && wait_warp(smem_u32(&sh->seg_empty[k % kDesc]), ((k / kDesc) & 1u) ^ 1u, &sh->watch, status)) {
            if (lane == 0) {
                sh->seg[k % kDesc].n = -1;
                mbar_arrive(smem_u32(&sh->seg_full[k % kDesc]));
            }
        } else {
            ok = false;
        }
        if (!ok && lane == 0) set_abort(&sh->watch, status);
        // every issued copy must land before the block exits
        if (lane == 0)
            for (uint32_t x = g > S / 2 ? g - S / 2 : 0; x < g; ++x)
                paged_drain(smem_u32(&sh->full[place_k(x) % S]), (place_k(x) / S) & 1u, status);
        __syncwarp();
    } else if (warp == kVLoad) {
        // ------------------------------------------------------------ V tiles
        uint32_t g = 0;
        bool ok = true;
        for (uint32_t k = 0; ok; ++k) {
            const Segment* sp = next_segment(k, ok);
            if (sp == nullptr) break;
            const Segment sg = *sp;
            hand_back(k);
            ok = load_tiles(sg, true, g);
        }
        if (!ok && lane == 0) set_abort(&sh->watch, status);
        if (lane == 0)
            for (uint32_t x = g > S / 2 ? g - S / 2 : 0; x < g; ++x)
                paged_drain(smem_u32(&sh->full[place_v(x) % S]), (place_v(x) / S) & 1u, status);
        __syncwarp();
    } else if (warp == kMmaQK) {
        // ------------------------------------------------------------ query tiles, S = Q K^T
        // (the whole warp walks the schedule; one elected lane issues a tile's MMAs
        // and their commit)
        const uint64_t dq = smem_desc_sw128(s_q, 16, 1024);
        const uint64_t dk = smem_desc_sw128(s_ring, 16, 1024);
        uint32_t g = 0, nq = 0;
        bool ok = true;
        for (uint32_t k = 0; ok; ++k) {
            const Segment* sp = next_segment(k, ok);
            if (sp == nullptr) break;
            const int32_t n = sp->n, kvh = sp->kvh, q0 = sp->q0, ntok = sp->ntok;
            hand_back(k);
            if (n == 0) continue;
            // the segment before is done with the query tile's place
            if (nq > 0) ok = wait_warp(smem_u32(&sh->q_empty), (nq - 1u) & 1u, &sh->watch, status);
            if (!ok) break;
            if (elect_one()) {
                const bool one = ntok == 1;
                const uint32_t bar = smem_u32(&sh->q_full);
                mbar_arrive_expect_tx(bar, (uint32_t)((one ? 1 : P.tpt) * P.group * D * 2));
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h)
                    tma_load_3d(s_q + h * kBox, one ? &P.map_q1 : &P.map_q, h * 64, kvh * P.group, q0, bar);
            }
            __syncwarp();
            ok = wait_warp(smem_u32(&sh->q_full), nq++ & 1u, &sh->watch, status);
            for (int32_t j = 0; j < n && ok; ++j, ++g) {
                if (g >= kSBuf) {
                    // S buffer g % 3 is free once PV_{g-3} has read P_{g-3}
                    const uint32_t pv = place_v(g - kSBuf);
                    ok = wait_warp(smem_u32(&sh->empty[pv % S]), (pv / S) & 1u, &sh->watch, status);
                }
                const uint32_t pos = place_k(g), slot = pos % S;
                ok = ok && wait_warp(smem_u32(&sh->full[slot]), (pos / S) & 1u, &sh->watch, status);
                if (!ok) break;
                tc_fence_after();
                const uint64_t ks = dk + (uint64_t)((slot * C::kTile) >> 4);
                const uint32_t d_col = (g % kSBuf) * 128u;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = ((kk >> 2) * kBox + (kk & 3) * 32) >> 4;
                        mma_ss(tmem + d_col, dq + off, ks + off, C::kIdescQK, kk > 0 ? 1u : 0u);
                    }
                    mma_commit(smem_u32(&sh->empty[slot]));
                    if (j == n - 1) mma_commit(smem_u32(&sh->q_empty));
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) set_abort(&sh->watch, status);
        if (nq > 0 && lane == 0) paged_drain(smem_u32(&sh->q_full), (nq - 1u) & 1u, status);
        __syncwarp();
        finish_products(ok);
    } else if (warp == kMmaPV) {
        // ------------------------------------------------------------ O += P V
        const uint64_t dv = smem_desc_sw128(s_ring, kBox, 1024);
        uint32_t g = 0, segs = 0;
        bool ok = true;
        for (uint32_t k = 0; ok; ++k) {
            const Segment* sp = next_segment(k, ok);
            if (sp == nullptr) break;
            const int32_t n = sp->n;
            int32_t tail = 128;
            if (n > 0) {
                // the segment's last tile may hold the sequence's end: value rows behind it are zeroed
                const int32_t x = sp->j0 + n - 1;
                int32_t kt;
                if constexpr (kLists) kt = P.list[(int64_t)sp->list * P.cap + x];
                else kt = x < sp->ns ? x : sp->lo + x - sp->ns;
                tail = min(sp->kl - kt * 128, 128);
            }
            hand_back(k);
            if (n == 0) continue;
            for (int32_t j = 0; j < n && ok; ++j, ++g) {
                const uint32_t pos = place_v(g), slot = pos % S;
                ok = wait_warp(smem_u32(&sh->full[slot]), (pos / S) & 1u, &sh->watch, status);
                if (ok && j == n - 1 && tail < 128) {
                    // 16-byte pieces of rows tail .. 127 (a zero is the same in any swizzle)
                    const uint32_t tile = s_ring + slot * C::kTile;
                    for (int32_t y = tail * 8 + lane; y < 128 * 8; y += 32)
#pragma unroll
                        for (int h = 0; h < C::kHalves; ++h)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + h * kBox + y * 16), "r"(0)
                                         : "memory");
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                ok = ok && wait_warp(smem_u32(&sh->p_full[g % kSBuf]), (g / kSBuf) & 1u, &sh->watch, status);
                // a segment's first product overwrites O: the epilogue before must have read it
                if (ok && j == 0 && segs > 0) ok = wait_warp(smem_u32(&sh->o_free), (segs - 1u) & 1u, &sh->watch, status);
                if (!ok) break;
                tc_fence_after();
                const uint64_t vs = dv + (uint64_t)((slot * C::kTile) >> 4);
                const uint32_t p_col = (g % kSBuf) * 128u;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ts(tmem + kColO, tmem + p_col + kk * 8, vs + (uint64_t)(kk * 2048 >> 4), C::kIdescPV,
                               (j > 0 || kk > 0) ? 1u : 0u);
                    mma_commit(smem_u32(&sh->empty[slot]));
                }
                __syncwarp();
            }
            ++segs;
        }
        if (!ok && lane == 0) set_abort(&sh->watch, status);
        finish_products(ok);
    } else if (warp < kStore0) {
        // ------------------------------------------------------------ softmax
        const int qd = warp & 3;  // a warp reaches TMEM lanes 32 (warp % 4) .. + 31
        const int half = (warp - kSoftmax0) >> 2;
        const int row[2] = {qd * 32 + half * 16 + (lane >> 2), qd * 32 + half * 16 + (lane >> 2) + 8};
        const int tok[2] = {row[0] / P.group, row[1] / P.group};
        const uint32_t t_base = tmem + ((uint32_t)(qd * 32 + half * 16) << 16);
        const int c0 = 2 * (lane & 3);  // this thread's columns: c0 + 8 k, c0 + 8 k + 1
        const int warp_tok0 = (qd * 32 + half * 16) / P.group, warp_tok1 = (qd * 32 + half * 16 + 15) / P.group;
        const float sl2 = P.scale_log2;
        uint32_t gb0 = 0, segs = 0;  // key tiles, segments with a key so far
        bool ok = true;
        for (uint32_t k = 0;; ++k) {
            const Segment* sg = next_segment(k, ok);
            if (sg == nullptr) break;
            const int32_t n = sg->n, j0 = sg->j0, lo_t = sg->lo, ns = sg->ns;
            const bool dead[2] = {tok[0] >= sg->ntok, tok[1] >= sg->ntok};
            if (n == 0) {
                hand_back(k);
                continue;
            }
            // Row x sees keys lo[x] .. hi[x] - 1 and 0 .. sk[x] - 1.  Key tiles from
            // some_lo on and below some_hi, or below some_sk, are seen by some row of this
            // warp, from all_lo on and below all_hi, or below all_sk, whole by every row.
            int32_t hi[2], lo[2] = {0, 0}, sk[2] = {0, 0};
            int32_t some_hi, all_hi, some_lo = 0, all_lo = 0, some_sk = 0, all_sk = 0;
            {
                const int32_t kl = sg->kl, p0 = sg->pos0;
                // this warp's first and last token with a row
                const int32_t pa = p0 + warp_tok0, pb = p0 + min(warp_tok1, sg->ntok - 1);
                auto end = [&](int32_t p) -> int32_t { return P.causal ? min(kl, p + 1) : kl; };
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    hi[x] = end(p0 + tok[x]);
                    if constexpr (kMode == kWindow) {
                        lo[x] = p0 + tok[x] - P.window + 1;
                        sk[x] = min(P.sinks, hi[x]);
                    }
                }
                all_hi = max(end(pa), 0) >> 7;
                some_hi = warp_tok0 < sg->ntok ? (max(end(pb), 0) + 127) >> 7 : 0;
                if constexpr (kMode == kWindow) {
                    all_lo = (max(pb - P.window + 1, 0) + 127) >> 7;
                    some_lo = max(pa - P.window + 1, 0) >> 7;
                    all_sk = min(P.sinks, max(end(pa), 0)) >> 7;
                    some_sk = warp_tok0 < sg->ntok ? (min(P.sinks, max(end(pb), 0)) + 127) >> 7 : 0;
                }
            }
            const int32_t* list = kLists ? P.list + (int64_t)sg->list * P.cap + j0 : nullptr;
            const uint32_t* who = kLists ? P.list_who + ((int64_t)sg->list * P.cap + j0) * P.words : nullptr;
            float m[2] = {dead[0] ? 0.0f : -INFINITY, dead[1] ? 0.0f : -INFINITY};
            float l[2] = {0.0f, 0.0f};  // this thread's share of each row
            bool fresh = true;
            int32_t kt_next = 0;
            uint32_t who_next[2] = {0u, 0u};
            auto look = [&](int32_t j) {
                if constexpr (kLists) {
                    kt_next = list[j];
                    // (a row without a token may lie behind the last word)
                    who_next[0] = dead[0] ? 0u : who[(int64_t)j * P.words + (tok[0] >> 5)];
                    who_next[1] = dead[1] ? 0u : who[(int64_t)j * P.words + (tok[1] >> 5)];
                }
            };
            look(0);
            for (int32_t j = 0; j < n; ++j) {
                const uint32_t gb = gb0 + (uint32_t)j;
                const uint32_t sbuf = (gb % kSBuf) * 128u;
                int32_t kt;
                if constexpr (kLists) kt = kt_next;
                else if constexpr (kMode == kWindow) kt = j0 + j < ns ? j0 + j : lo_t + j0 + j - ns;
                else kt = j0 + j;
                const int32_t kb = kt * 128;
                // bit 2 kk + e of vis[x]: row x sees this thread's column c0 + 8 kk + e
                uint32_t vis[2] = {~0u, ~0u};
                bool masked, visible;
                if constexpr (kLists) {
                    bool part = false, any = false;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const bool listed = (who_next[x] >> (tok[x] & 31)) & 1u;
                        vis[x] = listed ? columns_below(hi[x] - kb - c0) : 0u;
                        part |= !dead[x] && vis[x] != ~0u;
                        any |= !dead[x] && vis[x] != 0u;
                    }
                    if (j + 1 < n) look(j + 1);
                    masked = __any_sync(0xffffffffu, part);
                    visible = __any_sync(0xffffffffu, any);
                } else {
                    visible = (kt < some_hi && kt >= some_lo) || kt < some_sk;
                    masked = visible && !((kt < all_hi && kt >= all_lo) || kt < all_sk);
                    if (masked) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            vis[x] = columns_below(hi[x] - kb - c0);
                            if constexpr (kMode == kWindow)
                                vis[x] = (vis[x] & ~columns_below(lo[x] - kb - c0)) | columns_below(sk[x] - kb - c0);
                        }
                    }
                }
                const uint32_t pk = place_k(gb);
                const bool wt = paged_wait(smem_u32(&sh->empty[pk % S]), (pk / S) & 1u, &sh->watch, status);
                // (a failure elsewhere in the block or in another one ends this wait too)
                if (__any_sync(0xffffffffu, !wt)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (!visible) {
                    // no row of this warp sees a key of the tile: P = 0
                    store_p_zero(t_base + sbuf);
                    tc_fence_before();
                    mbar_arrive(smem_u32(&sh->p_full[gb % kSBuf]));
                    continue;
                }
                uint32_t sc[64];
                auto load_s = [&]() {
                    tmem_ld16x256_x16(t_base + sbuf, sc);
                    tmem_wait_ld();
                    if (masked) {
                        const uint32_t ninf = __float_as_uint(-INFINITY);
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int kk = 0; kk < 16; ++kk)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    sc[4 * kk + 2 * x + e] = (vis[x] >> (2 * kk + e)) & 1u ? sc[4 * kk + 2 * x + e] : ninf;
                    }
                };
                load_s();
                float alpha[2];
                const bool rescale = softmax_rows(sc, dead, sl2, fresh, m, l, alpha, load_s);
                tmem_st16x128_x16(t_base + sbuf, sc);
                if (rescale) {
                    // O must hold P_0 .. P_{j-1} V: wait for PV_{j-1}
                    const uint32_t pv = place_v(gb - 1u);
                    const bool wv = paged_wait(smem_u32(&sh->empty[pv % S]), (pv / S) & 1u, &sh->watch, status);
                    if (__any_sync(0xffffffffu, !wv)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    scale_o_rows<D>(t_base + kColO, alpha[0], alpha[1]);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(smem_u32(&sh->p_full[gb % kSBuf]));
            }
            if (!ok) break;
            hand_back(k);
            // maxima and sums of the rows to the storing warps
            const float la = row_sum4(l[0]), lb = row_sum4(l[1]);
            if (__any_sync(0xffffffffu, !paged_wait(smem_u32(&sh->ml_empty), (segs & 1u) ^ 1u, &sh->watch, status))) {
                ok = false;
                break;
            }
            if ((lane & 3) == 0) {
                sh->ml[row[0]] = make_float2(m[0], la);
                sh->ml[row[1]] = make_float2(m[1], lb);
            }
            mbar_arrive(smem_u32(&sh->ml_full));
            ++segs;
            gb0 += (uint32_t)n;
        }
        if (!ok && lane == 0) set_abort(&sh->watch, status);
    } else {
        // ------------------------------------------------------------ O and LSE of a segment
        // one thread per row
        const int qd = warp & 3;  // a warp reaches TMEM lanes 32 (warp % 4) .. + 31
        const int row = qd * 32 + lane, tok = row / P.group, head = row % P.group;
        const uint32_t t_row = tmem + ((uint32_t)(qd * 32) << 16) + kColO;
        uint32_t g = 0, segs = 0;
        bool ok = true;
        for (uint32_t k = 0;; ++k) {
            const Segment* sp = next_segment(k, ok);
            if (sp == nullptr) break;
            const int32_t n = sp->n, slot = sp->slot;
            const bool dead = tok >= sp->ntok;
            const int64_t at = (int64_t)(sp->q0 + tok) * P.H + sp->kvh * P.group + head;
            __nv_bfloat16* orow = P.o + at * D;
            if (n == 0) {
                // no key at all: O = 0, LSE = -inf
                if (!dead) {
#pragma unroll
                    for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(orow + c) = make_uint4(0, 0, 0, 0);
                    P.lse[at] = -INFINITY;
                }
                hand_back(k);
                continue;
            }
            const uint32_t pv = place_v(g + (uint32_t)n - 1u);
            // (the last product is the segment's: the next one waits for o_free)
            ok = wait_warp(smem_u32(&sh->ml_full), segs & 1u, &sh->watch, status) &&
                 wait_warp(smem_u32(&sh->empty[pv % S]), (pv / S) & 1u, &sh->watch, status);
            if (!ok) break;
            const float2 ml = sh->ml[row];
            mbar_arrive(smem_u32(&sh->ml_empty));
            tc_fence_after();
            // 1 / l; 0 for a row without a key, NaN where l is
            const float inv = ml.y == 0.0f ? 0.0f : 1.0f / ml.y;
            const int64_t part = (int64_t)max(slot, 0) * 128 + row;
            bool finite = true;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                __syncwarp();  // the lanes without a row skip the stores below
                tmem_ld32(t_row + c, o);
                tmem_wait_ld();
                // (a sum that overflows says "not finite" too: the row is computed again for nothing)
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 32; ++i) sum += __uint_as_float(o[i]);
                finite &= sum - sum == 0.0f;
                if (dead) continue;
                if (slot < 0) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        pk[i] = pack_bf16(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        reinterpret_cast<uint4*>(orow + c)[i] = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        reinterpret_cast<uint4*>(P.part_o + part * D + c)[i] =
                            make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
            }
            tc_fence_before();
            mbar_arrive(smem_u32(&sh->o_free));
            if (!dead) {
                if (slot < 0) P.lse[at] = ml.y == 0.0f ? -INFINITY : (ml.x + log2f(ml.y)) * kLn2;
                else P.part_ml[part] = ml;
            }
            const uint32_t again = __ballot_sync(0xffffffffu, !finite && !dead);
            if (again != 0u) rows_again<D, kMode>(P, *sp, row, again, ml.x, inv, &sh->watch.busy);
            hand_back(k);
            g += (uint32_t)n;
            ++segs;
        }
        if (!ok && lane == 0) set_abort(&sh->watch, status);
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaQK) tmem_dealloc(tmem, kTmemCols);
}

// Joins the parts of split rows: O = sum_c 2^(m_c - M) O_c / l with M the
// largest m_c and l = sum_c 2^(m_c - M) l_c, parts in key order.  Thread block
// (c, y) takes kJoinThreads / (D / 4) rows of the query tile that begins in each of
// k_paged_forward's block c's runs: the run's slot 1, then slot 0 of the runs after it.
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) k_paged_join(const __grid_constant__ Params P) {
    launch_dependents();
    wait_primary();
    constexpr int kLanes = D / 4;                       // threads of a row, four columns each
    constexpr int kRows = kJoinThreads / kLanes;
    const int c = threadIdx.x % kLanes;
    const int32_t r = blockIdx.y * kRows + threadIdx.x / kLanes;
    for (int32_t p = 0; p < kPhases; ++p) {
        const int32_t run = p * gridDim.x + blockIdx.x;
        const int4 jn = P.joins[run];
        const int32_t rows = jn.z * P.group;
        if (jn.x == 0 || (int32_t)(blockIdx.y * kRows) >= rows) continue;
        const bool live = r < rows;  // (the others' threads take part in the shuffles)
        auto part = [&](int32_t x) -> int64_t {
            return (((int64_t)run + x) * 2 + (x == 0 ? 1 : 0)) * 128 + (live ? r : 0);
        };
        float M = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
        // kLanes parts at a time, each thread the maximum and sum of one: all loads at once
        for (int32_t x0 = 0; x0 < jn.x; x0 += kLanes) {
            const int32_t n = min(jn.x - x0, kLanes);
            const float2 ml = c < n ? P.part_ml[part(x0 + c)] : make_float2(-INFINITY, 0.0f);
            const bool none = ml.x == -INFINITY && ml.y == 0.0f;  // no visible key in this part
            float top = ml.x;
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float M_new = fmaxf(M, top);
            const float keep = M == -INFINITY ? 1.0f : exp2f(M - M_new);  // (l and o are 0 still)
            M = M_new;
            const float f = none ? 0.0f : exp2f(ml.x - M);
            float sum = none ? 0.0f : f * ml.y;
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            l = fmaf(l, keep, sum);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] *= keep;
#pragma unroll 8
            for (int32_t x = 0; x < n; ++x) {
                const float fx = __shfl_sync(0xffffffffu, f, x, kLanes);
                const bool skip = __shfl_sync(0xffffffffu, (int)none, x, kLanes) != 0;
                const float4 v = *reinterpret_cast<const float4*>(P.part_o + part(x0 + x) * D + 4 * c);
                o[0] = skip ? o[0] : fmaf(fx, v.x, o[0]);
                o[1] = skip ? o[1] : fmaf(fx, v.y, o[1]);
                o[2] = skip ? o[2] : fmaf(fx, v.z, o[2]);
                o[3] = skip ? o[3] : fmaf(fx, v.w, o[3]);
            }
        }
        if (!live) continue;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int64_t at = (int64_t)(jn.y + r / P.group) * P.H + jn.w * P.group + r % P.group;
        *reinterpret_cast<uint2*>(P.o + at * D + 4 * c) =
            make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
        if (c == 0) P.lse[at] = l == 0.0f ? -INFINITY : (M + log2f(l)) * kLn2;
    }
}

// Tile lists from the tokens' lists: for each (query tile, key/value head)
// the blocks that some token of the tile lists and sees, ascending, each with
// one bit per token.  One thread block per tile; the bits of up to kUnionWords
// / words blocks at a time are set in shared memory.
constexpr int kUnionThreads = 128;
constexpr int kUnionWords = 8192;
struct UnionParams {
    PagedBatch b;
    const int32_t *sel, *sel_cnt;  // [tokens, H_kv, width], [tokens, H_kv]
    int32_t width, H_kv, tpt, causal;
    int32_t *list, *cnt;
    uint32_t* who;
    int32_t nt_cap, cap, words;
    int32_t group, least, most;    // only the sequences with least .. most rows (tokens * group)
};
__global__ void __launch_bounds__(kUnionThreads) k_paged_union(const __grid_constant__ UnionParams P) {
    __shared__ uint32_t bits[kUnionWords];
    __shared__ int64_t part[33];
    __shared__ int32_t hit[5];
    launch_dependents();
    wait_primary();
    int32_t t;
    PagedSeq q;
    const int32_t s = find_unit<kUnionThreads>(
        P.b, blockIdx.x,
        [&](const PagedSeq& y) -> int64_t {
            const int32_t rows = y.nq * P.group;
            return rows < P.least || rows > P.most ? 0 : (y.nq + P.tpt - 1) / P.tpt;
        },
        part, hit, t, q);
    if (s < 0) return;
    const int32_t first = t * P.tpt, ntok = min(P.tpt, q.nq - first);
    const int32_t kvh = blockIdx.y;
    const int32_t nkb = (q.kl + 127) / 128;  // blocks of the sequence
    const int64_t f = (int64_t)kvh * P.nt_cap + blockIdx.x;
    const int32_t span = kUnionWords / P.words;
    int32_t done = 0;
    for (int32_t b0 = 0; b0 < nkb; b0 += span) {
        const int32_t nb = min(span, nkb - b0);
        for (int32_t x = threadIdx.x; x < nb * P.words; x += kUnionThreads) bits[x] = 0u;
        __syncthreads();
        for (int32_t x = threadIdx.x; x < ntok * P.width; x += kUnionThreads) {
            const int32_t tt = x / P.width, e = x % P.width;
            const int64_t tk = ((int64_t)(q.q0 + first + tt)) * P.H_kv + kvh;
            const int32_t n = P.sel_cnt[tk];
            if (e == 0 && b0 == 0 && (n < 0 || n > P.width))
                atomicCAS(P.b.status, 0, n < 0 ? BSA_ERR_BOUNDS : BSA_ERR_OVERFLOW);
            if (e >= n) continue;
            const int32_t blk = P.sel[tk * P.width + e];
            if (blk < 0 || blk >= nkb) {
                if (b0 == 0) atomicCAS(P.b.status, 0, BSA_ERR_BOUNDS);
                continue;
            }
            const int32_t pos = q.kl - q.nq + first + tt;
            if (blk < b0 || blk >= b0 + nb || (P.causal && blk * 128 > pos)) continue;
            atomicOr(&bits[(blk - b0) * P.words + (tt >> 5)], 1u << (tt & 31));
        }
        __syncthreads();
        for (int32_t x0 = 0; x0 < nb; x0 += kUnionThreads) {
            const int32_t x = x0 + threadIdx.x;
            uint32_t any = 0u;
            if (x < nb)
                for (int32_t w = 0; w < P.words; ++w) any |= bits[x * P.words + w];
            int64_t total;
            const int32_t at = done + (int32_t)block_prefix<kUnionThreads>(any != 0u ? 1 : 0, part, total);
            if (any != 0u && at < P.cap) {
                P.list[f * P.cap + at] = b0 + x;
                for (int32_t w = 0; w < P.words; ++w) P.who[(f * P.cap + at) * P.words + w] = bits[x * P.words + w];
            }
            done += (int32_t)total;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) P.cnt[f] = min(done, P.cap);
}

// ---------------------------------------------------------------- host side
bool encode(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
    auto enc = get_encode();
    if (!enc) return false;
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box,
               ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Workspace: joins, maxima and sums, O parts; then the tile lists.
struct Layout {
    size_t joins, ml, o, cnt, list, who, total;
    int32_t nt_cap, cap, words, tpt;
};
Layout layout(const PagedForwardArgs& a) {
    Layout L{};
    const int32_t G = a.H / a.H_kv;
    L.tpt = 128 / G;
    // sum over sequences of ceil(n / tpt) <= tokens / tpt + seqs
    L.nt_cap = a.tokens / L.tpt + a.seqs;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t p = at;
        at += (bytes + 255) & ~(size_t)255;
        return p;
    };
    L.joins = take(sizeof(int4) * kPagedRuns);
    L.ml = take(sizeof(float2) * kPagedRuns * 2 * 128);
    L.o = take(sizeof(float) * kPagedRuns * 2 * 128 * (size_t)a.D);
    if (a.sel_width > 0) {
        const int64_t blocks = ((int64_t)a.max_pages * a.page + 127) / 128;
        const int64_t most = (int64_t)L.tpt * a.sel_width;
        L.cap = (int32_t)(blocks < most ? blocks : most);
        L.words = (L.tpt + 31) / 32;
        const size_t rows = (size_t)a.H_kv * L.nt_cap;
        L.cnt = take(sizeof(int32_t) * rows);
        L.list = take(sizeof(int32_t) * rows * L.cap);
        L.who = take(sizeof(uint32_t) * rows * L.cap * L.words);
    }
    L.total = at;
    return L;
}

template <int D, int kMode>
bsa_status launch_d(const Params& P, cudaStream_t stream) {
    constexpr size_t smem = 1024 + Cfg<D>::kData + sizeof(Shared);
    static_assert(smem <= 232448, "shared memory of a thread block");
    static DeviceSetup setup;
    static int sms[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return BSA_ERR_CUDA;
    const bool ready = setup.once(dev, [&] {
        return cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
               cudaFuncSetAttribute(k_paged_forward<D, kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) ==
                   cudaSuccess;
    });
    if (!ready) return BSA_ERR_CUDA;
    const int grid = sms[dev] < kPagedBlocks ? sms[dev] : kPagedBlocks;
    if (launch_chained(k_paged_forward<D, kMode>, dim3((unsigned)grid), kThreads, smem, stream, P) != cudaSuccess ||
        launch_chained(k_paged_join<D>, dim3((unsigned)grid, 128 / (kJoinThreads / (D / 4))), kJoinThreads, 0, stream, P) != cudaSuccess)
        return BSA_ERR_CUDA;
    return BSA_OK;
}

}  // namespace

size_t paged_forward_workspace(const PagedForwardArgs& a) { return layout(a).total; }

bsa_status launch_paged_union(const PagedForwardArgs& a, int32_t tpt, int32_t nt_cap, int32_t cap, int32_t words, int32_t* list,
                              int32_t* cnt, uint32_t* who, int32_t* status, cudaStream_t stream, int32_t least, int32_t most) {
    const PagedBatch b{a.q_start, a.kv_len, a.table, a.seqs, a.tokens, a.max_pages, a.page, a.n_pages, status};
    UnionParams U{b, a.sel, a.sel_cnt, a.sel_width, a.H_kv, tpt, a.causal, list, cnt, who, nt_cap, cap, words, a.H / a.H_kv, least, most};
    return launch_chained(k_paged_union, dim3((unsigned)nt_cap, (unsigned)a.H_kv), kUnionThreads, 0, stream, U) == cudaSuccess
               ? BSA_OK
               : BSA_ERR_CUDA;
}

bsa_status launch_paged_forward(const PagedForwardArgs& a, void* workspace, int32_t* status, cudaStream_t stream) {
    const Layout L = layout(a);
    Params P;
    memset(&P, 0, sizeof(P));
    const int32_t G = a.H / a.H_kv, D = a.D;
    {
        const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.H, (cuuint64_t)a.tokens};
        const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.q_stride * 2};
        const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)L.tpt}, box1[3] = {64, (cuuint32_t)G, 1};
        if (!encode(&P.map_q, a.q, 3, dims, strides, box) || !encode(&P.map_q1, a.q, 3, dims, strides, box1))
            return BSA_ERR_CUDA;
    }
    {
        const cuuint64_t slots = (cuuint64_t)a.n_pages * a.H_kv * a.page;
        const cuuint64_t dims[3] = {64, slots, (cuuint64_t)(D / 64)};
        const cuuint64_t strides[2] = {(cuuint64_t)D * 2, 128};
        const cuuint32_t box[3] = {64, (cuuint32_t)a.page, (cuuint32_t)(a.page == 128 ? D / 64 : 1)};
        if (!encode(&P.map_k, a.k_cache, 3, dims, strides, box) || !encode(&P.map_v, a.v_cache, 3, dims, strides, box))
            return BSA_ERR_CUDA;
    }
    P.b = PagedBatch{a.q_start, a.kv_len, a.table, a.seqs, a.tokens, a.max_pages, a.page, a.n_pages, status};
    P.H = a.H;
    P.H_kv = a.H_kv;
    P.group = G;
    P.tpt = L.tpt;
    P.causal = a.causal;
    P.window = min(a.window, kMaxWindow);
    P.sinks = a.sinks;
    P.scale_log2 = (a.scale > 0.f ? a.scale : 1.0f / sqrtf((float)D)) * kLog2e;
    P.q = static_cast<const __nv_bfloat16*>(a.q);
    P.q_stride = a.q_stride;
    P.k_cache = static_cast<const __nv_bfloat16*>(a.k_cache);
    P.v_cache = static_cast<const __nv_bfloat16*>(a.v_cache);
    P.o = static_cast<__nv_bfloat16*>(a.o);
    P.lse = a.lse;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    P.nt_cap = L.nt_cap;
    P.joins = reinterpret_cast<int4*>(ws + L.joins);
    P.part_ml = reinterpret_cast<float2*>(ws + L.ml);
    P.part_o = reinterpret_cast<float*>(ws + L.o);
    if (a.sel != nullptr) {
        P.cap = L.cap;
        P.words = L.words;
        int32_t* cnt = reinterpret_cast<int32_t*>(ws + L.cnt);
        int32_t* list = reinterpret_cast<int32_t*>(ws + L.list);
        uint32_t* who = reinterpret_cast<uint32_t*>(ws + L.who);
        P.list_cnt = cnt;
        P.list = list;
        P.list_who = who;
        const bsa_status u = launch_paged_union(a, L.tpt, L.nt_cap, L.cap, L.words, list, cnt, who, status, stream);
        if (u != BSA_OK) return u;
        return D == 128 ? launch_d<128, kListed>(P, stream) : launch_d<64, kListed>(P, stream);
    }
    if (a.window > 0) return D == 128 ? launch_d<128, kWindow>(P, stream) : launch_d<64, kWindow>(P, stream);
    return D == 128 ? launch_d<128, kPlain>(P, stream) : launch_d<64, kPlain>(P, stream);
}

}  // namespace bsa
