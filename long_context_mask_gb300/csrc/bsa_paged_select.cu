// Block selection over a paged key/value cache: for each new token and
// key/value head the blocks with the highest
//     score_j = sum over the head's query heads of  q . (mean key of block j).
//
// Sure of its choice.  The scores that are compared are those of the bf16
// inputs in exact arithmetic (64 bits stand for it).  fp32 sums decide all but
// the close calls: with a the vector of sums of |q| over the query heads, an
// fp32 score is off by at most
//     E = (n + G + 2) 2^-24 |a| max_j |mean_j|
// (n roundings on a product's way into the sum, kSteps of them; G - 1 of the
// query heads' sum; by the Cauchy-Schwarz inequality; and what underflows), so with tau the k-th largest fp32 score every
// block above tau + 2E is among the k best and none below tau - 2E is.  Blocks
// in between are scored again in fp64 where there are more of them than places.
//
// Measured, 32 + 8 heads of 128, 16 of up to 512 blocks: 16 tokens 21 us (both kernels
// wait for their loads: 12 MB, 128 rows), 1024 tokens 62 us (39 the scores, 1.1 GFLOP in
// packed fp32: tensor cores would not give sums with a bound on their rounding; tiles of
// 128 blocks, two to an SM instead of three, take 41).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "bsa_device_setup.h"
#include "bsa_internal.h"
#include "bsa_paged.cuh"
#include "bsa_rows.cuh"

namespace bsa {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kTileTok = 64, kTileBlk = 64;  // tokens and blocks of a score tile
constexpr int kFewTok = 4;                    // tokens up to which a tile is read as a decoding step
// Most roundings on a product's way into a score: its own and the additions of
// the 64-long chain (D / 2 values, every second) of the product tile, the last
// addition; a decoding step's path (8 in a thread, then D / 8 threads) has fewer.
constexpr int kSteps = 128 / 2 + 1;
// What a sum of at most 128 squares loses where they underflow: each of its fused
// additions rounds to a multiple of 2^-149, off by half of it at most.  (Means around
// 2^-80 have squares below all fp32 numbers, and products with q that are far above.)
constexpr float kLost = 0x1p-143f;

struct SelectParams {
    PagedBatch b;
    const __nv_bfloat16* q;
    int64_t q_stride;
    const __nv_bfloat16* k_mean;
    int32_t H_kv, group, topk, sink, local, width;
    int32_t *sel, *sel_cnt;
    int32_t nb_cap;   // blocks of the longest sequence that the table can hold
    int32_t chunks;   // ceil(nb_cap / kTileBlk)
    float* scores;    // [tokens, H_kv, nb_cap]
    int32_t pick_bytes;  // shared memory of a warp of k_paged_pick
    float* norms;     // [tokens, H_kv, chunks] largest |mean|^2 of the chunk, in the row of a tile's first token
};

// Blocks c0 .. c1 - 1 are ranked for the token at position pos.
__device__ __forceinline__ void ranked(const SelectParams& P, int32_t pos, int32_t& c0, int32_t& c1) {
    c0 = P.sink;
    c1 = pos >= 0 ? max(pos / kBlock - P.local + 1, c0) : c0;
}

// fp32 (fp64) scores as unsigned keys of the same order; NaN is the lowest.
__device__ __forceinline__ uint32_t key_of(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 counts as 0
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t key_of(double x) {
    if (x != x) return 0ull;
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

// Between lo < hi, above lo: halfway in value (the keys of floats crowd around
// zero, where no k-th best lies: bisecting the keys took twice the steps).
__device__ __forceinline__ uint32_t halfway(uint32_t lo, uint32_t hi, int step) {
    const uint32_t mid = hi - (hi - lo) / 2;
    if (step >= 24) return mid;  // (what is left is a matter of few keys)
    const uint32_t v = key_of(0.5f * of_key(lo) + 0.5f * of_key(hi));
    return v > lo && v <= hi ? v : mid;
}
__device__ __forceinline__ uint64_t halfway(uint64_t lo, uint64_t hi, int) { return hi - (hi - lo) / 2; }

__device__ __forceinline__ uint32_t warp_max(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }
__device__ __forceinline__ uint32_t warp_min(uint32_t x) { return __reduce_min_sync(0xffffffffu, x); }
__device__ __forceinline__ uint64_t warp_max(uint64_t x) {
    for (int d = 1; d < 32; d <<= 1) {
        const uint64_t y = __shfl_xor_sync(0xffffffffu, x, d);
        x = y > x ? y : x;
    }
    return x;
}
__device__ __forceinline__ uint64_t warp_min(uint64_t x) { return ~warp_max(~x); }

// The k-th largest (1 <= k <= n) of the warp's n keys, by bisection between the
// smallest and the largest; it stops early at a bound that exactly k keys reach.
// kHeld > 0: lane l's keys are held[i] = key number l + 32 i (0 behind the last);
// else they are keys[0 .. n - 1].
template <int kHeld, typename Key>
__device__ __forceinline__ Key kth_largest(const Key (&held)[kHeld > 0 ? kHeld : 1], const Key* keys, int32_t n, int32_t k) {
    const int lane = threadIdx.x & 31;
    auto each = [&](auto&& f) {
        if constexpr (kHeld > 0) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) f(held[i], lane + 32 * i < n);
        } else {
#pragma unroll 4
            for (int32_t x = lane; x < n; x += 32) f(keys[x], true);
        }
    };
    auto least = [&](Key bound) -> Key {  // of the keys >= bound
        Key v = ~(Key)0;
        each([&](Key x, bool in) { v = in && x >= bound && x < v ? x : v; });
        return warp_min(v);
    };
    Key mine = 0;  // this lane's largest
    each([&](Key x, bool in) { mine = in && x > mine ? x : mine; });
    Key hi = warp_max(mine), lo;
    if (k <= 32 && n >= 32) {
        // the k-th largest of the lanes' largest is a good first bound, and cheap to find
        lo = warp_min(mine);
        Key top = hi;
        for (int step = 0; lo < top; ++step) {
            const Key mid = halfway(lo, top, step);
            const int32_t c = __popc(__ballot_sync(0xffffffffu, mine >= mid));
            if (c >= k) lo = mid;
            else top = mid - 1;
            if (c == k) break;
        }
    } else {
        lo = least(0);
    }
    // at least k keys reach lo, fewer than k exceed hi
    for (int step = 0; lo < hi; ++step) {
        const Key mid = halfway(lo, hi, step);
        int32_t c = 0;  // keys >= mid (> 0: none is behind the last)
        each([&](Key x, bool) { c += x >= mid; });
        c = __reduce_add_sync(0xffffffffu, c);
        if (c == k) return least(mid);
        if (c > k) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float larger(float a, float b) { return (a > b || a != a) ? a : b; }  // NaN wins

// Scores of one (token tile, chunk of blocks, key/value head).
template <int D>
__global__ void __launch_bounds__(kScoreThreads) k_paged_scores(const __grid_constant__ SelectParams P) {
    extern __shared__ __align__(16) float tile[];  // sums of the query heads [tokens][D + 4], means [blocks][D + 4]
    constexpr int kRow = D + 4;                    // (rows 4 banks apart: 16-byte reads down a column meet no conflict)
    __shared__ int64_t part[33];
    __shared__ int32_t hit[5];
    __shared__ int32_t ids[kTileBlk];
    __shared__ float most[kScoreThreads / 32];
    ptx::launch_dependents();
    ptx::wait_primary();
    int32_t t;
    PagedSeq y;
    const int32_t s = find_unit<kScoreThreads>(
        P.b, blockIdx.x, [](const PagedSeq& q) -> int64_t { return (q.nq + kTileTok - 1) / kTileTok; }, part, hit, t, y);
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
        for (int32_t x = threadIdx.x; x < P.b.seqs; x += kScoreThreads) {
            PagedSeq y;
            if (!paged_seq(P.b, x, y)) atomicCAS(P.b.status, 0, BSA_ERR_BOUNDS);
        }
    if (s < 0) return;
    const int32_t first = t * kTileTok, ntok = min(kTileTok, y.nq - first);
    const int32_t kvh = blockIdx.z, b0 = blockIdx.y * kTileBlk;
    int32_t c0, c1;  // of the last token, which ranks the most
    ranked(P, y.kl - y.nq + first + ntok - 1, c0, c1);
    const int32_t tok0 = y.q0 + first;
    if (c1 - c0 <= P.topk || P.topk == 0 || b0 >= c1 || b0 + kTileBlk <= c0) return;
    const int32_t lo = max(b0, c0), nb = min(b0 + kTileBlk, c1) - lo;
    const int32_t per = kBlock / P.b.page;
    for (int32_t x = threadIdx.x; x < nb; x += kScoreThreads) {
        // mean key of a block: at the page of its last token
        int32_t id = P.b.table[(int64_t)s * P.b.max_pages + (int64_t)(lo + x + 1) * per - 1];
        if (id < 0 || id >= P.b.n_pages) {
            atomicCAS(P.b.status, 0, BSA_ERR_BOUNDS);
            id = 0;
        }
        ids[x] = id;
    }
    const __nv_bfloat16* q0 = P.q + (int64_t)tok0 * P.q_stride + (int64_t)kvh * P.group * D;
    float* out = P.scores + ((int64_t)tok0 * P.H_kv + kvh) * P.nb_cap + lo;  // of the tile's first token
    const int64_t out_row = (int64_t)P.H_kv * P.nb_cap;
    constexpr int kLanes = D / 8, kRows = kScoreThreads / kLanes;
    const int c = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
    // sum of a token's query heads, this thread's values 8 c .. 8 c + 7
    auto head_sum = [&](int32_t tk, float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.f;
#pragma unroll 4
        for (int g = 0; g < P.group; ++g) {
            const uint4 v = *reinterpret_cast<const uint4*>(q0 + (int64_t)tk * P.q_stride + g * D + 8 * c);
            const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 w = __bfloat1622float2(h[i]);
                f[2 * i] += w.x;
                f[2 * i + 1] += w.y;
            }
        }
    };
    float big = 0.f;
    if (ntok <= kFewTok) {
        float q[kFewTok][8];
#pragma unroll
        for (int k = 0; k < kFewTok; ++k)
            if (k < ntok) head_sum(k, q[k]);
        __syncthreads();
        constexpr int kDeep = 4;  // means in flight for each thread
        for (int32_t x0 = 0; x0 < nb; x0 += kRows * kDeep) {
            uint4 v[kDeep];
#pragma unroll
            for (int u = 0; u < kDeep; ++u) {
                const int32_t x = x0 + u * kRows + sub;
                v[u] = x < nb ? *reinterpret_cast<const uint4*>(P.k_mean + ((int64_t)ids[x] * P.H_kv + kvh) * D + 8 * c)
                              : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < kDeep; ++u) {
                const int32_t x = x0 + u * kRows + sub;
                const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v[u]);
                float m[8], sq = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 w = __bfloat1622float2(h[i]);
                    m[2 * i] = w.x;
                    m[2 * i + 1] = w.y;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) sq = fmaf(m[i], m[i], sq);
#pragma unroll
                for (int d = 1; d < kLanes; d <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, d);
                big = larger(sq, big);
#pragma unroll
                for (int k = 0; k < kFewTok; ++k) {
                    if (k >= ntok) break;
                    float dot = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) dot = fmaf(q[k][i], m[i], dot);
#pragma unroll
                    for (int d = 1; d < kLanes; d <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
                    if (c == 0 && x < nb) out[k * out_row + x] = dot;
                }
            }
        }
    } else {
        float* qs = tile;
        float* ms = tile + kTileTok * kRow;
        __syncthreads();
        constexpr int kDeep = kTileBlk / kRows < 4 ? kTileBlk / kRows : 4;  // loads in flight for each thread
        for (int32_t x0 = 0; x0 < kTileBlk; x0 += kRows * kDeep) {
            uint4 v[kDeep];
#pragma unroll
            for (int u = 0; u < kDeep; ++u) {
                const int32_t x = x0 + u * kRows + sub;
                v[u] = x < nb ? *reinterpret_cast<const uint4*>(P.k_mean + ((int64_t)ids[x] * P.H_kv + kvh) * D + 8 * c)
                              : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < kDeep; ++u) {
                const int32_t x = x0 + u * kRows + sub;
                const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v[u]);
                float m[8], sq = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 w = __bfloat1622float2(h[i]);
                    m[2 * i] = w.x;
                    m[2 * i + 1] = w.y;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) sq = fmaf(m[i], m[i], sq);
#pragma unroll
                for (int d = 1; d < kLanes; d <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, d);
                big = larger(sq, big);
                *reinterpret_cast<float4*>(ms + x * kRow + 8 * c) = make_float4(m[0], m[1], m[2], m[3]);
                *reinterpret_cast<float4*>(ms + x * kRow + 8 * c + 4) = make_float4(m[4], m[5], m[6], m[7]);
            }
        }
#pragma unroll 2
        for (int32_t k = sub; k < kTileTok; k += kRows) {
            float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (k < ntok) head_sum(k, f);
            *reinterpret_cast<float4*>(qs + k * kRow + 8 * c) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4*>(qs + k * kRow + 8 * c + 4) = make_float4(f[4], f[5], f[6], f[7]);
        }
        __syncthreads();
        // thread (ty, tx): tokens 4 ty .. 4 ty + 3, blocks tx + 16 j (j < kCols); even and
        // odd values of d add up apart
        const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
        constexpr int kCols = kTileBlk / 16;
        if (4 * ty < ntok) {
            uint64_t acc[4][kCols];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < kCols; ++j) acc[i][j] = 0ull;
#pragma unroll 1
            for (int d = 0; d < D; d += 4) {
                ulonglong2 m[kCols];
#pragma unroll
                for (int j = 0; j < kCols; ++j) m[j] = *reinterpret_cast<const ulonglong2*>(ms + (tx + 16 * j) * kRow + d);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(qs + (4 * ty + i) * kRow + d);
#pragma unroll
                    for (int j = 0; j < kCols; ++j) acc[i][j] = fma2(q.y, m[j].y, fma2(q.x, m[j].x, acc[i][j]));
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int32_t k = 4 * ty + i;
                if (k >= ntok) break;
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    const int32_t x = tx + 16 * j;
                    float a, b;
                    f2unpack(acc[i][j], a, b);
                    if (x < nb) out[k * out_row + x] = a + b;
                }
            }
        }
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) big = larger(__shfl_xor_sync(0xffffffffu, big, d), big);
    if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = big;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < kScoreThreads / 32; ++w) big = larger(most[w], big);
        P.norms[((int64_t)tok0 * P.H_kv + kvh) * P.chunks + blockIdx.y] = big;
    }
}

constexpr int kHeld = 16;  // up to 512 scores of a row stay in registers (16 to a lane)

// One warp per (token, key/value head).
template <int D>
__global__ void __launch_bounds__(128) k_paged_pick(const __grid_constant__ SelectParams P) {
    extern __shared__ __align__(16) uint8_t dyn[];
    const int lane = threadIdx.x & 31;
    const int32_t warp = threadIdx.x >> 5;
    // the warp's own: fp64 keys of close calls, keys (of rows too long for registers),
    // chosen blocks, places of close calls
    uint64_t* key64 = reinterpret_cast<uint64_t*>(dyn + (size_t)warp * P.pick_bytes);
    uint32_t* keys = reinterpret_cast<uint32_t*>(key64 + P.nb_cap);
    uint32_t* chosen = keys + (P.nb_cap > 32 * kHeld ? P.nb_cap : 0);
    uint16_t* close = reinterpret_cast<uint16_t*>(chosen + P.nb_cap / 32 + 1);
    ptx::launch_dependents();
    ptx::wait_primary();
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
    if (row >= (int64_t)P.b.tokens * P.H_kv) return;
    const int32_t tok = (int32_t)(row / P.H_kv), kvh = (int32_t)(row - (int64_t)tok * P.H_kv);
    // the last sequence that starts at or before the token, 32 probes at a time
    int32_t s = 0;
    for (int32_t n = P.b.seqs; n > 1;) {  // it is among s .. s + n - 1, or there is none
        const int32_t step = (n + 31) / 32;
        const int32_t x = s + lane * step;
        const uint32_t m = __ballot_sync(0xffffffffu, lane * step < n && P.b.q_start[x] <= tok);
        if (m == 0u) return;
        const int32_t last = 31 - __clz(m);
        s += last * step;
        n = min(step, n - last * step);
    }
    PagedSeq y;
    if (!paged_seq(P.b, s, y) || tok < y.q0 || tok >= y.q0 + y.nq) return;  // of no sequence: left as it was
    const int32_t pos = y.kl - y.nq + (tok - y.q0);
    int32_t* sel = P.sel + row * P.width;
    const int32_t own = pos >= 0 ? pos / kBlock : -1;  // the token's own block
    int32_t c0, c1;                                    // blocks c0 .. c1 - 1 are ranked
    ranked(P, pos, c0, c1);
    const int32_t nc = c1 - c0;
    const int32_t words = (own + 32) / 32;
    // blocks 0 .. own, all of them chosen unless they are ranked
    for (int32_t w = lane; w < words; w += 32) {
        auto below = [&](int32_t v) -> uint32_t {  // bits of blocks < v
            const int32_t n = v - 32 * w;
            return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u);
        };
        chosen[w] = nc <= P.topk ? below(own + 1) : below(min(c0, own + 1)) | (below(own + 1) & ~below(c1));
    }
    if (nc > P.topk && P.topk > 0) {
        const __nv_bfloat16* qrow = P.q + (int64_t)tok * P.q_stride + (int64_t)kvh * P.group * D;
        constexpr int kPer = D / 32;  // values of a lane
        // |a|^2 with a the sums of |q| over the query heads
        float a[kPer], norm_a = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) a[i] = 0.f;
#pragma unroll 4
        for (int g = 0; g < P.group; ++g)
#pragma unroll
            for (int i = 0; i < kPer; i += 2) {
                const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(qrow + g * D + lane * kPer + i));
                a[i] += fabsf(f.x);
                a[i + 1] += fabsf(f.y);
            }
        // the largest |mean|^2 of the chunks that hold a ranked block
        const int32_t tile_tok = y.q0 + (tok - y.q0) / kTileTok * kTileTok;
        const float* norms = P.norms + ((int64_t)tile_tok * P.H_kv + kvh) * P.chunks;
        float most = 0.f;
        for (int32_t x = c0 / kTileBlk + lane; x <= (c1 - 1) / kTileBlk; x += 32) most = larger(norms[x], most);
        const float* scores = P.scores + row * P.nb_cap + c0;
        uint32_t held[kHeld];
        const bool in_regs = nc <= 32 * kHeld;
        if (in_regs) {
            // (all loads first: 16 of them, each under a condition, waited one for another)
            float sc[kHeld];
#pragma unroll
            for (int i = 0; i < kHeld; ++i) sc[i] = scores[min(lane + 32 * i, nc - 1)];
#pragma unroll
            for (int i = 0; i < kHeld; ++i) held[i] = lane + 32 * i < nc ? key_of(sc[i]) : 0u;
        } else {
#pragma unroll 8
            for (int32_t x = lane; x < nc; x += 32) keys[x] = key_of(scores[x]);
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) norm_a = fmaf(a[i], a[i], norm_a);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            norm_a += __shfl_xor_sync(0xffffffffu, norm_a, d);
            most = larger(__shfl_xor_sync(0xffffffffu, most, d), most);
        }
        __syncwarp();
        // (1.01 covers the rounding of E itself, 1e-36 products that underflow, kLost squares that do)
        const float E = 1.01f * (float)(kSteps + P.group + 2) * 5.9604645e-8f * sqrtf(norm_a + kLost) * sqrtf(most + kLost) + 1e-36f;
        const uint32_t none32[1] = {0u};
        const float tau = of_key(in_regs ? kth_largest<kHeld>(held, keys, nc, P.topk) : kth_largest<0>(none32, keys, nc, P.topk));
        // without a finite bound every block is a close call
        const bool bound = tau - tau == 0.0f && E - E == 0.0f;
        const uint32_t hi = bound ? key_of(tau + 2.0f * E) : 0xffffffffu;  // surely chosen: keys above
        const uint32_t lo = bound ? key_of(tau - 2.0f * E) : 0u;           // surely not: keys below
        // bits of places x0 .. x0 + 31 among the chosen blocks
        auto choose = [&](int32_t x0, uint32_t bits) {
            if (bits == 0u) return;
            const int32_t b0 = c0 + x0, sh = b0 & 31;
            atomicOr(&chosen[b0 >> 5], bits << sh);
            if (sh != 0 && (bits >> (32 - sh)) != 0u) atomicOr(&chosen[(b0 >> 5) + 1], bits >> (32 - sh));
        };
        // the blocks in between, in ascending order
        int32_t n_close = 0, n_sure = 0;
        for (int32_t base = 0; base < nc; base += 32 * kHeld) {
            // bit i of a lane's masks: its place base + 32 i + lane.  (The long part is in
            // loops of few instructions: laid out 16 times and run once it waited for
            // its instructions.)
            uint32_t sure = 0u, maybe = 0u;
            if (in_regs) {
#pragma unroll
                for (int i = 0; i < kHeld; ++i) {
                    sure |= held[i] > hi ? 1u << i : 0u;
                    maybe |= held[i] >= lo ? 1u << i : 0u;
                }
            } else {
                for (int i = 0; i < kHeld && base + 32 * i + lane < nc; ++i) {
                    const uint32_t k = keys[base + 32 * i + lane];
                    sure |= (uint32_t)(k > hi) << i;
                    maybe |= (uint32_t)(k >= lo) << i;
                }
            }
            // (places behind the last: their key 0 may reach lo = 0)
            const int32_t mine = nc - base - lane;
            const int32_t held_n = mine <= 0 ? 0 : min((mine + 31) / 32, kHeld);
            maybe &= ((1u << held_n) - 1u) & ~sure;
            // lane i < kHeld: the masks of places base + 32 i .. + 31
            uint32_t sure_w = 0u, maybe_w = 0u;
#pragma unroll 1
            for (int i = 0; i < kHeld; ++i) {
                const uint32_t a = __ballot_sync(0xffffffffu, (sure >> i) & 1u), b = __ballot_sync(0xffffffffu, (maybe >> i) & 1u);
                if (lane == i) {
                    sure_w = a;
                    maybe_w = b;
                }
            }
            choose(base + 32 * lane, sure_w);
            int32_t at = __popc(maybe_w);
#pragma unroll
            for (int d = 1; d < kHeld; d <<= 1) {
                const int32_t v = __shfl_up_sync(0xffffffffu, at, d);
                if (lane >= d) at += v;
            }
            const int32_t total = __shfl_sync(0xffffffffu, at, kHeld - 1);
            at += n_close - __popc(maybe_w);
            for (uint32_t bits = maybe_w; bits; bits &= bits - 1u) close[at++] = (uint16_t)(base + 32 * lane + __ffs(bits) - 1);
            n_close += total;
            n_sure += __reduce_add_sync(0xffffffffu, __popc(sure));
        }
        __syncwarp();
        const int32_t need = P.topk - n_sure;  // places left for the close calls
        uint64_t edge = 0;                     // (all of them fit)
        int32_t left = n_close;
        if (n_close > need) {
            const int32_t* table = P.b.table + (int64_t)s * P.b.max_pages;
            const int32_t per = kBlock / P.b.page;
            double q[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) q[i] = 0.0;
#pragma unroll 4
            for (int g = 0; g < P.group; ++g)
#pragma unroll
                for (int i = 0; i < kPer; ++i) q[i] += (double)__bfloat162float(qrow[g * D + lane * kPer + i]);
            for (int32_t x0 = 0; x0 < n_close; x0 += 32) {
                // (a bad page has been reported with the scores)
                int32_t id = x0 + lane < n_close ? table[(int64_t)(c0 + close[x0 + lane] + 1) * per - 1] : 0;
                id = id < 0 || id >= P.b.n_pages ? 0 : id;
#pragma unroll 4
                for (int32_t x = x0; x < min(x0 + 32, n_close); ++x) {
                    const __nv_bfloat16* m =
                        P.k_mean + ((int64_t)__shfl_sync(0xffffffffu, id, x - x0) * P.H_kv + kvh) * D + lane * kPer;
                    double dot = 0.0;
#pragma unroll
                    for (int i = 0; i < kPer; ++i) dot = fma(q[i], (double)__bfloat162float(m[i]), dot);
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
                    if (lane == 0) key64[x] = key_of(dot);
                }
            }
            __syncwarp();
            if (n_close <= 32) {
                // a lane for each: how many are better (equal scores: the lower blocks)
                const uint64_t mine = lane < n_close ? key64[lane] : 0ull;
                int32_t better = 0;
                for (int32_t x = 0; x < n_close; ++x) {
                    const uint64_t k = __shfl_sync(0xffffffffu, mine, x);
                    better += k > mine || (k == mine && x < lane);
                }
                if (lane < n_close && better < need) atomicOr(&chosen[(c0 + close[lane]) >> 5], 1u << ((c0 + close[lane]) & 31));
                n_close = 0;  // (all done)
            } else {
                const uint64_t none64[1] = {0ull};
                edge = kth_largest<0>(none64, key64, n_close, need);
                int32_t better = 0;
                for (int32_t x = lane; x < n_close; x += 32) better += key64[x] > edge;
                left = need - __reduce_add_sync(0xffffffffu, better);  // of the equal scores at the edge, the lowest blocks
            }
        }
        for (int32_t x0 = 0; x0 < n_close; x0 += 32) {
            const int32_t x = x0 + lane;
            const uint64_t k = x >= n_close ? 0ull : (n_close > need ? key64[x] : edge);
            const uint32_t tie = __ballot_sync(0xffffffffu, x < n_close && k == edge);
            if (x < n_close && (k > edge || (k == edge && __popc(tie & ((1u << lane) - 1u)) < left)))
                atomicOr(&chosen[(c0 + close[x]) >> 5], 1u << ((c0 + close[x]) & 31));
            left -= __popc(tie);
        }
    }
    __syncwarp();
    // the chosen blocks in ascending order, then -1
    int32_t n = 0;
    for (int32_t w0 = 0; w0 < words; w0 += 32) {
        uint32_t bits = w0 + lane < words ? chosen[w0 + lane] : 0u;
        int32_t at = __popc(bits);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, at, d);
            if (lane >= d) at += v;
        }
        const int32_t total = __shfl_sync(0xffffffffu, at, 31);
        at += n - __popc(bits);
        while (bits) {
            sel[at++] = 32 * (w0 + lane) + __ffs(bits) - 1;
            bits &= bits - 1u;
        }
        n += total;
    }
    for (int32_t x = n + lane; x < P.width; x += 32) sel[x] = -1;
    if (lane == 0) P.sel_cnt[row] = n;
}

}  // namespace

namespace {
struct Layout {
    int32_t nb_cap, chunks;
    size_t norms, scores, total;
};
Layout layout(const PagedSelectArgs& a) {
    Layout L{};
    L.nb_cap = (int32_t)(((int64_t)a.max_pages * a.page + kBlock - 1) / kBlock);
    L.chunks = (L.nb_cap + kTileBlk - 1) / kTileBlk;
    const size_t rows = (size_t)a.tokens * a.H_kv;
    L.norms = 0;
    L.scores = (rows * L.chunks * sizeof(float) + 255) & ~(size_t)255;
    L.total = L.scores + rows * L.nb_cap * sizeof(float);
    return L;
}

template <int D>
bsa_status launch_d(const SelectParams& P, cudaStream_t stream) {
    // warps to a thread block of k_paged_pick: four, or as many as its shared memory holds
    const int32_t most = 196608 / P.pick_bytes, warps = most < 4 ? most : 4;
    constexpr size_t tile = (size_t)(kTileTok + kTileBlk) * (D + 4) * sizeof(float);
    static DeviceSetup setup;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return BSA_ERR_CUDA;
    const bool ready = setup.once(dev, [&] {
        return cudaFuncSetAttribute(k_paged_scores<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)tile) == cudaSuccess &&
               cudaFuncSetAttribute(k_paged_pick<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, 196608) == cudaSuccess;
    });
    if (!ready) return BSA_ERR_CUDA;
    // sum over sequences of ceil(n / kTileTok) <= tokens / kTileTok + seqs
    const dim3 tiles((unsigned)(P.b.tokens / kTileTok + P.b.seqs), (unsigned)P.chunks, (unsigned)P.H_kv);
    if (launch_chained(k_paged_scores<D>, tiles, kScoreThreads, tile, stream, P) != cudaSuccess ||
        launch_chained(k_paged_pick<D>, dim3((unsigned)(((int64_t)P.b.tokens * P.H_kv + warps - 1) / warps)), 32 * warps,
                       (size_t)warps * P.pick_bytes, stream, P) != cudaSuccess)
        return BSA_ERR_CUDA;
    return BSA_OK;
}
}  // namespace

size_t paged_select_workspace(const PagedSelectArgs& a) { return layout(a).total; }

bsa_status launch_paged_select(const PagedSelectArgs& a, void* workspace, int32_t* status, cudaStream_t stream) {
    const Layout L = layout(a);
    SelectParams P{};
    P.b = PagedBatch{a.q_start, a.kv_len, a.table, a.seqs, a.tokens, a.max_pages, a.page, a.n_pages, status};
    P.q = static_cast<const __nv_bfloat16*>(a.q);
    P.q_stride = a.q_stride;
    P.k_mean = static_cast<const __nv_bfloat16*>(a.k_mean);
    P.H_kv = a.H_kv;
    P.group = a.H / a.H_kv;
    P.topk = a.topk;
    P.sink = a.sink_blocks;
    P.local = a.local_blocks;
    P.width = a.width;
    P.sel = a.sel;
    P.sel_cnt = a.sel_cnt;
    P.nb_cap = L.nb_cap;
    P.chunks = L.chunks;
    P.pick_bytes = (L.nb_cap * (8 + (L.nb_cap > 32 * kHeld ? 4 : 0) + 2) + (L.nb_cap / 32 + 1) * 4 + 15) & ~15;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    P.norms = reinterpret_cast<float*>(ws + L.norms);
    P.scores = reinterpret_cast<float*>(ws + L.scores);
    return a.D == 128 ? launch_d<128>(P, stream) : launch_d<64>(P, stream);
}

}  // namespace bsa
