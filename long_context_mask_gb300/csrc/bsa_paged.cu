// Appending new tokens to a paged key/value cache.
//
// For every new token and head:
//     y = x                                   (no norm)
//     y = x * w / sqrt(mean(x^2) + eps)       (q_norm / k_norm, over the head's D values)
//     (y_i, y_j) -> (y_i cos a - y_j sin a, y_j cos a + y_i sin a)
// with cos a, sin a of the token's position from the table, and the pairs
// (i, i + rot/2) or (2i, 2i + 1) of the first rot values.  Queries go to
// q_out, keys to their page slots, values (untouched) to theirs.  All of it is
// in fp32 with one rounding to bf16 at the end.  When a 128-token block of a
// sequence is full, the mean of its keys as the cache holds them (fp32 sum,
// one rounding to bf16: it is compared as a key is) goes to k_mean at the
// page of the block's last token.
//
// Work mapping.  A thread block takes one 128-position block that a sequence's
// new tokens touch and either four query heads of its tokens (long chunks: of a
// half or a quarter of them), or the key and the value of one key/value head, two tokens at a
// time.  The block that writes a head's keys writes all of this position block's, so the mean needs no other's work and adds in a
// fixed order, whatever chunks the tokens came in.  A row of D values is held by
// D / 8 neighbouring threads, eight values each: where the whole head turns by
// halves, four of either half (a pair meets in one thread), else eight in a row,
// with the rotation partner's values by shuffles.  Every thread loads its four
// rows before it works on the first.  (A prompt of 8192 tokens, 32 + 8 heads of
// 128 with norms, 206 MB: 43 us, 0.71 of the copy rate; 107 us with one row at a time,
// 62 us when each row found its place for itself, 234 instructions a row.  A step of 32
// tokens: 5.7 us, most of it the launch.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "bsa_internal.h"
#include "bsa_paged.cuh"

namespace bsa {
namespace {

constexpr int kAppendThreads = 128;

struct AppendParams {
    PagedBatch b;
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_stride, k_stride, v_stride, qo_stride;  // elements between tokens
    __nv_bfloat16* q_out;
    __nv_bfloat16 *k_cache, *v_cache, *k_mean;
    const float* rope;
    int32_t rope_len, rot, interleaved;
    const __nv_bfloat16 *q_norm, *k_norm;
    float eps;
    int32_t H_kv, group;
    int32_t q_blocks;  // thread blocks (y) of query heads; those of keys and values follow
    int32_t q_parts;   // of a position block's tokens that a thread block of query heads takes one of: 1, 2 or 4
    int32_t page_shift;
};

__device__ __forceinline__ void unpack8(const uint4& x, float (&f)[8]) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __bfloat1622float2(h[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint4 x;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&x);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    return x;
}

// A thread's eight values of a row (c: its place among the row's D / 8): 8 c ..
// 8 c + 7, or with kHalves 4 c .. 4 c + 3 of either half.
template <int D, bool kHalves>
__device__ __forceinline__ uint4 load_row(const __nv_bfloat16* row, int c) {
    if constexpr (!kHalves) return *reinterpret_cast<const uint4*>(row + 8 * c);
    const uint2 a = *reinterpret_cast<const uint2*>(row + 4 * c), b = *reinterpret_cast<const uint2*>(row + D / 2 + 4 * c);
    return make_uint4(a.x, a.y, b.x, b.y);
}
template <int D, bool kHalves>
__device__ __forceinline__ void store_row(__nv_bfloat16* row, int c, const uint4& x) {
    if constexpr (!kHalves) {
        *reinterpret_cast<uint4*>(row + 8 * c) = x;
    } else {
        *reinterpret_cast<uint2*>(row + 4 * c) = make_uint2(x.x, x.y);
        *reinterpret_cast<uint2*>(row + D / 2 + 4 * c) = make_uint2(x.z, x.w);
    }
}

// RMS norm of one row over its D values.  Every thread of the warp calls it.
template <int D>
__device__ __forceinline__ void norm_row(float (&x)[8], const float (&w)[8], float eps) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int d = 1; d < D / 8; d <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    const float r = rsqrtf(ss * (1.0f / D) + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
}

// The angles that this thread's values of a row turn by: with kHalves values i
// and 4 + i, interleaved values 2 i and 2 i + 1 by (co[i], si[i]), i < 4; else
// value i, with its partner half the rotated part away.
struct Angles {
    float co[8], si[8];
};
template <bool kHalves>
__device__ __forceinline__ void load_angles(const AppendParams& P, int c, int32_t pos, Angles& a) {
    const int half = P.rot >> 1;  // a multiple of 8
    const float* cs = P.rope + (int64_t)pos * P.rot;
    if (!kHalves && 8 * c >= P.rot) return;
    if (kHalves || P.interleaved) {
        *reinterpret_cast<float4*>(a.co) = *reinterpret_cast<const float4*>(cs + 4 * c);
        *reinterpret_cast<float4*>(a.si) = *reinterpret_cast<const float4*>(cs + half + 4 * c);
        return;
    }
    const int at = 8 * c < half ? 8 * c : 8 * c - half;
    *reinterpret_cast<float4*>(a.co) = *reinterpret_cast<const float4*>(cs + at);
    *reinterpret_cast<float4*>(a.co + 4) = *reinterpret_cast<const float4*>(cs + at + 4);
    *reinterpret_cast<float4*>(a.si) = *reinterpret_cast<const float4*>(cs + half + at);
    *reinterpret_cast<float4*>(a.si + 4) = *reinterpret_cast<const float4*>(cs + half + at + 4);
}

// Rotation of one row.  Every thread of the warp calls it.
template <bool kHalves>
__device__ __forceinline__ void rotate_row(const AppendParams& P, float (&x)[8], int c, const Angles& a) {
    if constexpr (kHalves) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float u = x[i], v = x[4 + i];
            x[i] = u * a.co[i] - v * a.si[i];
            x[4 + i] = v * a.co[i] + u * a.si[i];
        }
        return;
    }
    if (P.interleaved) {
        if (8 * c < P.rot) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = x[2 * i], v = x[2 * i + 1];
                x[2 * i] = u * a.co[i] - v * a.si[i];
                x[2 * i + 1] = v * a.co[i] + u * a.si[i];
            }
        }
        return;
    }
    // values 8 c .. pair with those of the thread rot / 16 places further (or nearer)
    const int step = P.rot >> 4;
    const bool first = c < step, turned = 8 * c < P.rot;
    const int from = (threadIdx.x & 31) + (turned ? (first ? step : -step) : 0);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], from);
    if (turned) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = first ? x[i] * a.co[i] - y[i] * a.si[i] : x[i] * a.co[i] + y[i] * a.si[i];
    }
}

template <int D, bool kHalves>
__global__ void __launch_bounds__(kAppendThreads) k_paged_append(const __grid_constant__ AppendParams P) {
    constexpr int kLanes = D / 8;
    constexpr int kRows = kAppendThreads / kLanes;  // rows in flight
    __shared__ int64_t part[33];
    __shared__ int32_t hit[5];
    __shared__ int32_t pages[8];  // the block's pages (128 / page of them)
    __shared__ float sums[kRows][D];
    ptx::launch_dependents();
    ptx::wait_primary();
    int32_t blk;
    PagedSeq q;
    const int32_t s = find_unit<kAppendThreads>(
        P.b, blockIdx.x,
        [](const PagedSeq& q) -> int64_t {
            // 128-position blocks that the new tokens touch (those at positions >= 0)
            return q.nq > 0 && q.kl > 0 ? (q.kl - 1) / kBlock - max(q.kl - q.nq, 0) / kBlock + 1 : 0;
        },
        part, hit, blk, q);
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        for (int32_t i = threadIdx.x; i < P.b.seqs; i += kAppendThreads) {
            PagedSeq q;
            // a chunk longer than its sequence has tokens before position 0
            if (!paged_seq(P.b, i, q) || q.nq > q.kl) atomicCAS(P.b.status, 0, BSA_ERR_BOUNDS);
        }
    }
    if (s < 0) return;
    const int32_t first = q.kl - q.nq;                  // position of the first new token
    blk += max(first, 0) / kBlock;
    const int32_t base = blk * kBlock;
    const int32_t lo = max(max(first, 0), base), hi = min(q.kl, base + kBlock);  // new positions of this block
    const int sub = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
    const bool queries = (int32_t)blockIdx.y < P.q_blocks;
    const int32_t h0 = queries ? 4 * (blockIdx.y / P.q_parts) : blockIdx.y - P.q_blocks;  // first head
    const int32_t heads = min(4, P.H_kv * P.group - h0);  // (of queries)
    if (P.rope != nullptr && hi > P.rope_len && threadIdx.x == 0) atomicCAS(P.b.status, 0, BSA_ERR_BOUNDS);
    const __nv_bfloat16* w = queries ? P.q_norm : P.k_norm;
    float wf[8];
    if (w != nullptr) unpack8(load_row<D, kHalves>(w, c), wf);
    if (queries) {
        const int32_t span = kBlock / P.q_parts, at = base + span * (blockIdx.y % P.q_parts);
        const int32_t from = max(lo, at), to = min(hi, at + span);
        // With kHalves the next token's rows are on their way while this one's are worked
        // on (46.7 -> 44.1 us); the other forms need the registers (11.3 us, 12.8 with it).
        uint4 next[4];
        auto fetch = [&](int32_t pos) {
            const __nv_bfloat16* src = P.q + ((int64_t)q.q0 + (pos - first)) * P.q_stride + h0 * D;
#pragma unroll
            for (int u = 0; u < 4; ++u)
                next[u] = pos < to && u < heads ? load_row<D, kHalves>(src + u * D, c) : make_uint4(0, 0, 0, 0);
        };
        if constexpr (kHalves) fetch(from + sub);
        for (int32_t p0 = from; p0 < to; p0 += kRows) {
            // whole warps stay in the loop: the shuffles need them
            const int32_t pos = p0 + sub;
            if constexpr (!kHalves) fetch(pos);
            uint4 raw[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) raw[u] = next[u];
            Angles a{};
            if (P.rope != nullptr) load_angles<kHalves>(P, c, min(pos, P.rope_len - 1), a);
            if constexpr (kHalves) fetch(pos + kRows);
            __nv_bfloat16* out = P.q_out + ((int64_t)q.q0 + (pos - first)) * P.qo_stride + h0 * D;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float x[8];
                unpack8(raw[u], x);
                if (w != nullptr) norm_row<D>(x, wf, P.eps);
                if (P.rope != nullptr) rotate_row<kHalves>(P, x, c, a);
                if (pos < to && u < heads) store_row<D, kHalves>(out + u * D, c, pack8(x));
            }
        }
        return;
    }
    const int32_t page = P.b.page, per = kBlock / page;
    if (threadIdx.x < per) {
        const int32_t at = base / page + threadIdx.x;
        int32_t id = -1;
        if (at * page < q.kl) {  // pages behind the sequence's end are not looked at
            id = P.b.table[(int64_t)s * P.b.max_pages + at];
            if (id < 0 || id >= P.b.n_pages) {
                atomicCAS(P.b.status, 0, BSA_ERR_BOUNDS);
                id = -1;
            }
        }
        pages[threadIdx.x] = id;
    }
    __syncthreads();

    uint4 next[2][2];  // [token][key, value]
    auto fetch = [&](int32_t p0) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int32_t pos = p0 + u * kRows + sub;
            const int64_t tok = (int64_t)q.q0 + (pos - first);
            next[u][0] = pos < hi ? load_row<D, kHalves>(P.k + tok * P.k_stride + h0 * D, c) : make_uint4(0, 0, 0, 0);
            next[u][1] = pos < hi ? load_row<D, kHalves>(P.v + tok * P.v_stride + h0 * D, c) : make_uint4(0, 0, 0, 0);
        }
    };
    if constexpr (kHalves) fetch(lo);
    for (int32_t p0 = lo; p0 < hi; p0 += 2 * kRows) {
        if constexpr (!kHalves) fetch(p0);
        uint4 raw[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int x = 0; x < 2; ++x) raw[u][x] = next[u][x];
        if constexpr (kHalves) fetch(p0 + 2 * kRows);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int32_t pos = p0 + u * kRows + sub;
            Angles a{};
            if (P.rope != nullptr) load_angles<kHalves>(P, c, min(pos, P.rope_len - 1), a);
            float x[8];
            unpack8(raw[u][0], x);
            if (w != nullptr) norm_row<D>(x, wf, P.eps);
            if (P.rope != nullptr) rotate_row<kHalves>(P, x, c, a);
            const int32_t id = pos < hi ? pages[(pos - base) >> P.page_shift] : -1;
            if (id >= 0) {
                const int64_t slot = ((((int64_t)id * P.H_kv + h0) << P.page_shift) + (pos & (page - 1))) * D;
                store_row<D, kHalves>(P.k_cache + slot, c, pack8(x));
                store_row<D, kHalves>(P.v_cache + slot, c, raw[u][1]);
            }
        }
    }

    if (P.k_mean == nullptr || hi != base + kBlock) return;  // (the whole thread block agrees)
    // the block is full: the mean of its 128 keys as the cache holds them
    const int32_t last = pages[per - 1];
    bool whole = true;
    for (int p = 0; p < per; ++p) whole &= pages[p] >= 0;
    if (!whole) return;
    __syncthreads();  // the keys above are written
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int p = sub; p < kBlock; p += kRows) {
        const __nv_bfloat16* row = P.k_cache + (((int64_t)pages[p / page] * P.H_kv + h0) * page + p % page) * D;
        float f[8];
        unpack8(*reinterpret_cast<const uint4*>(row + 8 * c), f);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += f[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[sub][8 * c + j] = acc[j];
    __syncthreads();
    if (threadIdx.x < D) {
        float t = 0.f;
#pragma unroll
        for (int g = 0; g < kRows; ++g) t += sums[g][threadIdx.x];
        P.k_mean[((int64_t)last * P.H_kv + h0) * D + threadIdx.x] = __float2bfloat16_rn(t * (1.0f / kBlock));
    }
}

}  // namespace

bsa_status launch_paged_append(const PagedAppendArgs& a, int32_t* status, cudaStream_t stream) {
    AppendParams P{};
    P.b = PagedBatch{a.q_start, a.kv_len, a.table, a.seqs, a.tokens, a.max_pages, a.page, a.n_pages, status};
    P.q = static_cast<const __nv_bfloat16*>(a.q);
    P.k = static_cast<const __nv_bfloat16*>(a.k);
    P.v = static_cast<const __nv_bfloat16*>(a.v);
    P.q_stride = a.q_stride;
    P.k_stride = a.k_stride;
    P.v_stride = a.v_stride;
    P.qo_stride = a.qo_stride;
    P.q_out = static_cast<__nv_bfloat16*>(a.q_out);
    P.k_cache = static_cast<__nv_bfloat16*>(a.k_cache);
    P.v_cache = static_cast<__nv_bfloat16*>(a.v_cache);
    P.k_mean = static_cast<__nv_bfloat16*>(a.k_mean);
    P.rope = a.rope;
    P.rope_len = a.rope_len;
    P.rot = a.rot;
    P.interleaved = a.interleaved;
    P.q_norm = static_cast<const __nv_bfloat16*>(a.q_norm);
    P.k_norm = static_cast<const __nv_bfloat16*>(a.k_norm);
    P.eps = a.eps;
    P.H_kv = a.H_kv;
    P.group = a.H / a.H_kv;
    P.page_shift = __builtin_ctz((unsigned)a.page);
    // long chunks: blocks of fewer tokens fill the card more evenly (8192 tokens, 32 + 8
    // heads of 128: whole ones 46 us, halves 43.8, quarters 42.2; chunks of up to 700, 14 + 2
    // heads of 64 without kHalves: halves 10.8 us, quarters 12.0); short ones find their
    // place less often
    const bool halves = a.rope != nullptr && a.rot == a.D && !a.interleaved;
    P.q_parts = a.tokens / a.seqs >= kBlock ? (halves ? 4 : 2) : 1;
    P.q_blocks = a.q != nullptr ? (a.H + 3) / 4 * P.q_parts : 0;
    // a sequence's n > 0 new tokens touch at most (n + 126) / 128 + 1 blocks
    const int64_t units = (int64_t)a.tokens / kBlock + 2 * (int64_t)a.seqs;
    const dim3 grid((unsigned)units, (unsigned)(P.q_blocks + a.H_kv));
    const auto kernel = a.D == 128 ? (halves ? k_paged_append<128, true> : k_paged_append<128, false>)
                                   : (halves ? k_paged_append<64, true> : k_paged_append<64, false>);
    const cudaError_t e = launch_chained(kernel, grid, kAppendThreads, 0, stream, P);
    return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // namespace bsa
