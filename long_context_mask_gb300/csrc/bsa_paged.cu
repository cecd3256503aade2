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
// new tokens touch and a run of the tokens' rows, a token's rows being (key,
// value, queries) of its key/value heads in turn.  The block that writes a
// head's keys writes all of this position block's, so the mean needs no other's
// work and adds in a fixed order, whatever chunks the tokens came in.  A row of
// D values is held by D / 8 neighbouring threads, eight values each: where the
// whole head turns by halves, four of either half (a pair meets in one thread),
// else eight in a row, with the rotation partner's values by shuffles.  Every thread loads kUnroll rows before it
// works on the first (one row at a time left 16 KB in flight on an SM: a prompt
// of 8192 tokens, 32 + 8 heads of 128, took 107 us, 1.9 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "bsa_internal.h"
#include "bsa_paged.cuh"

namespace bsa {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kUnroll = 4;  // rows that a thread holds at a time

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
    int32_t per_head;        // rows of a token and key/value head: key, value, queries
    int32_t rows_per_block;  // rows of a token that one thread block takes
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

// RMS norm of one row over its D values; w null: left as it is.  Every thread
// of the warp calls it.
template <int D, bool kHalves>
__device__ __forceinline__ void norm_row(float (&x)[8], int c, const __nv_bfloat16* w, float eps) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int d = 1; d < D / 8; d <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    if (w == nullptr) return;
    const float r = 1.0f / sqrtf(ss * (1.0f / D) + eps);
    float wf[8];
    unpack8(load_row<D, kHalves>(w, c), wf);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * wf[i];
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
    __shared__ int32_t hit[2];
    __shared__ int32_t pages[8];  // the block's pages (128 / page of them)
    __shared__ float sums[kRows][D];
    ptx::launch_dependents();
    ptx::wait_primary();
    int32_t blk;
    const int32_t s = find_unit(
        P.b, blockIdx.x,
        [](const PagedSeq& q) -> int64_t {
            // 128-position blocks that the new tokens touch (those at positions >= 0)
            return q.nq > 0 && q.kl > 0 ? (q.kl - 1) / kBlock - max(q.kl - q.nq, 0) / kBlock + 1 : 0;
        },
        part, hit, blk);
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        for (int32_t i = threadIdx.x; i < P.b.seqs; i += kAppendThreads) {
            PagedSeq q;
            // a chunk longer than its sequence has tokens before position 0
            if (!paged_seq(P.b, i, q) || q.nq > q.kl) atomicCAS(P.b.status, 0, BSA_ERR_BOUNDS);
        }
    }
    if (s < 0) return;
    PagedSeq q;
    paged_seq(P.b, s, q);
    const int32_t first = q.kl - q.nq;                  // position of the first new token
    blk += max(first, 0) / kBlock;
    const int32_t base = blk * kBlock;
    const int32_t lo = max(max(first, 0), base), hi = min(q.kl, base + kBlock);  // new positions of this block
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

    const int sub = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
    const int32_t row0 = blockIdx.y * P.rows_per_block;
    const int32_t n_rows = min(P.rows_per_block, P.H_kv * P.per_head - row0);
    // a thread's rows: token t, rows r .. r + kUnroll - 1 of the block's n_rows
    const int32_t groups = (n_rows + kUnroll - 1) / kUnroll;
    const int32_t items = (hi - lo) * groups;
    if (P.rope != nullptr && hi > P.rope_len && threadIdx.x == 0) atomicCAS(P.b.status, 0, BSA_ERR_BOUNDS);
    for (int32_t i0 = 0; i0 < items; i0 += kRows) {
        // whole warps stay in the loop: the shuffles need them
        const int32_t i = i0 + sub;
        const int32_t t = i < items ? i / groups : 0;
        const int32_t r0 = i < items ? (i - t * groups) * kUnroll : n_rows;
        const int32_t pos = lo + t;
        const int64_t tok = (int64_t)q.q0 + (pos - first);
        uint4 raw[kUnroll];
        __nv_bfloat16* dst[kUnroll];
        int kind[kUnroll];  // 0: key, 1: value, 2: query
        const int32_t id = pages[(pos - base) / page];
        const int64_t slot = ((int64_t)id * P.H_kv) * page + pos % page;
        int32_t h = (row0 + r0) / P.per_head, k = row0 + r0 - h * P.per_head;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            raw[u] = make_uint4(0, 0, 0, 0);
            dst[u] = nullptr;
            kind[u] = 1;
            if (r0 + u < n_rows) {
                const __nv_bfloat16* src;
                kind[u] = min(k, 2);
                if (k < 2) {
                    src = k == 0 ? P.k + tok * P.k_stride + h * D : P.v + tok * P.v_stride + h * D;
                    if (id >= 0) dst[u] = (k == 0 ? P.k_cache : P.v_cache) + (slot + (int64_t)h * page) * D;
                } else {
                    const int32_t hq = h * P.group + k - 2;
                    src = P.q + tok * P.q_stride + hq * D;
                    dst[u] = P.q_out + tok * P.qo_stride + hq * D;
                }
                raw[u] = load_row<D, kHalves>(src, c);
            }
            if (++k == P.per_head) {
                k = 0;
                ++h;
            }
        }
        Angles a{};
        if (P.rope != nullptr) load_angles<kHalves>(P, c, min(pos, P.rope_len - 1), a);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float x[8];
            unpack8(raw[u], x);
            // every lane takes part in the shuffles; a value's row is written as it came
            if (P.q_norm != nullptr || P.k_norm != nullptr)
                norm_row<D, kHalves>(x, c, kind[u] == 0 ? P.k_norm : (kind[u] == 2 ? P.q_norm : nullptr), P.eps);
            if (P.rope != nullptr) rotate_row<kHalves>(P, x, c, a);
            if (dst[u] != nullptr) store_row<D, kHalves>(dst[u], c, kind[u] == 1 ? raw[u] : pack8(x));
        }
    }

    if (P.k_mean == nullptr || hi != base + kBlock) return;  // (the whole thread block agrees)
    // the block is full: the mean of its 128 keys as the cache holds them
    const int32_t last = pages[per - 1];
    bool whole = true;
    for (int p = 0; p < per; ++p) whole &= pages[p] >= 0;
    if (!whole) return;
    for (int32_t h = (row0 + P.per_head - 1) / P.per_head; h * P.per_head < row0 + n_rows; ++h) {
        __syncthreads();  // the keys above are written; sums is free again
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int p = sub; p < kBlock; p += kRows) {
            const __nv_bfloat16* row = P.k_cache + (((int64_t)pages[p / page] * P.H_kv + h) * page + p % page) * D;
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
#pragma unroll 8
            for (int g = 0; g < kRows; ++g) t += sums[g][threadIdx.x];
            P.k_mean[((int64_t)last * P.H_kv + h) * D + threadIdx.x] = __float2bfloat16_rn(t * (1.0f / kBlock));
        }
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
    P.per_head = (a.q != nullptr ? P.group : 0) + 2;
    // a sequence's n > 0 new tokens touch at most (n + 126) / 128 + 1 blocks
    const int64_t units = (int64_t)a.tokens / kBlock + 2 * (int64_t)a.seqs;
    // About 512 rows to a thread block, four of a block's 128 tokens, but no more
    // than a key/value head's: a decoding step's means (one block of 128 keys each,
    // for some sequences) are read head by head (32 sequences with all 48 rows in
    // one thread block: 16 us instead of 6).
    const int64_t per_seq = (a.tokens + a.seqs - 1) / a.seqs;
    const int64_t span = per_seq < kBlock ? per_seq : kBlock;
    int64_t rows = 512 / span;
    if (rows > P.per_head) rows = P.per_head;
    P.rows_per_block = (int32_t)rows;
    const dim3 grid((unsigned)units, (unsigned)(((int64_t)a.H_kv * P.per_head + rows - 1) / rows));
    const bool halves = a.rope != nullptr && a.rot == a.D && !a.interleaved;
    const auto kernel = a.D == 128 ? (halves ? k_paged_append<128, true> : k_paged_append<128, false>)
                                   : (halves ? k_paged_append<64, true> : k_paged_append<64, false>);
    const cudaError_t e = launch_chained(kernel, grid, kAppendThreads, 0, stream, P);
    return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // namespace bsa
