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
// Work mapping.  One thread block per (128-position block that a sequence's
// new tokens touch, group of key/value heads): the block's keys are all
// written by this thread block, so the mean needs no other's work and adds in
// a fixed order, whatever chunks the tokens came in.  A row of D values is
// held by D / 8 neighbouring threads, 16 bytes each; the rotation partner's
// values come by shuffles.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "bsa_internal.h"
#include "bsa_paged.cuh"

namespace bsa {
namespace {

constexpr int kAppendThreads = 256;

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
    int32_t heads_per_block;  // key/value heads of one thread block (with their query heads)
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

// RMS norm of one row over its D values, this thread's values 8 c .. 8 c + 7
// (c: the thread's place among the row's D / 8); w null: left as it is.  Every
// thread of the warp calls it.
template <int D>
__device__ __forceinline__ void norm_row(float (&x)[8], int c, const __nv_bfloat16* w, float eps) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int d = 1; d < D / 8; d <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    if (w == nullptr) return;
    const float r = 1.0f / sqrtf(ss * (1.0f / D) + eps);
    float wf[8];
    unpack8(*reinterpret_cast<const uint4*>(w + 8 * c), wf);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * wf[i];
}

// Rotation of one row at position pos (see norm_row).
__device__ __forceinline__ void rotate_row(const AppendParams& P, float (&x)[8], int c, int32_t pos) {
    const int half = P.rot >> 1;  // a multiple of 8
    const float* cs = P.rope + (int64_t)pos * P.rot;
    if (P.interleaved) {
        if (8 * c < P.rot) {
            const float4 co = *reinterpret_cast<const float4*>(cs + 4 * c);
            const float4 si = *reinterpret_cast<const float4*>(cs + half + 4 * c);
            const float cf[4] = {co.x, co.y, co.z, co.w}, sf[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = x[2 * i], b = x[2 * i + 1];
                x[2 * i] = a * cf[i] - b * sf[i];
                x[2 * i + 1] = b * cf[i] + a * sf[i];
            }
        }
        return;
    }
    // values 8 c .. pair with those of the thread half / 8 places further (or nearer)
    const int step = half >> 3;
    const bool first = c < step, turned = 8 * c < P.rot;
    const int row0 = (threadIdx.x & 31) - c;
    const int from = row0 + (turned ? (first ? c + step : c - step) : c);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], from);
    if (turned) {
        const int at = 8 * (first ? c : c - step);
        float cf[8], sf[8];
        *reinterpret_cast<float4*>(cf) = *reinterpret_cast<const float4*>(cs + at);
        *reinterpret_cast<float4*>(cf + 4) = *reinterpret_cast<const float4*>(cs + at + 4);
        *reinterpret_cast<float4*>(sf) = *reinterpret_cast<const float4*>(cs + half + at);
        *reinterpret_cast<float4*>(sf + 4) = *reinterpret_cast<const float4*>(cs + half + at + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = first ? x[i] * cf[i] - y[i] * sf[i] : x[i] * cf[i] + y[i] * sf[i];
    }
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads) k_paged_append(const __grid_constant__ AppendParams P) {
    constexpr int kLanes = D / 8;
    constexpr int kRows = kAppendThreads / kLanes;  // rows in flight
    __shared__ int64_t part[33];
    __shared__ int32_t hit[2];
    __shared__ int32_t pages[8];  // the block's pages (128 / page of them)
    __shared__ float sums[kRows][D];
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
    const int32_t h0 = blockIdx.y * P.heads_per_block, h1 = min(h0 + P.heads_per_block, P.H_kv);
    const int32_t per_head = (P.q != nullptr ? P.group : 0) + 2;  // rows of a token and key/value head
    const int32_t per_token = (h1 - h0) * per_head;
    const int64_t items = (int64_t)(hi - lo) * per_token;
    for (int64_t i0 = 0; i0 < items; i0 += kRows) {
        // whole warps stay in the loop: the shuffles of turn_row need them
        const int64_t i = i0 + sub;
        const bool live = i < items;
        const int32_t t = live ? (int32_t)(i / per_token) : 0;
        const int32_t r = live ? (int32_t)(i - (int64_t)t * per_token) : 0;
        const int32_t h = h0 + r / per_head, kind = r % per_head;  // 0: key, 1: value, 2 ..: queries
        const int32_t pos = lo + t;
        const int64_t tok = (int64_t)q.q0 + (pos - first);
        const __nv_bfloat16* src;
        __nv_bfloat16* dst = nullptr;
        const __nv_bfloat16* w = nullptr;
        if (kind < 2) {
            const int32_t id = pages[(pos - base) / page];
            const int64_t slot = (((int64_t)id * P.H_kv + h) * page + pos % page) * D;
            src = kind == 0 ? P.k + tok * P.k_stride + h * D : P.v + tok * P.v_stride + h * D;
            if (id >= 0) dst = (kind == 0 ? P.k_cache : P.v_cache) + slot;
            if (kind == 0) w = P.k_norm;
        } else {
            const int32_t hq = h * P.group + kind - 2;
            src = P.q + tok * P.q_stride + hq * D;
            dst = P.q_out + tok * P.qo_stride + hq * D;
            w = P.q_norm;
        }
        const int32_t rp = min(pos, P.rope_len - 1);
        if (P.rope != nullptr && pos >= P.rope_len) {
            if (live && c == 0) atomicCAS(P.b.status, 0, BSA_ERR_BOUNDS);
        }
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (live) raw = *reinterpret_cast<const uint4*>(src + 8 * c);
        float x[8];
        unpack8(raw, x);
        // every lane takes part in the shuffles; a value's row is written as it came
        if (P.q_norm != nullptr || P.k_norm != nullptr) norm_row<D>(x, c, w, P.eps);
        if (P.rope != nullptr) rotate_row(P, x, c, rp);
        if (live && dst != nullptr) *reinterpret_cast<uint4*>(dst + 8 * c) = kind == 1 ? raw : pack8(x);
    }

    if (P.k_mean == nullptr || hi != base + kBlock) return;  // (the whole thread block agrees)
    // the block is full: the mean of its 128 keys as the cache holds them
    const int32_t last = pages[per - 1];
    bool whole = true;
    for (int p = 0; p < per; ++p) whole &= pages[p] >= 0;
    if (!whole) return;
    for (int32_t h = h0; h < h1; ++h) {
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
    P.heads_per_block = 1;
    // a sequence's n > 0 new tokens touch at most (n + 126) / 128 + 1 blocks
    const int64_t units = (int64_t)a.tokens / kBlock + 2 * (int64_t)a.seqs;
    const dim3 grid((unsigned)units, (unsigned)a.H_kv);
    if (a.D == 128) k_paged_append<128><<<grid, kAppendThreads, 0, stream>>>(P);
    else k_paged_append<64><<<grid, kAppendThreads, 0, stream>>>(P);
    return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // namespace bsa
