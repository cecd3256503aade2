// Reading a key/value cache held in 4 bits back: the last new tokens of every
// sequence of a ragged batch, out of their pages, as bf16 rows [tokens, H_kv, D].
//
// A value is level * scale, exact in fp32, times the head's gain, rounded once (see read_values).
// The work is bound by its bytes (nine read for every 64 written; 131072 tokens of 8 heads of 128, 687 MB:
// 109 us, 0.93 of the copy rate, 114 with gains; 6 tails of up to 150 tokens: 3.1 us, a launch's latency).  A thread block takes up to
// 64 tokens' keys or values; a thread has one place of a token's H_kv D values, eight of
// them, and goes through the tokens, four loads under way at a time, so that the
// block's threads write whole tokens one after another.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bsa_fp4.cuh"
#include "bsa_internal.h"
#include "bsa_paged.cuh"

namespace bsa {
namespace {

constexpr int kReadThreads = 256;
constexpr int kReadTokens = 64;   // of a thread block, at most

struct ReadParams {
    PagedBatch b;
    const uint8_t *codes[2], *scales[2];  // keys, values
    const float* gain[2];
    __nv_bfloat16* out[2];
    int64_t stride[2];
    int32_t H_kv;
    int32_t first;  // blockIdx.y 0 is this one of the two
    int32_t span;   // tokens of a thread block, at most kReadTokens
};

// Eight values of codes w under a scale y, as they are (exact) or times the gain g: the bf16 numbers nearest to the
// products.  A product rounded to fp32 and then to bf16 goes astray only where the first rounding has ended halfway
// between two bf16 numbers (low half 0x8000: one value in some 2^16); read_halfway moves it there by its last bit towards
// the product, which is exact in fp64 (6 + 24 bits).
__device__ __forceinline__ void fp4_products(uint32_t w, uint32_t y, float2 (&x)[4]) {
    __half2 h[4];
    fp4_levels(w, h);
    const __half2 sc = __half2half2(__low2half(fp4_scales(y)));
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __half22float2(__hmul2(h[i], sc));
}
__device__ __noinline__ uint4 read_halfway(uint32_t w, uint32_t y, float g) {
    float2 x[4];
    fp4_products(w, y, x);
    auto nearest = [&](float v) -> float {
        const float p = v * g;
        const double off = fma((double)v, (double)g, -(double)p);
        if ((__float_as_uint(p) & 0xffffu) != 0x8000u || off == 0.0) return p;
        return __uint_as_float(__float_as_uint(p) + ((off > 0.0) == (p > 0.0f) ? 1u : ~0u));
    };
    return make_uint4(pack_bf16(nearest(x[0].x), nearest(x[0].y)), pack_bf16(nearest(x[1].x), nearest(x[1].y)),
                      pack_bf16(nearest(x[2].x), nearest(x[2].y)), pack_bf16(nearest(x[3].x), nearest(x[3].y)));
}
template <bool kGain>
__device__ __forceinline__ uint4 read_values(uint32_t w, uint32_t y, float g) {
    float2 x[4];
    fp4_products(w, y, x);
    if constexpr (kGain) {
        uint32_t low[4];  // two products' low halves: as signed numbers, 0x8000 is the smallest
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i].x *= g;
            x[i].y *= g;
            low[i] = __byte_perm(__float_as_uint(x[i].x), __float_as_uint(x[i].y), 0x5410);
        }
        const uint32_t least = __vimin3_s16x2(__vimin3_s16x2(low[0], low[1], low[2]), low[3], low[3]);
        if ((least & 0xffffu) == 0x8000u || least >> 16 == 0x8000u) return read_halfway(w, y, g);
    }
    return make_uint4(pack_bf16(x[0].x, x[0].y), pack_bf16(x[1].x, x[1].y), pack_bf16(x[2].x, x[2].y), pack_bf16(x[3].x, x[3].y));
}

template <int D, bool kGain>
__global__ void __launch_bounds__(kReadThreads, 8) k_paged_read(const __grid_constant__ ReadParams P) {
    __shared__ int64_t part[33];
    __shared__ int32_t hit[5];
    __shared__ int32_t slot[kReadTokens];  // row of head 0 of each token (-1: none)
    ptx::launch_dependents();
    ptx::wait_primary();
    int32_t chunk;
    PagedSeq q;
    const int32_t s = find_unit<kReadThreads>(
        P.b, blockIdx.x, [&](const PagedSeq& q) -> int64_t { return ((int64_t)q.nq + P.span - 1) / P.span; }, part, hit, chunk, q);
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        for (int32_t i = threadIdx.x; i < P.b.seqs; i += kReadThreads) {
            PagedSeq x;
            // more tokens than the sequence has: those before position 0 are left out
            if (!paged_seq(P.b, i, x) || x.nq > x.kl) atomicCAS(P.b.status, 0, BSA_ERR_BOUNDS);
        }
    }
    if (s < 0) return;
    const int32_t t0 = chunk * P.span, n = min(P.span, q.nq - t0);
    const int32_t page = P.b.page;
    if (threadIdx.x < n) {
        const int32_t pos = q.kl - q.nq + t0 + threadIdx.x;
        int32_t at = -1;
        if (pos >= 0) {
            const int32_t id = P.b.table[(int64_t)s * P.b.max_pages + pos / page];
            if (id >= 0 && id < P.b.n_pages) at = id * P.H_kv * page + pos % page;
            else atomicCAS(P.b.status, 0, BSA_ERR_BOUNDS);
        }
        slot[threadIdx.x] = at;
    }
    __syncthreads();
    const int which = P.first + blockIdx.y;
    const uint8_t* codes = which ? P.codes[1] : P.codes[0];
    const uint8_t* scales = which ? P.scales[1] : P.scales[0];
    const float* gain = which ? P.gain[1] : P.gain[0];
    __nv_bfloat16* out = which ? P.out[1] : P.out[0];
    const int64_t stride = which ? P.stride[1] : P.stride[0];
    const int32_t places = P.H_kv * (D / 8), wide = min(places, kReadThreads);
    const int32_t abreast = kReadThreads / wide, sub = threadIdx.x / wide;
    if (sub >= abreast) return;
    for (int32_t x = threadIdx.x - sub * wide; x < places; x += wide) {
        const int32_t head = x / (D / 8), c = x % (D / 8);
        const float g = kGain && gain != nullptr ? gain[head] : 1.0f;
        for (int32_t t = sub; t < n; t += 4 * abreast) {
            uint32_t w[4], y[4];
            int32_t at[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int32_t tu = t + u * abreast;
                at[u] = tu < n ? slot[tu] : -1;
                const int64_t row = (int64_t)max(at[u], 0) + head * page;
                w[u] = at[u] >= 0 ? *reinterpret_cast<const uint32_t*>(codes + row * (D / 2) + 4 * c) : 0u;
                y[u] = at[u] >= 0 ? scales[row * (D / kFp4Group) + (c >> 1)] : 0u;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (at[u] < 0) continue;
                __nv_bfloat16* to = out + ((int64_t)q.q0 + t0 + t + u * abreast) * stride + head * D + 8 * c;
                *reinterpret_cast<uint4*>(to) = read_values<kGain>(w[u], y[u], g);
            }
        }
    }
}

}  // namespace

bsa_status launch_paged_read(const PagedReadArgs& a, int32_t* status, cudaStream_t stream) {
    ReadParams P{};
    P.b = PagedBatch{a.q_start, a.kv_len, a.table, a.seqs, a.tokens, a.max_pages, a.page, a.n_pages, status};
    P.codes[0] = static_cast<const uint8_t*>(a.k);
    P.codes[1] = static_cast<const uint8_t*>(a.v);
    P.scales[0] = static_cast<const uint8_t*>(a.k_scale);
    P.scales[1] = static_cast<const uint8_t*>(a.v_scale);
    P.gain[0] = a.k_gain;
    P.gain[1] = a.v_gain;
    P.out[0] = static_cast<__nv_bfloat16*>(a.k_out);
    P.out[1] = static_cast<__nv_bfloat16*>(a.v_out);
    P.stride[0] = a.k_stride;
    P.stride[1] = a.v_stride;
    P.H_kv = a.H_kv;
    P.first = a.k_out != nullptr ? 0 : 1;
    // Tokens of a thread block: fewer where there would be too few blocks to hide the loads (an SM holds eight), as long as
    // a thread keeps a few pieces.  (8 heads of 128, spans of 64, 32, 16, 8: 8192 tokens 14.6, 11.0, 8.8, 10.9 us; 32768
    // 35.2, 31.7, 33.5, 40.9; 131072 110.0, 111.5, 123, 155; 40 heads, 8192: 76, 50, 46, 40.)
    const int64_t sides = a.k_out != nullptr && a.v_out != nullptr ? 2 : 1;
    P.span = kReadTokens;
    while (P.span > 8) {
        const int64_t blocks = ((int64_t)a.tokens / P.span + a.seqs) * sides, pieces = (int64_t)P.span * a.H_kv * (a.D / 8);
        if (!(pieces > 16 * kReadThreads && blocks < 8 * kPagedBlocks) && !(pieces > 4 * kReadThreads && blocks < 4 * kPagedBlocks)) break;
        P.span /= 2;
    }
    // sum over sequences of ceil(n / span) <= tokens / span + seqs
    const dim3 grid((unsigned)(a.tokens / P.span + a.seqs), (unsigned)sides);
    const bool gains = (a.k_out != nullptr && a.k_gain != nullptr) || (a.v_out != nullptr && a.v_gain != nullptr);
    const auto kernel = a.D == 128 ? (gains ? k_paged_read<128, true> : k_paged_read<128, false>)
                                   : (gains ? k_paged_read<64, true> : k_paged_read<64, false>);
    const cudaError_t e = launch_chained(kernel, grid, kReadThreads, 0, stream, P);
    return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // namespace bsa
