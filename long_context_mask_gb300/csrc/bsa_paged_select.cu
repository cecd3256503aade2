// Block selection over a paged key/value cache: for each new token and
// key/value head the blocks with the highest
//     score_j = sum over the head's query heads of  q . (mean key of block j).
//
// Sure of its choice.  The scores that are compared are those of the bf16
// inputs in exact arithmetic (64 bits stand for it).  fp32 sums decide all but
// the close calls: with a the vector of sums of |q| over the query heads, an
// fp32 score is off by at most
//     E = (D + G + 4) 2^-24 |a| max_j |mean_j|
// (D products and additions, G - 1 additions of the query heads, by the
// Cauchy-Schwarz inequality), so with tau the k-th largest fp32 score every
// block above tau + 2E is among the k best and none below tau - 2E is.  Blocks
// in between are scored again in fp64 where there are more of them than places.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "bsa_internal.h"
#include "bsa_paged.cuh"

namespace bsa {
namespace {

constexpr int kSelThreads = 128;

struct SelectParams {
    PagedBatch b;
    const __nv_bfloat16* q;
    int64_t q_stride;
    const __nv_bfloat16* k_mean;
    int32_t H_kv, group, topk, sink, local, width;
    int32_t *sel, *sel_cnt;
    int32_t nb_cap;  // blocks of the longest sequence that the table can hold
};

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

// The k-th largest (1 <= k <= n) of keys[0 .. n - 1]; above: how many are
// larger.  Radix selection, eight bits a pass.  The whole thread block calls
// it; hist: 256 words, box: 2 words of shared memory.
template <typename Key>
__device__ Key kth_largest(const Key* keys, int32_t n, int32_t k, int32_t& above, uint32_t* hist, int32_t* box) {
    Key prefix = 0, mask = 0;
    int32_t want = k;
    above = 0;
    for (int shift = 8 * (int)sizeof(Key) - 8; shift >= 0; shift -= 8) {
        for (int x = threadIdx.x; x < 256; x += kSelThreads) hist[x] = 0u;
        __syncthreads();
        for (int32_t x = threadIdx.x; x < n; x += kSelThreads) {
            const Key v = keys[x];
            if ((v & mask) == prefix) atomicAdd(&hist[(uint32_t)(v >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (threadIdx.x < 32) {
            // lane l: bins 255 - 8 l .. 248 - 8 l, from the top
            uint32_t sum = 0;
            for (int x = 0; x < 8; ++x) sum += hist[255 - 8 * (int)threadIdx.x - x];
            uint32_t incl = sum;
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, incl, d);
                if ((int)threadIdx.x >= d) incl += y;
            }
            uint32_t before = incl - sum;
            if ((int32_t)before < want && (int32_t)incl >= want) {
                int x = 0;
                while ((int32_t)(before + hist[255 - 8 * (int)threadIdx.x - x]) < want)
                    before += hist[255 - 8 * (int)threadIdx.x - x++];
                box[0] = 255 - 8 * (int)threadIdx.x - x;
                box[1] = (int32_t)before;
            }
        }
        __syncthreads();
        prefix |= (Key)(uint32_t)box[0] << shift;
        mask |= (Key)255 << shift;
        above += box[1];
        want -= box[1];
        __syncthreads();
    }
    return prefix;
}

// One thread block per (token, key/value head).
template <int D>
__global__ void __launch_bounds__(kSelThreads) k_paged_select(const __grid_constant__ SelectParams P) {
    extern __shared__ __align__(16) uint8_t dyn[];
    // scores as keys; then, for close calls: their blocks and fp64 keys
    uint64_t* key64 = reinterpret_cast<uint64_t*>(dyn);
    uint32_t* keys = reinterpret_cast<uint32_t*>(key64 + P.nb_cap);
    int32_t* close = reinterpret_cast<int32_t*>(keys + P.nb_cap);
    __shared__ uint32_t chosen[kMaxSelectBlocks / 32];
    __shared__ float qs[D];      // sum of the query heads
    __shared__ float top[2][kSelThreads / 32];
    __shared__ uint32_t hist[256];
    __shared__ int32_t box[2];
    __shared__ int64_t part[33];
    const int32_t tok = blockIdx.x, kvh = blockIdx.y;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kWarps = kSelThreads / 32;

    if (threadIdx.x == 0) box[0] = -1;
    __syncthreads();
    for (int32_t s = threadIdx.x; s < P.b.seqs; s += kSelThreads) {
        PagedSeq y;
        if (!paged_seq(P.b, s, y) && tok == 0 && kvh == 0) atomicCAS(P.b.status, 0, BSA_ERR_BOUNDS);
        if (tok >= y.q0 && tok < y.q0 + y.nq) box[0] = s;
    }
    __syncthreads();
    const int32_t s = box[0];
    if (s < 0) return;  // behind the last sequence: left as it was
    PagedSeq y;
    paged_seq(P.b, s, y);
    const int32_t pos = y.kl - y.nq + (tok - y.q0);
    int32_t* sel = P.sel + ((int64_t)tok * P.H_kv + kvh) * P.width;
    int32_t* cnt = P.sel_cnt + (int64_t)tok * P.H_kv + kvh;
    const int32_t own = pos >= 0 ? pos / kBlock : -1;       // the token's own block
    const int32_t c0 = P.sink, c1 = own - P.local + 1;      // blocks c0 .. c1 - 1 are ranked
    const int32_t nc = max(c1 - c0, 0);
    const int32_t words = (own + 32) / 32;
    // blocks 0 .. own, all of them chosen unless they are ranked
    for (int32_t w = threadIdx.x; w < words; w += kSelThreads) {
        uint32_t bits = 0u;
        for (int i = 0; i < 32; ++i) {
            const int32_t j = 32 * w + i;
            if (j <= own && (nc <= P.topk || j < c0 || j >= c1)) bits |= 1u << i;
        }
        chosen[w] = bits;
    }
    if (nc > P.topk && P.topk > 0) {
        const int32_t* table = P.b.table + (int64_t)s * P.b.max_pages;
        const int32_t per = kBlock / P.b.page;
        const __nv_bfloat16* qrow = P.q + (int64_t)tok * P.q_stride + (int64_t)kvh * P.group * D;
        float norm_a = 0.f;
        for (int d = threadIdx.x; d < D; d += kSelThreads) {
            float sum = 0.f, a = 0.f;
            for (int g = 0; g < P.group; ++g) {
                const float x = __bfloat162float(qrow[g * D + d]);
                sum += x;
                a += fabsf(x);
            }
            qs[d] = sum;
            norm_a = fmaf(a, a, norm_a);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) norm_a += __shfl_xor_sync(0xffffffffu, norm_a, d);
        if (lane == 0) top[0][warp] = norm_a;
        __syncthreads();
        norm_a = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) norm_a += top[0][w];
        // mean key of block j: at the page of its last token
        auto mean_of = [&](int32_t j) -> const __nv_bfloat16* {
            int32_t id = table[(int64_t)(j + 1) * per - 1];
            if (id < 0 || id >= P.b.n_pages) {
                if (lane == 0) atomicCAS(P.b.status, 0, BSA_ERR_BOUNDS);
                id = 0;
            }
            return P.k_mean + ((int64_t)id * P.H_kv + kvh) * D;
        };
        constexpr int kPer = D / 32;  // values of a lane
        float qv[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) qv[i] = qs[lane * kPer + i];
        float most = 0.f;  // largest |mean|^2
        for (int32_t x = warp; x < nc; x += kWarps) {
            const __nv_bfloat16* m = mean_of(c0 + x) + lane * kPer;
            float dot = 0.f, sq = 0.f;
#pragma unroll
            for (int i = 0; i < kPer; i += 2) {
                const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(m + i));
                dot = fmaf(qv[i], f.x, dot);
                dot = fmaf(qv[i + 1], f.y, dot);
                sq = fmaf(f.x, f.x, sq);
                sq = fmaf(f.y, f.y, sq);
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                dot += __shfl_xor_sync(0xffffffffu, dot, d);
                sq += __shfl_xor_sync(0xffffffffu, sq, d);
            }
            if (lane == 0) keys[x] = key_of(dot);
            most = (sq > most || sq != sq) ? sq : most;
        }
        if (lane == 0) top[1][warp] = most;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) most = (top[1][w] > most || top[1][w] != top[1][w]) ? top[1][w] : most;
        // (1.01 covers the rounding of E itself, 1e-36 products that underflow)
        const float E = 1.01f * (float)(D + P.group + 4) * 5.9604645e-8f * sqrtf(norm_a) * sqrtf(most) + 1e-36f;
        int32_t above;
        const uint32_t kth = kth_largest(keys, nc, P.topk, above, hist, box);
        const float tau = of_key(kth);
        // without a finite bound every block is a close call
        const bool bound = tau - tau == 0.0f && E - E == 0.0f;
        const uint32_t hi = bound ? key_of(tau + 2.0f * E) : 0xffffffffu;  // surely chosen: keys above
        const uint32_t lo = bound ? key_of(tau - 2.0f * E) : 0u;           // surely not: keys below
        // the blocks in between, in ascending order
        int32_t n_close = 0, n_sure = 0;
        for (int32_t x0 = 0; x0 < nc; x0 += kSelThreads) {
            const int32_t x = x0 + threadIdx.x;
            const uint32_t k = x < nc ? keys[x] : 0u;
            const bool sure = x < nc && k > hi, maybe = x < nc && k <= hi && k >= lo;
            int64_t total;
            const int64_t at = block_prefix(((int64_t)sure << 32) | (int64_t)maybe, part, total);
            if (sure) atomicOr(&chosen[(c0 + x) >> 5], 1u << ((c0 + x) & 31));
            if (maybe) close[n_close + (int32_t)(at & 0xffffffff)] = x;
            n_sure += (int32_t)(total >> 32);
            n_close += (int32_t)(total & 0xffffffff);
        }
        __syncthreads();
        const int32_t need = P.topk - n_sure;  // places left for the close calls
        if (n_close <= need) {
            for (int32_t x = threadIdx.x; x < n_close; x += kSelThreads)
                atomicOr(&chosen[(c0 + close[x]) >> 5], 1u << ((c0 + close[x]) & 31));
        } else {
            for (int32_t x = warp; x < n_close; x += kWarps) {
                const __nv_bfloat16* m = mean_of(c0 + close[x]) + lane * kPer;
                double dot = 0.0;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    double q = 0.0;
                    for (int g = 0; g < P.group; ++g) q += (double)__bfloat162float(qrow[g * D + lane * kPer + i]);
                    dot = fma(q, (double)__bfloat162float(m[i]), dot);
                }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
                if (lane == 0) key64[x] = key_of(dot);
            }
            __syncthreads();
            int32_t better;
            const uint64_t edge = kth_largest(key64, n_close, need, better, hist, box);
            // equal scores: the lowest blocks
            int32_t left = need - better;
            for (int32_t x0 = 0; x0 < n_close; x0 += kSelThreads) {
                const int32_t x = x0 + threadIdx.x;
                const uint64_t k = x < n_close ? key64[x] : 0ull;
                const bool tie = x < n_close && k == edge;
                int64_t total;
                const int64_t at = block_prefix(tie ? 1 : 0, part, total);
                if (x < n_close && (k > edge || (tie && at < left)))
                    atomicOr(&chosen[(c0 + close[x]) >> 5], 1u << ((c0 + close[x]) & 31));
                left -= (int32_t)total;
            }
        }
    }
    __syncthreads();
    // the chosen blocks in ascending order, then -1
    int32_t n = 0;
    for (int32_t w0 = 0; w0 < words; w0 += kSelThreads) {
        const int32_t w = w0 + threadIdx.x;
        uint32_t bits = w < words ? chosen[w] : 0u;
        int64_t total;
        int32_t at = n + (int32_t)block_prefix(__popc(bits), part, total);
        while (bits) {
            const int b = __ffs(bits) - 1;
            bits &= bits - 1u;
            sel[at++] = 32 * w + b;
        }
        n += (int32_t)total;
    }
    for (int32_t x = n + threadIdx.x; x < P.width; x += kSelThreads) sel[x] = -1;
    if (threadIdx.x == 0) *cnt = n;
}

}  // namespace

size_t paged_select_workspace(const PagedSelectArgs&) { return 0; }

bsa_status launch_paged_select(const PagedSelectArgs& a, void*, int32_t* status, cudaStream_t stream) {
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
    P.nb_cap = (int32_t)(((int64_t)a.max_pages * a.page + kBlock - 1) / kBlock);
    const size_t smem = (size_t)P.nb_cap * 16;
    const dim3 grid((unsigned)a.tokens, (unsigned)a.H_kv);
    auto kernel = a.D == 128 ? k_paged_select<128> : k_paged_select<64>;
    if (smem > 32768 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return BSA_ERR_CUDA;
    kernel<<<grid, kSelThreads, smem, stream>>>(P);
    return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // namespace bsa
