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
//
// Into a cache in 4 bits.  Keys and values are quantised on the way (bsa_fp4.cuh's formulas): some 1.5 times
// the instructions of a bf16 row, most of them for the codes.  Keys and values of a head are two thread blocks' work,
// keys', which take longest, come first in the grid, and a thread block goes through its rows one at a time in a short
// loop; products and quotients are two to an instruction.  (The prompt of 8192: 48 us, 182 MB, 0.56 of the copy rate,
// issue slots 69 % full: the instructions bound it; 75 us with keys and values of two tokens at a time
// in one block, 62 before values went by two.  A step of 32 tokens 5.7 us, 24 ragged chunks 11.5.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "bsa_fp4.cuh"
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
    // a cache in 4 bits: k_cache and v_cache hold codes
    uint8_t *k_scale, *v_scale;
    const float *k_gain, *v_gain;
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

// u a - v b and u a + v b; kEach: each product rounded by itself.
template <bool kEach>
__device__ __forceinline__ float turn_minus(float u, float a, float v, float b) {
    if constexpr (kEach) return __fsub_rn(__fmul_rn(u, a), __fmul_rn(v, b));
    return u * a - v * b;
}
template <bool kEach>
__device__ __forceinline__ float turn_plus(float u, float a, float v, float b) {
    if constexpr (kEach) return __fadd_rn(__fmul_rn(u, a), __fmul_rn(v, b));
    return u * a + v * b;
}

// Rotation of one row.  Every thread of the warp calls it.
template <bool kHalves, bool kEach = false>
__device__ __forceinline__ void rotate_row(const AppendParams& P, float (&x)[8], int c, const Angles& a) {
    if constexpr (kHalves) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float u = x[i], v = x[4 + i];
            x[i] = turn_minus<kEach>(u, a.co[i], v, a.si[i]);
            x[4 + i] = turn_plus<kEach>(v, a.co[i], u, a.si[i]);
        }
        return;
    }
    if (P.interleaved) {
        if (8 * c < P.rot) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = x[2 * i], v = x[2 * i + 1];
                x[2 * i] = turn_minus<kEach>(u, a.co[i], v, a.si[i]);
                x[2 * i + 1] = turn_plus<kEach>(v, a.co[i], u, a.si[i]);
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
        for (int i = 0; i < 8; ++i)
            x[i] = first ? turn_minus<kEach>(x[i], a.co[i], y[i], a.si[i]) : turn_plus<kEach>(x[i], a.co[i], y[i], a.si[i]);
    }
}

// ---------------------------------------------------------------- a cache in 4 bits
// A value next to the middle between two levels goes one way or the other by its last
// bit.  So that the codes do not hang on the order of a sum or on a product and a sum
// being one instruction, keys are worked on in steps that are each rounded by
// themselves, and the norm's factor is 1 / sqrt(mean(x^2) + eps) rounded once (but for
// one row in some 10^5).

// a + b = s + the returned error, exactly (Knuth's two-sum).
__device__ __forceinline__ float two_sum(float a, float b, float& s) {
    s = __fadd_rn(a, b);
    const float t = __fsub_rn(s, a);
    return __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
}
// RMS norm of one row.  Squares of bf16 numbers are exact in fp32; their sum is held
// in two words, and one Newton step on the device's reciprocal root takes its error out.
template <int D>
__device__ __forceinline__ void norm_row_each(float (&x)[8], const float (&w)[8], float eps) {
    // (two chains of four values side by side)
    const uint64_t minus = f2pack(-1.0f, -1.0f);
    uint64_t h2 = f2pack(0.f, 0.f), l2 = h2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t v = f2pack(x[2 * i], x[2 * i + 1]), p = fma2(v, v, f2pack(0.f, 0.f));
        const uint64_t sum = add2(h2, p), t = fma2(h2, minus, sum);
        l2 = add2(l2, add2(fma2(fma2(t, minus, sum), minus, h2), fma2(t, minus, p)));
        h2 = sum;
    }
    float ha, hb, la, lb, hi;
    f2unpack(h2, ha, hb);
    f2unpack(l2, la, lb);
    float lo = two_sum(ha, hb, hi);
    lo = __fadd_rn(__fadd_rn(la, lb), lo);
#pragma unroll
    for (int d = 1; d < D / 8; d <<= 1) {
        const float h = __shfl_xor_sync(0xffffffffu, hi, d), l = __shfl_xor_sync(0xffffffffu, lo, d);
        // (the larger first: hi is not less than what is left of the sum; the same in every thread)
        const float big = fmaxf(hi, h), small = fminf(hi, h);
        hi = __fadd_rn(big, small);
        lo = __fadd_rn(__fadd_rn(lo, l), __fsub_rn(small, __fsub_rn(hi, big)));
    }
    float m;
    const float e = two_sum(hi * (1.0f / D), eps, m);
    const float rest = __fadd_rn(lo * (1.0f / D), e);
    const float r0 = rsqrtf(m), t = __fmul_rn(m, r0);
    float off = fmaf(-t, r0, 1.0f);              // 1 - (m + rest) r0^2
    off = fmaf(-fmaf(m, r0, -t), r0, off);
    off = fmaf(-rest * r0, r0, off);
    const float r = fmaf(0.5f * r0, off, r0);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], r), w[i]);
}

// Quantises and stores this thread's eight values of a row (load_row's places).  Every
// thread of the warp calls it; row < 0: nothing is stored.  recip = 1 / gain, rounded.  Returns
// whether a value of a stored row is not finite (a quotient by the gain that is not is only out of range).
template <int D, bool kHalves>
__device__ __forceinline__ bool store_row_fp4(float (&x)[8], float gain, float recip, uint8_t* codes, uint8_t* scales,
                                              int64_t row, int c) {
    uint64_t t2[4], z = f2pack(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) t2[i] = f2pack(x[2 * i], x[2 * i + 1]);
    if (gain != 1.0f) fp4_quotients(t2, gain, recip, t2);
    float t[8], z0, z1, top[2] = {0.f, 0.f};  // (top: of values 0 .. 3 and 4 .. 7)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        z = fma2(t2[i], f2pack(0.0f, 0.0f), z);  // (NaN where a number is not finite)
        f2unpack(t2[i], t[2 * i], t[2 * i + 1]);
    }
    f2unpack(z, z0, z1);
    bool bad = false;
    if (__any_sync(0xffffffffu, !(z0 + z1 == 0.0f))) {
        // infinities, and what the gain makes one: the largest number; NaN: 0
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            bad |= !(fabsf(x[i]) <= FLT_MAX);
            t[i] = fabsf(t[i]) <= FLT_MAX ? t[i] : x[i] == x[i] ? copysignf(FLT_MAX, x[i]) : 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) top[i >> 2] = fmaxf(top[i >> 2], fabsf(t[i]));
    if constexpr (kHalves) {  // four threads hold a group, in either half
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], d));
            top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], d));
        }
    } else {                  // two threads
        top[0] = fmaxf(top[0], top[1]);
        top[0] = top[1] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], 1));
    }
    float scale[2];
    uint32_t byte[2], code[2];
    byte[0] = fp4_scale_of(top[0], scale[0]);
    byte[1] = byte[0];
    scale[1] = scale[0];
    if constexpr (kHalves) byte[1] = fp4_scale_of(top[1], scale[1]);
    // (no level but 0 where the scale is 0)
    uint64_t y2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y2[i] = f2pack(t[2 * i], t[2 * i + 1]);
    float s[2], r[2];
    s[0] = scale[0] > 0.0f ? scale[0] : FLT_MAX;
    r[0] = scale[0] > 0.0f ? __frcp_rn(scale[0]) : 0.0f;
    if constexpr (kHalves) {
        s[1] = scale[1] > 0.0f ? scale[1] : FLT_MAX;
        r[1] = scale[1] > 0.0f ? __frcp_rn(scale[1]) : 0.0f;
    } else {
        s[1] = s[0];
        r[1] = r[0];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint64_t r2 = f2pack(r[h], r[h]), s2 = f2pack(-s[h], -s[h]);
        float y[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint64_t v = y2[2 * h + i], q = fma2(v, r2, f2pack(0.0f, 0.0f));
            f2unpack(fma2(fma2(q, s2, v), r2, q), y[2 * i], y[2 * i + 1]);
        }
        code[h] = fp4_codes4(y[0], y[1], y[2], y[3]);
    }
    if (row < 0) return false;
    uint8_t* to = codes + row * (D / 2);
    uint8_t* ts = scales + row * (D / kFp4Group);
    if constexpr (kHalves) {
        *reinterpret_cast<uint16_t*>(to + 2 * c) = (uint16_t)code[0];
        *reinterpret_cast<uint16_t*>(to + D / 4 + 2 * c) = (uint16_t)code[1];
        if ((c & 3) == 0) {
            ts[c >> 2] = (uint8_t)byte[0];
            ts[D / 32 + (c >> 2)] = (uint8_t)byte[1];
        }
    } else {
        *reinterpret_cast<uint32_t*>(to + 4 * c) = code[0] | code[1] << 16;
        if ((c & 1) == 0) ts[c >> 1] = (uint8_t)byte[0];
    }
    return bad;
}
// Values 8 c .. 8 c + 7 of a row, without the gain.
template <int D>
__device__ __forceinline__ void load_row_fp4(const uint8_t* codes, const uint8_t* scales, int64_t row, int c, float (&x)[8]) {
    __half2 h[4];
    fp4_levels(*reinterpret_cast<const uint32_t*>(codes + row * (D / 2) + 4 * c), h);
    const __half2 s = __half2half2(__low2half(fp4_scales(scales[row * (D / kFp4Group) + (c >> 1)])));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(__hmul2(h[i], s));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <int D, bool kHalves, bool kFp4>
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
    // (a cache in 4 bits: its keys, which take longest, and values come first)
    const int32_t kv_first = kFp4 ? 2 * P.H_kv : 0;
    const int32_t by = (int32_t)blockIdx.y < kv_first ? P.q_blocks + (int32_t)blockIdx.y : (int32_t)blockIdx.y - kv_first;
    const bool queries = by < P.q_blocks;
    // a cache in 4 bits: keys and values of a head are two blocks' work
    const bool values = kFp4 && ((by - P.q_blocks) & 1) != 0;
    const int32_t h0 = queries ? 4 * (by / P.q_parts) : (by - P.q_blocks) / (kFp4 ? 2 : 1);  // first head
    const int32_t heads = min(4, P.H_kv * P.group - h0);  // (of queries)
    if (P.rope != nullptr && hi > P.rope_len && threadIdx.x == 0) atomicCAS(P.b.status, 0, BSA_ERR_BOUNDS);
    const __nv_bfloat16* w = queries ? P.q_norm : P.k_norm;
    float wf[8];
    if (w != nullptr) unpack8(load_row<D, kHalves>(w, c), wf);
    if (queries) {
        const int32_t span = kBlock / P.q_parts, at = base + span * (by % P.q_parts);
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

    if constexpr (kFp4) {
        // one row at a time in a short loop, the next one under way; whole warps stay in it
        const __nv_bfloat16* src = (values ? P.v : P.k) + h0 * D;
        const int64_t stride = values ? P.v_stride : P.k_stride;
        const float* gains = values ? P.v_gain : P.k_gain;
        const float gain = gains != nullptr ? gains[h0] : 1.0f, recip = __frcp_rn(gain);
        uint8_t* codes = reinterpret_cast<uint8_t*>(values ? P.v_cache : P.k_cache);
        uint8_t* scales = values ? P.v_scale : P.k_scale;
        auto fetch = [&](int32_t pos) -> uint4 {
            return pos < hi ? load_row<D, kHalves>(src + ((int64_t)q.q0 + (pos - first)) * stride, c) : make_uint4(0, 0, 0, 0);
        };
        bool bad = false;  // a value that is not finite
        uint4 next = fetch(lo + sub);
#pragma unroll 1
        for (int32_t pos = lo + sub; pos - sub < hi; pos += kRows) {
            float x[8];
            unpack8(next, x);
            next = fetch(pos + kRows);
            if (!values) {
                if (w != nullptr) norm_row_each<D>(x, wf, P.eps);
                if (P.rope != nullptr) {
                    Angles a{};
                    load_angles<kHalves>(P, c, min(pos, P.rope_len - 1), a);
                    rotate_row<kHalves, true>(P, x, c, a);
                }
            }
            const int32_t id = pos < hi ? pages[(pos - base) >> P.page_shift] : -1;
            const int64_t slot = id >= 0 ? (((int64_t)id * P.H_kv + h0) << P.page_shift) + (pos & (page - 1)) : -1;
            bad |= store_row_fp4<D, kHalves>(x, gain, recip, codes, scales, slot, c);
        }
        if (bad) atomicCAS(P.b.status, 0, BSA_ERR_NONFINITE);
        if (values) return;
    } else {
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
        const int64_t row = ((int64_t)pages[p / page] * P.H_kv + h0) * page + p % page;
        float f[8];
        if constexpr (kFp4) load_row_fp4<D>(reinterpret_cast<const uint8_t*>(P.k_cache), P.k_scale, row, c, f);
        else unpack8(*reinterpret_cast<const uint4*>(P.k_cache + row * D + 8 * c), f);
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
        t *= 1.0f / kBlock;  // (before the gain: fp32 holds the mean where it may not hold the sum)
        if (kFp4 && P.k_gain != nullptr) t *= P.k_gain[h0];
        P.k_mean[((int64_t)last * P.H_kv + h0) * D + threadIdx.x] = __float2bfloat16_rn(t);
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
    const bool fp4 = a.k_scale != nullptr;
    const dim3 grid((unsigned)units, (unsigned)(P.q_blocks + (fp4 ? 2 : 1) * a.H_kv));
    P.k_scale = static_cast<uint8_t*>(a.k_scale);
    P.v_scale = static_cast<uint8_t*>(a.v_scale);
    P.k_gain = a.k_gain;
    P.v_gain = a.v_gain;
    const auto kernel =
        fp4 ? (a.D == 128 ? (halves ? k_paged_append<128, true, true> : k_paged_append<128, false, true>)
                          : (halves ? k_paged_append<64, true, true> : k_paged_append<64, false, true>))
            : (a.D == 128 ? (halves ? k_paged_append<128, true, false> : k_paged_append<128, false, false>)
                          : (halves ? k_paged_append<64, true, false> : k_paged_append<64, false, false>));
    const cudaError_t e = launch_chained(kernel, grid, kAppendThreads, 0, stream, P);
    return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // namespace bsa
