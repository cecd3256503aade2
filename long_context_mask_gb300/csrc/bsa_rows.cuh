// Device helpers shared by the attention kernels: packed fp32 arithmetic, and
// the row-split softmax and epilogue over tensor-memory tiles (two warps per
// lane quadrant, four threads per query row).
#pragma once

#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "bsa_math.cuh"
#include "bsa_ptx.cuh"

namespace bsa {

using namespace ptx;

__device__ __forceinline__ void raise_status(int32_t* status, int32_t code) {
    atomicCAS(status, 0, code);
}

// Bits lo .. hi-1 of a 32-bit word, the bounds clamped to [0, 32].
__device__ __forceinline__ uint32_t run_bits(int32_t lo, int32_t hi) {
    const uint32_t l = (uint32_t)min(max(lo, 0), 32), h = (uint32_t)min(max(hi, 0), 32);
    return h > l ? (uint32_t)(((1ull << h) - 1ull) ^ ((1ull << l) - 1ull)) : 0u;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}

// Two fp32 values in one 64-bit register pair, and the packed f32x2
// arithmetic of sm_100+ (each lane rounds exactly as fmaf / +).
__device__ __forceinline__ uint64_t f2pack(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2unpack(uint64_t r, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// ---------------------------------------------------------------- row split
// Two softmax warps per TMEM lane quadrant, each over 16 lanes (query rows):
// thread t holds rows t/4 and t/4 + 8 of its warp's 16 ("a" and "b") and,
// of each, the 32 columns 2 (t % 4) + 8 k and 2 (t % 4) + 8 k + 1 (the
// tcgen05 16x256b layout: s[4k], s[4k+1] row a, s[4k+2], s[4k+3] row b).
// The four threads of a row are lanes 4 (t/4) .. 4 (t/4) + 3 of the warp.

// Row maxima of rows a and b over all 128 columns (shuffles within the row's
// four threads).
__device__ __forceinline__ void max_rows(const uint32_t (&s)[64], float& ma, float& mb) {
    float a0 = -INFINITY, a1 = -INFINITY, b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
        a0 = fmax3(a0, __uint_as_float(s[4 * k + 0]), __uint_as_float(s[4 * k + 1]));
        b0 = fmax3(b0, __uint_as_float(s[4 * k + 2]), __uint_as_float(s[4 * k + 3]));
        a1 = fmax3(a1, __uint_as_float(s[4 * k + 4]), __uint_as_float(s[4 * k + 5]));
        b1 = fmax3(b1, __uint_as_float(s[4 * k + 6]), __uint_as_float(s[4 * k + 7]));
    }
    ma = fmaxf(a0, a1);
    mb = fmaxf(b0, b1);
    ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, 1));
    mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
    ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, 2));
    mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
}

// P = 2^(s * sl2 + bias) for this thread's 64 scores, packed as bf16 pairs
// in the 16x128b layout (s[2k] row a, s[2k+1] row b, column (t % 4) + 4 k);
// la, lb receive this thread's share of the two row sums.
template <int kPoly>
__device__ __forceinline__ void exp_rows(uint32_t (&s)[64], float sl2, float bias_a, float bias_b, float& la,
                                         float& lb) {
    const uint64_t a2 = f2pack(sl2, sl2), ba = f2pack(bias_a, bias_a), bb = f2pack(bias_b, bias_b);
    uint64_t acc_a0 = f2pack(0.f, 0.f), acc_a1 = acc_a0, acc_b0 = acc_a0, acc_b1 = acc_a0;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        float x[4];
        f2unpack(fma2(f2pack(__uint_as_float(s[4 * k]), __uint_as_float(s[4 * k + 1])), a2, ba), x[0], x[1]);
        f2unpack(fma2(f2pack(__uint_as_float(s[4 * k + 2]), __uint_as_float(s[4 * k + 3])), a2, bb), x[2], x[3]);
        float p[4];
        // column of x[i]: 2 (t % 4) + 8 k + (i & 1); its residue mod 8 decides the unit
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = kPoly > 0 && (((threadIdx.x & 3) * 2 + (i & 1)) < kPoly) ? exp2_fma(x[i]) : ex2(x[i]);
        if (k & 1) {
            acc_a1 = add2(acc_a1, f2pack(p[0], p[1]));
            acc_b1 = add2(acc_b1, f2pack(p[2], p[3]));
        } else {
            acc_a0 = add2(acc_a0, f2pack(p[0], p[1]));
            acc_b0 = add2(acc_b0, f2pack(p[2], p[3]));
        }
        s[2 * k] = pack_bf16(p[0], p[1]);
        s[2 * k + 1] = pack_bf16(p[2], p[3]);
    }
    float x0, x1;
    f2unpack(add2(acc_a0, acc_a1), x0, x1);
    la = x0 + x1;
    f2unpack(add2(acc_b0, acc_b1), x0, x1);
    lb = x0 + x1;
}

// P = 0 for this warp's 16 rows of a score buffer (the 16x128b layout the
// softmax writes P in), for a block that no row of its quadrant sees.
__device__ __forceinline__ void store_p_zero(uint32_t taddr) {
    uint32_t z[32];
#pragma unroll
    for (int c = 0; c < 32; ++c) z[c] = 0u;
    tmem_st16x128_x16(taddr, z);
    tmem_wait_st();
}

// A row's sum over its four threads (the same value in each).
__device__ __forceinline__ float row_sum4(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// Transpose of a 4 x 4 block of words held by the four threads of a row
// (thread c of the row holds x[0..3]; afterwards x[j] is thread j's former
// x[c]), by two butterfly exchanges.
__device__ __forceinline__ void transpose4(uint32_t x[4], int c) {
#pragma unroll
    for (int m = 2; m >= 1; m >>= 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j & m) continue;
            const bool hi = (c & m) != 0;
            const uint32_t recv = __shfl_xor_sync(0xffffffffu, hi ? x[j] : x[j | m], m);
            if (hi) x[j] = recv;
            else x[j | m] = recv;
        }
    }
}

// O rows a and b (16x256b layout: o[4k..4k+3] = row a's columns 8k + 2c,
// 8k + 2c + 1, then row b's, c = thread % 4) divided by their sums, as bf16
// pairs: pk[k] row a's, pk[D/8 + k] row b's.
template <int D>
__device__ __forceinline__ void pack_o_pairs(const uint32_t* o, float inv_a, float inv_b, uint32_t* pk) {
#pragma unroll
    for (int k = 0; k < D / 8; ++k) {
        pk[k] = pack_bf16(__uint_as_float(o[4 * k]) * inv_a, __uint_as_float(o[4 * k + 1]) * inv_a);
        pk[D / 8 + k] = pack_bf16(__uint_as_float(o[4 * k + 2]) * inv_b, __uint_as_float(o[4 * k + 3]) * inv_b);
    }
}

// Stores packed O rows.  Within each group of four words the row's four
// threads exchange words, so that thread c then holds 8 consecutive columns,
// 8 (4g + c) .., and writes them with one 16-byte store: the four threads of
// a row write 64 bytes of it per store instead of 16.  Every lane takes part
// in the exchanges; a null row pointer skips that row's stores.
template <int D>
__device__ __forceinline__ void store_packed_pairs(const uint32_t* pk, __nv_bfloat16* row_a, __nv_bfloat16* row_b) {
    const int c = threadIdx.x & 3;
#pragma unroll
    for (int g = 0; g < D / 32; ++g) {
        uint32_t xa[4], xb[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            xa[j] = pk[4 * g + j];
            xb[j] = pk[D / 8 + 4 * g + j];
        }
        transpose4(xa, c);
        transpose4(xb, c);
        if (row_a) *reinterpret_cast<uint4*>(row_a + 8 * (4 * g + c)) = make_uint4(xa[0], xa[1], xa[2], xa[3]);
        if (row_b) *reinterpret_cast<uint4*>(row_b + 8 * (4 * g + c)) = make_uint4(xb[0], xb[1], xb[2], xb[3]);
    }
}

template <int D>
__device__ __forceinline__ void store_o_pairs(const uint32_t* o, float inv_a, float inv_b, __nv_bfloat16* row_a,
                                              __nv_bfloat16* row_b) {
    uint32_t pk[D / 4];
    pack_o_pairs<D>(o, inv_a, inv_b, pk);
    store_packed_pairs<D>(pk, row_a, row_b);
}

// O columns of rows a and b out of tensor memory (16x256b layout, D / 4 per
// row per thread), multiplied by per-row factors, back in.
template <int D>
__device__ __forceinline__ void scale_o_rows(uint32_t taddr, float fa, float fb) {
    uint32_t o[D / 2];
    if constexpr (D == 128) tmem_ld16x256_x16(taddr, o);
    else tmem_ld16x256_x8(taddr, o);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < D / 2; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * (((i >> 1) & 1) ? fb : fa));
    if constexpr (D == 128) tmem_st16x256_x16(taddr, o);
    else tmem_st16x256_x8(taddr, o);
}

// Normalised O of rows a and b (bf16) to their output rows: this thread's
// column pairs 2 (t % 4) + 8 k.
template <int D>
__device__ __forceinline__ void store_o_rows(uint32_t taddr, float inv_a, float inv_b, __nv_bfloat16* row_a,
                                             __nv_bfloat16* row_b) {
    uint32_t o[D / 2];
    if constexpr (D == 128) tmem_ld16x256_x16(taddr, o);
    else tmem_ld16x256_x8(taddr, o);
    tmem_wait_ld();
    store_o_pairs<D>(o, inv_a, inv_b, row_a, row_b);
}

}  // namespace bsa
