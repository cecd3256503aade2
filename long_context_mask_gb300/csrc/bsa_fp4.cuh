// Rows of a key/value cache held in 4 bits.
//
// A row (one token and head, D values) is D / 2 bytes of codes and D / 16
// scales.  Value d is level(code_d) * scale_(d / 16) * gain: the code a 4-bit
// float e2m1 (value 2 i in the low half of byte i), the scale an 8-bit float
// e4m3, the gain one fp32 number for the head.  Level and scale together have
// at most six significant bits between 2^-10 and 2688, so their product is exact
// in fp16 and in bf16; what multiplies all of a head's values alike, the gain, is
// left to the score's factor and to the end of the sum over values.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "bsa_rows.cuh"

namespace bsa {

constexpr int kFp4Group = 16;        // values that share a scale
constexpr float kFp4Most = 6.0f;     // the largest level

// The scales of two groups (one byte each) as fp16 numbers.  A scale is a
// magnitude: a negative or NaN byte, which no append writes, counts as 0, so that
// nothing read from the cache is ever infinite or NaN.
__device__ __forceinline__ __half2 fp4_scales(uint32_t two_bytes) {
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two_bytes));
    return __hmax2(*reinterpret_cast<__half2*>(&r), __half2half2(__ushort_as_half(0)));
}

// The eight levels of a word of codes, in pairs (values 2 i and 2 i + 1).
__device__ __forceinline__ void fp4_levels(uint32_t w, __half2 (&x)[4]) {
    uint32_t r[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<__half2*>(&r[i]);
}

// x / y rounded to nearest, given recip = 1 / y rounded to nearest: a product, and one step of the
// remainder (Markstein's theorem, IBM J. Res. Dev. 34 (1990), makes it the rounded quotient where
// nothing over- or underflows).  Not finite where x or the quotient is not, or recip.
__device__ __forceinline__ float fp4_quotient(float x, float y, float recip) {
    const float q = x * recip;
    return fmaf(fmaf(-q, y, x), recip, q);
}
// The same for eight numbers, two at a time.
__device__ __forceinline__ void fp4_quotients(const uint64_t (&x)[4], float y, float recip, uint64_t (&out)[4]) {
    const uint64_t y2 = f2pack(-y, -y), r2 = f2pack(recip, recip), none = f2pack(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t q = fma2(x[i], r2, none);
        out[i] = fma2(fma2(q, y2, x[i]), r2, q);
    }
}

// The scale byte of a group whose largest magnitude is `most` (finite), and the scale.
__device__ __forceinline__ uint32_t fp4_scale_of(float most, float& scale) {
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tcvt.u32.u16 %0, t;\n\t}"
        : "=r"(r) : "f"(0.0f), "f"(fp4_quotient(most, kFp4Most, 1.0f / kFp4Most)));
    scale = __low2float(fp4_scales(r));
    return r;
}

// Codes of four ratios, the first in the lowest bits.
__device__ __forceinline__ uint32_t fp4_codes4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b8 lo, hi;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi, lo, hi};\n\t}"
        : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r & 0xffffu;
}

}  // namespace bsa
