// fa_kv4.cuh -- the 4-bit cache's numbers: e2m1 codes in groups of 32 with an
// e5m3 scale (sm_103a).
//
// A row of d values is d/2 bytes of codes and d/32 bytes of scales.  A scale byte
// is bits 14 to 7 of an fp16 (5 exponent bits of bias 15, 3 fraction bits, no
// sign), so byte << 7 is that fp16; 0xFC is NaN.  A code has 2 significant bits
// and a scale 4, so every value is exact in bf16, and code times power of two in
// fp16.
//
// Order of a row's codes: element i of group g = i / 32 is nibble ((i % 32) / 4 *
// (d / 32) + g) * 4 + i % 4, low nibble first.  Eight lanes r hold a row, lane r
// the d/32 adjacent 16-bit pieces with elements 32 g + 4 r to + 3: one load or store
// a lane, in which each piece belongs to one group; lanes 2c and 2c + 1 together
// hold the eight adjacent elements 32 g + 8 c to + 7.
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

#include "fa_prim.cuh"

namespace fa {

constexpr uint32_t kScaleNaN = 0xFC, kScaleMost = 0xF7;   // 0xF7: 61440

// The four bytes of x as pairs of codes, each pair as f16x2 (low nibble in the
// low half): four conversions, two cycles an SM of the ALU's 64 lanes.  Picking 4-bit
// integers apart (shift, mask, subtract) takes three times that.
__device__ __forceinline__ void codes_f16(uint32_t x, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\tmov.b32 {t0, t1, t2, t3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, t0;\n\tcvt.rn.f16x2.e2m1x2 %1, t1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, t2;\n\tcvt.rn.f16x2.e2m1x2 %3, t3;\n\t}"
        : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(x));
}

__device__ __forceinline__ float scale_f32(uint32_t byte) {
    return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}

// The scale byte of a group whose largest magnitude has the bits `most` (an
// integer maximum of them, so a NaN is the largest): the nearest e5m3 number to a
// sixth of it, ties to even; a group with an infinity or a NaN gets NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t most) {
    if (most >= 0x7f800000u) return kScaleNaN;
    const float s = __fdiv_rn(__uint_as_float(most), 6.f);
    if (s < 6.103515625e-5f) return (uint32_t)__float2int_rn(s * 131072.f);   // below 2^-14: steps of 2^-17
    const uint32_t b = __float_as_uint(s);
    const uint32_t r = ((b + 0x7ffffu + ((b >> 20) & 1u)) >> 20) - ((127u - 15u) << 3);
    return r < kScaleMost ? r : kScaleMost;
}

// Codes of four values (two pairs) for scale s with reciprocal inv, both twice: 16
// bits, the first value lowest; ties go to the even code, what is above 6 to 6.  The
// quotient x / s has to be right where it lies on a tie, which bf16 values often do:
// t = x inv is corrected by its remainder x - t s, which an FMA gives exactly, so a
// quotient that fits 24 bits comes out as it is.
__device__ __forceinline__ uint32_t codes_of(uint64_t x01, uint64_t x23, uint64_t minus_s, uint64_t inv) {
    uint64_t t01 = f2_mul(x01, inv), t23 = f2_mul(x23, inv);
    t01 = f2_fma(f2_fma(t01, minus_s, x01), inv, t01);
    t23 = f2_fma(f2_fma(t23, minus_s, x23), inv, t23);
    float t[4];
    f2_unpack(t01, t[0], t[1]);
    f2_unpack(t23, t[2], t[3]);
    uint32_t out;
    asm("{\n\t.reg .b8 lo, hi, z;\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e2m1x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 hi, %4, %3;\n\tmov.b16 h, {lo, hi};\n\tcvt.u32.u16 %0, h;\n\t}"
        : "=r"(out) : "f"(t[0]), "f"(t[1]), "f"(t[2]), "f"(t[3]));
    return out;
}

}  // namespace fa
