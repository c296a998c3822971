// E4M3 quantization shared by the FP8 appends.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

// E4M3 codes of correctly rounded float32 quotients x / s (s > 0) without a
// division, r = the correctly rounded reciprocal of s.
//
// q0 = RN(x * r) lies within one ulp of x / s (the rounding of the product
// and r's own half ulp).  One correction step then gives the correctly
// rounded quotient: e = x - s * q0 is exact (one fused multiply-add), and
// RN(q0 + e * r) = RN(x / s) when r = RN(1/s) and q0 is within one ulp, in
// the normal range (Markstein's theorem on the final step of an FMA
// division: P. Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", IBM J. Res. Dev. 34(1), 1990).  The step is
// taken where the last ulp can change the E4M3 code, 2^-11 <= |q0| <= 512:
// below, the code is a zero of x's sign; above, E4M3 saturates (448); NaN
// stays NaN.  Checked against the IEEE quotient on every bf16 input for
// thousands of scales, codes compared, and against the oracle's codes in the
// GPU tests.
__device__ __forceinline__ float e4m3_quotient(float x, float s, float r)
{
    const float q0 = __fmul_rn(x, r);
    const float e = __fmaf_rn(-s, q0, x);
    const float q1 = __fmaf_rn(e, r, q0);
    const uint32_t a = __float_as_uint(q0) & 0x7FFFFFFFu;
    return (a - 0x3A000000u) <= 0x0A000000u ? q1 : q0;  // 2^-11 .. 512 as bits
}

__device__ __forceinline__ uint32_t quant4(uint32_t a, uint32_t b, float s, float r)
{
    // bf16 pairs a = (x0, x1), b = (x2, x3) -> codes x0 | x1 << 8 | x2 << 16 | x3 << 24
    const float q0 = e4m3_quotient(bf16lo_to_f32(a), s, r);
    const float q1 = e4m3_quotient(bf16hi_to_f32(a), s, r);
    const float q2 = e4m3_quotient(bf16lo_to_f32(b), s, r);
    const float q3 = e4m3_quotient(bf16hi_to_f32(b), s, r);
    return static_cast<uint32_t>(f32x2_to_e4m3x2(q0, q1)) |
           (static_cast<uint32_t>(f32x2_to_e4m3x2(q2, q3)) << 16);
}

}  // namespace pkv
