// E4M3 quantization shared by the FP8 appends.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

// E4M3 codes of correctly rounded float32 quotients x / s (s > 0) without a
// division, r = the correctly rounded reciprocal of s.
//
// q0 = RN(x * r) is off x / s by up to 1.5 ulp: half an ulp of the product's
// rounding, up to one from r's (2^-24 relative).  One correction step, the final
// step of an FMA division (P. Markstein, "Computation of elementary functions on
// the IBM RISC System/6000 processor", IBM J. Res. Dev. 34(1), 1990), brings the
// quotient to its rounding but for rare last bits: e = x - s * q0 in one fused
// multiply-add is exact or, at 25 bits, off by 2^-24 relative, and e * r by as
// much again, so that q0 + e * r, before its rounding, is off x / s by at most
// 1.5 ulp * 2^-23 = 3 * 2^-24 ulp.  The E4M3 code can differ from the quotient's
// only where x / s lies that close to the rounding boundary beside a midpoint
// between two codes; the significands of x and s for which it does are few, and
// each of them was tried and gives the quotient's code (the CPU tests do it, for
// any float32 x, beside every bf16 x at hundreds of scales; the GPU tests compare
// with the oracle's codes).  The step is taken where the last ulp can change the
// code, 2^-11 <= |q0| <= 512: below, the code is a zero of x's sign; above, E4M3
// saturates (448); NaN stays NaN.  All this for scales of 2^-92 to 2^126, where
// the last bits of e and r are normal.
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
