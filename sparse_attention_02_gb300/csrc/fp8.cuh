// E4M3 helpers shared by the kernels that write FP8 codes.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "f32x2.cuh"

namespace dsa {

// Smallest power of two not below a positive finite fp32 r (exact, bit level).
__device__ __forceinline__ float pow2_ceil(float r)
{
    const uint32_t u = __float_as_uint(r);
    const uint32_t ex = u & 0x7F800000u, man = u & 0x007FFFFFu;
    if (ex != 0u) // normal: r itself when the mantissa is zero, else the next exponent
        return man == 0u ? r : __uint_as_float(ex + 0x00800000u);
    // subnormal r = man * 2^-149: the next power of two of man, in the same units
    const uint32_t p = (man & (man - 1u)) == 0u ? man : (1u << (32 - __clz(man - 1u)));
    return __uint_as_float(p);
}

// Two fp32 -> two E4M3 codes (round to nearest even, saturating), lo in byte 0.
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Division of many values by one scale, each quotient correctly rounded (the
// same bits as y / s): with inv = RN(1 / s), q0 = RN(y inv) and the remainder
// y - q0 s, exact in an fma, RN(q0 + remainder inv) is RN(y / s) (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990), as long as nothing under- or overflows on the way; scales so small
// that 1 / s might, divide.  Three operations for the ten or so of a division,
// which bounded the norm's FP8 output (115 us for 92 with a bare product at
// 8191 x 8192).
struct ScaleDivider {
    float s, inv;
    bool plain;
    __device__ __forceinline__ explicit ScaleDivider(float scale) : s(scale), inv(1.f / scale), plain(!(scale > 1e-30f)) {}
    __device__ __forceinline__ float operator()(float y, bool in_range = true) const
    {
        if (plain || !in_range)
            return y / s;
        const float q = y * inv;
        return fmaf(fmaf(-q, s, y), inv, q);
    }
    __device__ __forceinline__ uint16_t codes(float lo, float hi) const // of two quotients
    {
        if (plain)
            return e4m3x2(lo / s, hi / s);
        const F2 y(lo, hi), q = y * F2(inv);
        fma2(fma2(q, F2(-s), y), F2(inv), q).get(lo, hi);
        return e4m3x2(lo, hi);
    }
};

// Scale of values whose largest magnitude is amax: amax / 448, or the smallest
// power of two not below it (mode 1); 1 for zeros and where the quotient is
// below the smallest fp32.
__device__ __forceinline__ float fp8_scale(float amax, int mode)
{
    const float ratio = ScaleDivider(448.f)(amax, amax > 1e-30f && amax < 1e38f);
    if (!(ratio > 0.f))
        return 1.f;
    return mode == 0 ? ratio : pow2_ceil(ratio);
}

// Four values as E4M3 codes over a scale, the first in byte 0.
__device__ __forceinline__ uint32_t e4m3x4(const ScaleDivider &d, float a, float b, float c, float e)
{
    return d.codes(a, b) | ((uint32_t)d.codes(c, e) << 16);
}

} // namespace dsa
