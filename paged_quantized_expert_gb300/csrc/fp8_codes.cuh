// fp8_codes.cuh -- E4M3 codes of fp32 values under one scale (internal): what
// the norm and the block quantiser share.
#pragma once

#include "f32x2.cuh"
#include "pqe_common.cuh"

namespace pqe {
namespace fp8 {

// eight bf16 values to fp32
__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// bits of |f|: they order as the values do, with NaN above infinity
__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

// the scale of values whose largest |.| has these bits: amax / 448; 1 for zeros, or where fp32 does not hold it
__device__ __forceinline__ float scale_of(uint32_t top) {
    const float s = top > 0x7F800000u ? __uint_as_float(0x7FC00000u) : __uint_as_float(top) / 448.f;
    return s == 0.f ? 1.f : s;
}

// eight codes, RNE_e4m3(f / s) saturating at 448
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float s) {
    uint32_t o[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
        o[e] = (uint32_t)f32x2_to_e4m3x2(f[4 * e] / s, f[4 * e + 1] / s) |
               (uint32_t)f32x2_to_e4m3x2(f[4 * e + 2] / s, f[4 * e + 3] / s) << 16;
    return make_uint2(o[0], o[1]);
}

// The same scale and codes with one reciprocal for all eight; a quotient is 8 to 10 instructions. With r = f / s to within a unit
// or so, from a rounded 1 / s, the quotient is r + (f - r s) / s, the remainder exact in an fma (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990: correctly rounded where nothing leaves the normal range, which
// values far from 1 could).
__device__ __forceinline__ uint2 codes8_block(const float (&f)[8], uint32_t top, float &s) {
    using namespace f32x2;
    const float amax = __uint_as_float(top);
    if (!(amax > 0x1p-100f && amax < 0x1p100f)) {
        s = scale_of(top);
        return codes8(f, s);
    }
    s = amax * (1.f / 448);
    s = fmaf(fmaf(-s, 448.f, amax), 1.f / 448, s);
    const uint64_t inv = pair(__frcp_rn(s)), minus = pair(-s);
    uint16_t o[4];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const uint64_t x = pair(f[e], f[e + 1]), r = mul2(x, inv);
        const float2 q = unpair(fma2(fma2(r, minus, x), inv, r));
        o[e / 2] = f32x2_to_e4m3x2(q.x, q.y);
    }
    return make_uint2((uint32_t)o[0] | (uint32_t)o[1] << 16, (uint32_t)o[2] | (uint32_t)o[3] << 16);
}

}  // namespace fp8
}  // namespace pqe
