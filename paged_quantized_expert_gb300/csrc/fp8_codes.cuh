// fp8_codes.cuh -- E4M3 codes of fp32 values under one scale (internal): what
// the norm and the block quantiser share.
#pragma once

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

}  // namespace fp8
}  // namespace pqe
