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

// the largest of eight |.|, NaN if one is NaN, as bits
__device__ __forceinline__ uint32_t top8(const float (&f)[8]) {
    float m = f[7];
#pragma unroll
    for (int e = 0; e < 6; e += 2) asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(f[e]), "f"(f[e + 1]));
    asm("max.NaN.abs.f32 %0, %0, %1, %1;" : "+f"(m) : "f"(f[6]));
    return __float_as_uint(m);
}

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

// Blocks of 128 values lie in sixteen neighbouring lanes, V vectors of eight in a lane. Sixteen lanes bring V maxima together:
// in the first step a lane keeps the even or the odd vectors, by bit 0 of its number, and sends the others, and so on. Lane j (of
// sixteen) returns the maximum of vector j: about V + 4 exchanges for all vectors, V * 4 one vector after the other.
template <int V>
__device__ __forceinline__ uint32_t block_tops(uint32_t (&t)[V]) {
    static_assert(V >= 1 && V <= 16);
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int bit = 1, n = V; bit < 16; bit *= 2, n = (n + 1) / 2) {
        if (n == 1) {
            t[0] = max(t[0], __shfl_xor_sync(0xffffffffu, t[0], bit));
            continue;
        }
#pragma unroll
        for (int k = 0; k < (n + 1) / 2; ++k) {
            const uint32_t even = t[2 * k], odd = 2 * k + 1 < n ? t[2 * k + 1] : 0u;
            const uint32_t other = __shfl_xor_sync(0xffffffffu, lane & bit ? even : odd, bit);
            t[k] = max(lane & bit ? odd : even, other);
        }
    }
    return t[0];
}

// A block's scale, and its reciprocal for codes8_block (0: the block is one of those that take a division for each value).
__device__ __forceinline__ void block_scale(uint32_t top, float &s, float &inv) {
    const float amax = __uint_as_float(top);
    if (amax > 0x1p-100f && amax < 0x1p100f) {
        s = amax * (1.f / 448);
        s = fmaf(fmaf(-s, 448.f, amax), 1.f / 448, s);
        inv = __frcp_rn(s);
    } else {
        s = scale_of(top);
        inv = 0.f;
    }
}

// The same codes as codes8 with one reciprocal for the block; a quotient is 8 to 10 instructions. With r = f / s to within a unit
// or so, from a rounded 1 / s, the quotient is r + (f - r s) / s, the remainder exact in an fma (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990: correctly rounded where nothing leaves the normal range, which
// values far from 1 could).
__device__ __forceinline__ uint2 codes8_block(const float (&f)[8], float s, float inv) {
    using namespace f32x2;
    if (inv == 0.f) return codes8(f, s);
    const uint64_t inv2 = pair(inv), minus = pair(-s);
    uint16_t o[4];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const uint64_t x = pair(f[e], f[e + 1]), r = mul2(x, inv2);
        const float2 q = unpair(fma2(fma2(r, minus, x), inv2, r));
        o[e / 2] = f32x2_to_e4m3x2(q.x, q.y);
    }
    return make_uint2((uint32_t)o[0] | (uint32_t)o[1] << 16, (uint32_t)o[2] | (uint32_t)o[3] << 16);
}

}  // namespace fp8
}  // namespace pqe
