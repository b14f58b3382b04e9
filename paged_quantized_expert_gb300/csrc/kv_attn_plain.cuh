// kv_attn_plain.cuh -- one query row over the 4-bit paged cache in fp32 throughout (internal).
//
// The attention kernels hold K and V (or the probabilities that meet them) in f16, relative to the largest scale that any of the
// rows of a tile sees. Where that is far above what one of those rows sees, the row's own values would be lost under a token that
// it does not see. Such tiles take this form instead: a warp per row, K, V and p as they are, nothing in common with other rows.
// 16 rows at once on an SM take some 9 us for every 32 tokens, waiting on loads; a model whose values lie within a few orders of
// magnitude of one another does not come here. (Two chunks of 2048 tokens over 5000 to 8192 with one token's V 2^40 above the others: 38 ms, without it 0.18; 32
// sequences of 5 tokens over 4000: 2.3 ms, 0.045; 8 prompts of 300 tokens whose first V is 2^40 below the others: 138 us, 32.)
#pragma once

#include "kv_attn.cuh"

namespace pqe {
namespace kv {

// 2^(x - 127) of an E8M0 byte, NaN for 255
__device__ __forceinline__ float scale_value(uint32_t x) {
    return __uint_as_float(x == 255u ? 0x7FC00000u : x == 0u ? 0x00400000u : x << 23);
}

// A row's sums over some tokens: m the largest exponent of two, l = sum p and o = sum p v with p = 2^(s - m), the lane's D / 32
// channels from lane * D / 32 on
template <int D>
struct PlainRow {
    float m, l, o[D / 32];
};

// The row at q over tokens [lo, hi) of a sequence, for a whole warp. scale: times log2(e).
template <int D>
__device__ __forceinline__ PlainRow<D> plain_row(const Cache &c, const int32_t *table, int head, const uint16_t *q, float scale,
                                                 int lo, int hi) {
    constexpr int E = D / 32, NB = D / 32;
    const int lane = threadIdx.x & 31, e0 = lane * E, mask = (1 << c.page_shift) - 1;
    PlainRow<D> r;
    r.m = -INFINITY;
    r.l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) r.o[e] = 0.f;
    bool finite = true;
#pragma unroll
    for (int e = 0; e < E; ++e) finite = finite && (q[e0 + e] & 0x7F80u) != 0x7F80u;
    finite = __all_sync(0xffffffffu, finite);
    for (int j0 = lo & ~31; j0 < hi; j0 += 32) {
        // a token a lane: its score
        const int j = j0 + lane;
        const int page = j >= lo && j < hi ? table[j >> c.page_shift] : -1;
        const bool in = page >= 0 && page < c.n_pages;
        const uint8_t *blk = block_of<D>(c, in ? page : 0, in ? j & mask : 0, head);
        float s = -INFINITY;
        if (in) {
            const int tok = j & 15;
            float part[NB] = {};
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int G = 0; G < NB; ++G) {
                    uint32_t h[4];
                    e2m1x8_to_f16(*reinterpret_cast<const uint32_t *>(blk + tok * (D / 2) + t * (D / 8) + 4 * G), h);
                    const uint4 u = *reinterpret_cast<const uint4 *>(q + 32 * G + 8 * t);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float2 k;
                        asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
                            : "=f"(k.x), "=f"(k.y)
                            : "r"(h[i]));
                        part[G] = fmaf(__uint_as_float(w[i] << 16), k.x, part[G]);
                        part[G] = fmaf(__uint_as_float(w[i] & 0xFFFF0000u), k.y, part[G]);
                    }
                }
            s = 0.f;
#pragma unroll
            for (int G = 0; G < NB; ++G) s = fmaf(part[G] * scale, scale_value(blk[k_scale<D>(tok, G)]), s);
            if (!finite) s = __uint_as_float(0x7FC00000u);
        }
        float now = fmaxf(r.m, s);
#pragma unroll
        for (int o = 16; o; o >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, o));
        const float base = now == -INFINITY ? 0.f : now, keep = exp2_approx(r.m - base), p = exp2_approx(s - base);
        r.m = now;
        r.l = fmaf(r.l, keep, p);
#pragma unroll
        for (int e = 0; e < E; ++e) r.o[e] *= keep;
        // its value, by all lanes
        const uint32_t there = __ballot_sync(0xffffffffu, in);
#pragma unroll 8
        for (int x = 0; x < 32; ++x) {
            const uint8_t *b = reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(blk), x));
            const float px = __shfl_sync(0xffffffffu, p, x);
            if (!(there >> x & 1)) continue;
            const int tok = (j0 + x) & 15;
            const float f = scale_value(b[v_scale<D>(tok, e0 / 32)]);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 v = e2m1x2_to_f32x2(b[v_code<D>(tok, e0 + e)]);
                r.o[e] = fmaf(px, v.x * f, r.o[e]);
                r.o[e + 1] = fmaf(px, v.y * f, r.o[e + 1]);
            }
        }
    }
    r.l = warp_sum(r.l);
    return r;
}

}  // namespace kv
}  // namespace pqe
