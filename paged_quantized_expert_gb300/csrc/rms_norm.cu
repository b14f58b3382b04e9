// rms_norm.cu -- residual addition, RMS norm, and the result in E4M3 codes
// with scales.
//
// h = x + r, y = h * rsqrt(mean h^2 + eps) * w, codes of y. A row is read once
// and stays in registers through the sum of squares, the amax and the
// quantisation, all in fp32; the codes are made from the unrounded y.
#include "pqe_common.cuh"

namespace pqe {
namespace norm {

struct Args {
    const uint16_t *x, *r, *w;
    int64_t x_stride, r_stride;
    uint16_t *sum_out, *y_out;
    uint8_t *q;
    void *q_scale;
    int H, fmt;
    float eps;
    float c, mean;  // a power of two near 1 / sqrt(H), and 1 / (c * c * H)
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

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

// One CTA per row; thread i holds the vectors of eight values i, i + blockDim, ...
template <int V>
__global__ void __launch_bounds__(512) add_rms_norm_kernel(const Args a) {
    __shared__ float part_sum[16];
    __shared__ uint32_t part_max[16];
    const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int nv = a.H / 8;
    float h[V][8];
    float ss = 0.f;
    pdl_acquire();
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = threadIdx.x + j * blockDim.x;
        if (i >= nv) break;
        unpack8(reinterpret_cast<const uint4 *>(a.x + row * a.x_stride)[i], h[j]);
        if (a.r) {
            float f[8];
            unpack8(reinterpret_cast<const uint4 *>(a.r + row * a.r_stride)[i], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[j][e] += f[e];
        }
        if (a.sum_out)
            reinterpret_cast<uint4 *>(a.sum_out + (size_t)row * a.H)[i] =
                make_uint4(pack_bf16(h[j][0], h[j][1]), pack_bf16(h[j][2], h[j][3]), pack_bf16(h[j][4], h[j][5]),
                           pack_bf16(h[j][6], h[j][7]));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float u = h[j][e] * a.c;  // the sum overflows only where the mean does
            ss = fmaf(u, u, ss);
        }
    }
    ss = warp_sum(ss);
    if (lane == 0) part_sum[warp] = ss;
    __syncthreads();
    ss = 0.f;
    for (int i = 0; i < nw; ++i) ss += part_sum[i];
    const float inv = rsqrtf(fmaf(ss, a.mean, a.eps));
    uint32_t top = 0;  // of the row
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = threadIdx.x + j * blockDim.x;
        uint32_t t = 0;
        if (i < nv) {
            float w[8];
            unpack8(reinterpret_cast<const uint4 *>(a.w)[i], w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[j][e] = h[j][e] * inv * w[e];
                t = max(t, abs_bits(h[j][e]));
            }
            if (a.y_out)
                reinterpret_cast<uint4 *>(a.y_out + (size_t)row * a.H)[i] =
                    make_uint4(pack_bf16(h[j][0], h[j][1]), pack_bf16(h[j][2], h[j][3]), pack_bf16(h[j][4], h[j][5]),
                               pack_bf16(h[j][6], h[j][7]));
        }
        top = max(top, t);
        if (a.q && a.fmt == PQE_Q8_MX) {
            // 32 values lie in four neighbouring lanes (H % 32 == 0: all four hold values, or none)
            t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
            t = max(t, __shfl_xor_sync(0xffffffffu, t, 2));
            if (i < nv) {
                const bool bad = t >= 0x7F800000u;
                const uint32_t e8 = (uint32_t)max((int)(t >> 23) - 8, 0);
                const float s = bad ? __uint_as_float(0x7FC00000u) : __uint_as_float((254u - e8) << 23);
                uint32_t o[2];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    o[e] = (uint32_t)f32x2_to_e4m3x2(h[j][4 * e] * s, h[j][4 * e + 1] * s) |
                           (uint32_t)f32x2_to_e4m3x2(h[j][4 * e + 2] * s, h[j][4 * e + 3] * s) << 16;
                reinterpret_cast<uint2 *>(a.q + (size_t)row * a.H)[i] = make_uint2(o[0], o[1]);
                if (i % 4 == 0)
                    static_cast<uint8_t *>(a.q_scale)[(size_t)row * (a.H / 32) + i / 4] = bad ? 255 : (uint8_t)e8;
            }
        }
    }
    if (!a.q || a.fmt != PQE_Q8_ROW) return;
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) part_max[warp] = top;
    __syncthreads();
    top = 0;
    for (int i = 0; i < nw; ++i) top = max(top, part_max[i]);
    const float s = top > 0x7F800000u ? __uint_as_float(0x7FC00000u) : top == 0 ? 1.f : __uint_as_float(top) / 448.f;
    if (threadIdx.x == 0) static_cast<float *>(a.q_scale)[row] = s;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = threadIdx.x + j * blockDim.x;
        if (i >= nv) break;
        uint32_t o[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            o[e] = (uint32_t)f32x2_to_e4m3x2(h[j][4 * e] / s, h[j][4 * e + 1] / s) |
                   (uint32_t)f32x2_to_e4m3x2(h[j][4 * e + 2] / s, h[j][4 * e + 3] / s) << 16;
        reinterpret_cast<uint2 *>(a.q + (size_t)row * a.H)[i] = make_uint2(o[0], o[1]);
    }
}

}  // namespace norm
}  // namespace pqe

using namespace pqe;

extern "C" {

int add_rms_norm(const void *x, int64_t x_stride, const void *residual, int64_t r_stride, const void *weight,
                 float eps, int T, int H, void *sum_out, void *y_out, uint8_t *q, void *q_scale, int q_fmt,
                 void *stream) {
    PQE_CHECK_ARG(T >= 0 && H >= 32 && H <= 16384 && H % 32 == 0 && eps >= 0.f);
    if (T == 0) return PQE_OK;
    PQE_CHECK_ARG(x && weight && (sum_out || y_out || q) && x_stride >= H && x_stride % 8 == 0);
    PQE_CHECK_ARG(!residual || (r_stride >= H && r_stride % 8 == 0));
    PQE_CHECK_ARG(aligned(x, 16) && aligned(residual, 16) && aligned(weight, 16) && aligned(sum_out, 16) &&
                  aligned(y_out, 16) && aligned(q, 8));
    PQE_CHECK_ARG(!q || (q_scale && (q_fmt == PQE_Q8_MX || (q_fmt == PQE_Q8_ROW && aligned(q_scale, 4)))));
    float c = 1.f;
    while (c * c * (float)H > 1.f) c *= 0.5f;
    const norm::Args a{static_cast<const uint16_t *>(x), static_cast<const uint16_t *>(residual),
                       static_cast<const uint16_t *>(weight), x_stride, r_stride, static_cast<uint16_t *>(sum_out),
                       static_cast<uint16_t *>(y_out), q, q_scale, H, q_fmt, eps, c, 1.f / (c * c * (float)H)};
    const int nv = H / 8;
    // the fewest vectors a thread that 512 threads hold the row with
    const int V = nv <= 512 ? 1 : nv <= 1024 ? 2 : 4;
    const int threads = ((nv + V - 1) / V + 31) / 32 * 32;
    auto kern = V == 1 ? norm::add_rms_norm_kernel<1> : V == 2 ? norm::add_rms_norm_kernel<2> : norm::add_rms_norm_kernel<4>;
    return launch_pdl(kern, dim3((unsigned)T), dim3((unsigned)threads), 0, as_stream(stream), a);
}

}  // extern "C"
