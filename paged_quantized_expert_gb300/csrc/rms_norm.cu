// rms_norm.cu -- residual addition, RMS norm, and the result in E4M3 codes
// with scales.
//
// h = x + r, y = h * rsqrt(mean h^2 + eps) * w, codes of y. A row is read once
// and stays in registers through the sum of squares, the amax and the
// quantisation, all in fp32; the codes are made from the unrounded y. (The sum of
// squares is of c h, c a power of two near 1 / sqrt(H), so that it overflows where
// the mean does and not before.)
//
// A warp a row where there are many rows of up to 2560 values, else a CTA a row;
// bound by memory then (16384 rows of 2560, bf16 sum and codes out: 49.5 us, 5.96
// TB/s), by the latency of one load, two reductions and a store where there are
// few (64 rows of 2048: 2.4 us).
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

// What a thread (of a warp or a CTA that shares a row) does with its V vectors of eight values, vector j at index
// first + j * step of the row.
template <int V>
struct Part {
    float h[V][8];
    uint4 w[V];

    // h = x + r, sum_out; returns the thread's sum of (c h)^2. The weights are asked for along with the row.
    __device__ __forceinline__ float load(const Args &a, int row, int first, int step) {
        const int nv = a.H / 8;
        uint4 x[V], r[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = first + j * step;
            if (i >= nv) break;
            x[j] = reinterpret_cast<const uint4 *>(a.x + row * a.x_stride)[i];
            if (a.r) r[j] = reinterpret_cast<const uint4 *>(a.r + row * a.r_stride)[i];
            w[j] = reinterpret_cast<const uint4 *>(a.w)[i];
        }
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = first + j * step;
            if (i >= nv) break;
            unpack8(x[j], h[j]);
            if (a.r) {
                float f[8];
                unpack8(r[j], f);
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
        return ss;
    }

    // y, y_out, and the codes with a scale for each 32 values; returns the thread's largest |y| (bits). Threads of
    // neighbouring indices are neighbouring lanes, and all 32 lanes are here.
    __device__ __forceinline__ uint32_t scale(const Args &a, int row, int first, int step, float inv) {
        const int nv = a.H / 8;
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = first + j * step;
            uint32_t t = 0;
            if (i < nv) {
                float f[8];
                unpack8(w[j], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    h[j][e] = h[j][e] * inv * f[e];
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
        return top;
    }

    // the codes with one scale for the row
    __device__ __forceinline__ void codes(const Args &a, int row, int first, int step, uint32_t top) {
        const int nv = a.H / 8;
        float s = top > 0x7F800000u ? __uint_as_float(0x7FC00000u) : __uint_as_float(top) / 448.f;
        if (s == 0.f) s = 1.f;  // a row of zeros, or one so small that fp32 does not hold its scale
        if (first == 0) static_cast<float *>(a.q_scale)[row] = s;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = first + j * step;
            if (i >= nv) break;
            uint32_t o[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                o[e] = (uint32_t)f32x2_to_e4m3x2(h[j][4 * e] / s, h[j][4 * e + 1] / s) |
                       (uint32_t)f32x2_to_e4m3x2(h[j][4 * e + 2] / s, h[j][4 * e + 3] / s) << 16;
            reinterpret_cast<uint2 *>(a.q + (size_t)row * a.H)[i] = make_uint2(o[0], o[1]);
        }
    }
};

// A CTA per row: the most loads in flight where rows are few, or long.
template <int V>
__global__ void __launch_bounds__(512) norm_cta_kernel(const Args a) {
    __shared__ float part_sum[16];
    __shared__ uint32_t part_max[16];
    const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    Part<V> p;
    pdl_acquire();
    float ss = warp_sum(p.load(a, row, threadIdx.x, blockDim.x));
    if (lane == 0) part_sum[warp] = ss;
    __syncthreads();
    ss = 0.f;
    for (int i = 0; i < nw; ++i) ss += part_sum[i];
    uint32_t top = p.scale(a, row, threadIdx.x, blockDim.x, rsqrtf(fmaf(ss, a.mean, a.eps)));
    if (!a.q || a.fmt != PQE_Q8_ROW) return;
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) part_max[warp] = top;
    __syncthreads();
    top = 0;
    for (int i = 0; i < nw; ++i) top = max(top, part_max[i]);
    p.codes(a, row, threadIdx.x, blockDim.x, top);
}

// A warp per row: no barrier, and as many rows in flight as registers hold.
constexpr int ROW_WARPS = 4;
template <int V>
__global__ void __launch_bounds__(32 * ROW_WARPS) norm_warp_kernel(const Args a, int T) {
    const int row = blockIdx.x * ROW_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    pdl_acquire();
    if (row >= T) return;
    Part<V> p;
    const float ss = warp_sum(p.load(a, row, lane, 32));
    const uint32_t top = p.scale(a, row, lane, 32, rsqrtf(fmaf(ss, a.mean, a.eps)));
    if (a.q && a.fmt == PQE_Q8_ROW) p.codes(a, row, lane, 32, __reduce_max_sync(0xffffffffu, top));
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
    cudaStream_t st = as_stream(stream);
    int dev = 0, sms = 0;
    const int rc = device_info(dev, sms);
    if (rc != PQE_OK) return rc;
    // Rows that a warp's registers hold, and enough of them for eight warps an SM.
    if (nv <= 32 * 10 && T >= 8 * sms) {
        auto kern = nv <= 32 ? norm::norm_warp_kernel<1> : nv <= 64 ? norm::norm_warp_kernel<2>
                    : nv <= 128 ? norm::norm_warp_kernel<4> : nv <= 256 ? norm::norm_warp_kernel<8>
                                                                         : norm::norm_warp_kernel<10>;
        return launch_pdl(kern, dim3((unsigned)((T + norm::ROW_WARPS - 1) / norm::ROW_WARPS)), dim3(32 * norm::ROW_WARPS), 0,
                          st, a, T);
    }
    // the fewest vectors a thread that 512 threads hold the row with
    const int V = nv <= 512 ? 1 : nv <= 1024 ? 2 : 4;
    const int threads = ((nv + V - 1) / V + 31) / 32 * 32;
    auto kern = V == 1 ? norm::norm_cta_kernel<1> : V == 2 ? norm::norm_cta_kernel<2> : norm::norm_cta_kernel<4>;
    return launch_pdl(kern, dim3((unsigned)T), dim3((unsigned)threads), 0, st, a);
}

}  // extern "C"
