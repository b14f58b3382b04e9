// fp8_matmul.cu -- fp8_block_matmul: E4M3 codes times E4M3 codes, an fp32 scale
// for each 128 values of a row of x and for each 128 x 128 tile of W.
//
// out[m, n] = sum_b xs[m, b] ws[n / 128, b] (sum over the block's k of x w): the
// block's products are summed in fp32 by themselves, then scaled into the result.
// The simplest form: a 64 x 64 tile a CTA, 4 x 4 of it a thread, codes expanded
// to fp32 in shared memory 16 columns at a time.
#include "pqe_common.cuh"

namespace pqe {
namespace fp8mm {

struct Args {
    const uint8_t *x, *w;
    const float *xs, *ws;
    void *out;
    int64_t x_stride, out_stride;
    int M, N, K, kb, fp32;
};

constexpr int TILE = 64, CHUNK = 16;

__global__ void __launch_bounds__(256) matmul_kernel(const Args a) {
    __shared__ float sx[TILE][CHUNK + 1], sw[TILE][CHUNK + 1];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t m0 = (int64_t)blockIdx.y * TILE, n0 = (int64_t)blockIdx.x * TILE;
    const int lr = threadIdx.x >> 2, lc = (threadIdx.x & 3) * 4;  // the four codes that a thread expands
    pdl_acquire();
    float acc[4][4] = {};
    for (int b = 0; b < a.kb; ++b) {
        float part[4][4] = {};
        for (int k0 = b * 128; k0 < min(b * 128 + 128, a.K); k0 += CHUNK) {
            uint32_t cx = 0, cw = 0;
            if (m0 + lr < a.M) cx = *reinterpret_cast<const uint32_t *>(a.x + (m0 + lr) * a.x_stride + k0 + lc);
            if (n0 + lr < a.N) cw = *reinterpret_cast<const uint32_t *>(a.w + (n0 + lr) * a.K + k0 + lc);
            __syncthreads();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 fx = e4m3x2_to_f32x2((uint16_t)(cx >> 16 * h)), fw = e4m3x2_to_f32x2((uint16_t)(cw >> 16 * h));
                sx[lr][lc + 2 * h] = fx.x, sx[lr][lc + 2 * h + 1] = fx.y;
                sw[lr][lc + 2 * h] = fw.x, sw[lr][lc + 2 * h + 1] = fw.y;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < CHUNK; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) part[i][j] = fmaf(sx[ty + 16 * i][k], sw[tx + 16 * j][k], part[i][j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + ty + 16 * i;
            const float s = m < a.M ? a.xs[m * a.kb + b] * a.ws[n0 / 128 * a.kb + b] : 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(part[i][j], s, acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m >= a.M || n >= a.N) continue;
            if (a.fp32) static_cast<float *>(a.out)[m * a.out_stride + n] = acc[i][j];
            else static_cast<uint16_t *>(a.out)[m * a.out_stride + n] = f32_to_bf16_rn(acc[i][j]);
        }
}

}  // namespace fp8mm
}  // namespace pqe

using namespace pqe;

extern "C" {

int fp8_block_matmul(const uint8_t *x, int64_t x_stride, const float *x_scale, const uint8_t *w, const float *w_scale,
                     int M, int N, int K, void *out, int64_t out_stride, int out_fp32, int32_t *status, void *stream) {
    PQE_CHECK_ARG(M >= 0 && N >= 1 && N <= 1 << 22 && K >= 16 && K <= 32768 && K % 16 == 0);
    if (M == 0) return PQE_OK;
    PQE_CHECK_ARG(x && x_scale && w && w_scale && out && status && x_stride >= K && x_stride % 16 == 0 && out_stride >= N);
    PQE_CHECK_ARG(aligned(x, 16) && aligned(w, 16) && aligned(x_scale, 4) && aligned(w_scale, 4) && aligned(status, 4) &&
                  aligned(out, out_fp32 ? 4 : 2));
    const fp8mm::Args a{x, w, x_scale, w_scale, out, x_stride, out_stride, M, N, K, (K + 127) / 128, out_fp32};
    const int64_t mt = ((int64_t)M + fp8mm::TILE - 1) / fp8mm::TILE;
    PQE_CHECK_ARG(mt <= 65535);
    return launch_pdl(fp8mm::matmul_kernel, dim3((unsigned)((N + fp8mm::TILE - 1) / fp8mm::TILE), (unsigned)mt), dim3(256), 0,
                      as_stream(stream), a);
}

}  // extern "C"
