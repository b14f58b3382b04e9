// fp8_quant.cu -- rows and weights to E4M3 codes with one fp32 scale for each
// 128 values (rows) or 128 x 128 values (weights).
//
// s = max|x| / 448, code = RNE_e4m3(x / s). A block of a row is sixteen lanes of
// eight values: one load of 16 bytes, a maximum over the lanes, eight quotients.
// Bound by memory: two bytes read and one written a value.
#include "fp8_codes.cuh"
#include "pqe_common.cuh"

namespace pqe {
namespace fp8 {

constexpr int BLOCK = 128;

struct RowArgs {
    const uint16_t *x;
    int64_t x_stride;
    int T, H, blocks;
    uint8_t *q;
    float *scale;
};

// A CTA takes 64 blocks in a row (of one row of x after the other), four of each sixteen lanes, all loads first.
constexpr int ROW_THREADS = 256, EACH = 4, TAKEN = ROW_THREADS / 16 * EACH;
__global__ void __launch_bounds__(ROW_THREADS) quantize_rows_kernel(const RowArgs a) {
    const int lane = threadIdx.x & 15;
    const int64_t units = (int64_t)a.T * a.blocks, u0 = (int64_t)blockIdx.x * TAKEN, row0 = u0 / a.blocks;
    const uint32_t b0 = (uint32_t)(u0 - row0 * a.blocks) + (threadIdx.x >> 4);
    pdl_acquire();
    uint4 x[EACH];
    bool on[EACH];
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
        const uint32_t b = b0 + j * (ROW_THREADS / 16), down = b / (uint32_t)a.blocks;
        const int i = (int)(b - down * a.blocks) * BLOCK + lane * 8;
        on[j] = row0 + down < a.T && i < a.H;
        x[j] = make_uint4(0, 0, 0, 0);
        if (on[j]) x[j] = *reinterpret_cast<const uint4 *>(a.x + (row0 + down) * a.x_stride + i);
    }
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
        const int64_t u = u0 + (threadIdx.x >> 4) + j * (ROW_THREADS / 16);
        if (u0 + (threadIdx.x >> 5) * 2 + j * (ROW_THREADS / 16) >= units) break;  // the whole warp: the shuffles need all lanes
        float f[8];
        unpack8(x[j], f);
        uint32_t t = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) t = max(t, abs_bits(f[e]));
#pragma unroll
        for (int o = 1; o < 16; o *= 2) t = max(t, __shfl_xor_sync(0xffffffffu, t, o));
        if (!on[j]) continue;
        float s;
        const uint32_t b = b0 + j * (ROW_THREADS / 16), down = b / (uint32_t)a.blocks;
        *reinterpret_cast<uint2 *>(a.q + (row0 + down) * a.H + (b - down * a.blocks) * BLOCK + lane * 8) = codes8_block(f, t, s);
        if (lane == 0) a.scale[u] = s;
    }
}

// A CTA for each tile of weights.
__global__ void __launch_bounds__(256) quantize_tiles_kernel(const float *w, int rows, int cols, uint8_t *q, float *scale) {
    __shared__ uint32_t part[8];
    const int r0 = blockIdx.y * BLOCK, c = blockIdx.x * BLOCK + (threadIdx.x & 127);
    pdl_acquire();
    uint32_t t = 0;
    for (int r = r0 + (threadIdx.x >> 7); r < min(r0 + BLOCK, rows); r += 2)
        if (c < cols) t = max(t, abs_bits(w[(size_t)r * cols + c]));
    t = __reduce_max_sync(0xffffffffu, t);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = t;
    __syncthreads();
    for (int i = 0; i < 8; ++i) t = max(t, part[i]);
    const float s = scale_of(t);
    if (threadIdx.x == 0) scale[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = s;
    for (int r = r0 + (threadIdx.x >> 7); r < min(r0 + BLOCK, rows); r += 2)
        if (c < cols) q[(size_t)r * cols + c] = (uint8_t)f32x2_to_e4m3x2(w[(size_t)r * cols + c] / s, 0.f);
}

}  // namespace fp8
}  // namespace pqe

using namespace pqe;

extern "C" {

int fp8_block_quantize(const void *x, int64_t x_stride, int T, int H, uint8_t *q, float *scale, void *stream) {
    PQE_CHECK_ARG(T >= 0 && H >= 16 && H <= 32768 && H % 16 == 0);
    if (T == 0) return PQE_OK;
    PQE_CHECK_ARG(x && q && scale && x_stride >= H && x_stride % 8 == 0);
    PQE_CHECK_ARG(aligned(x, 16) && aligned(q, 16) && aligned(scale, 4));
    const int blocks = (H + fp8::BLOCK - 1) / fp8::BLOCK;
    const fp8::RowArgs a{static_cast<const uint16_t *>(x), x_stride, T, H, blocks, q, scale};
    const int64_t ctas = ((int64_t)T * blocks + fp8::TAKEN - 1) / fp8::TAKEN;
    PQE_CHECK_ARG(ctas <= INT32_MAX);
    return launch_pdl(fp8::quantize_rows_kernel, dim3((unsigned)ctas), dim3(fp8::ROW_THREADS), 0, as_stream(stream), a);
}

int pqe_quantize_fp8_blocks(const float *w, int rows, int cols, uint8_t *q, float *scale, void *stream) {
    PQE_CHECK_ARG(w && q && scale && rows >= 1 && cols >= 1 && aligned(w, 4) && aligned(scale, 4));
    const int64_t rb = ((int64_t)rows + fp8::BLOCK - 1) / fp8::BLOCK, cb = ((int64_t)cols + fp8::BLOCK - 1) / fp8::BLOCK;
    PQE_CHECK_ARG(rb <= 65535);
    return launch_pdl(fp8::quantize_tiles_kernel, dim3((unsigned)cb, (unsigned)rb), dim3(256), 0, as_stream(stream), w, rows,
                      cols, q, scale);
}

}  // extern "C"
