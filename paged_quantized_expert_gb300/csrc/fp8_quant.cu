// fp8_quant.cu -- rows and weights to E4M3 codes with one fp32 scale for each
// 128 values (rows) or 128 x 128 values (weights).
//
// s = max|x| / 448, code = RNE_e4m3(x / s). A block of a row is sixteen lanes of
// eight values: one load of 16 bytes, a maximum over the lanes, eight quotients.
// Bound by memory, two bytes read and one written a value, and by issue close behind: 16384 x 2560 24 us, 5.3 TB/s; 64 x 2560 1.9
// us, a launch and a load. (Four blocks of sixteen lanes at a time: loads in flight, and fewer exchanges for four maxima
// together than one by one; 28 us with a maximum and a scale for each by itself, 45 with a division for each value.)
#include "fp8_codes.cuh"
#include "pqe_common.cuh"

namespace pqe {
namespace fp8 {

constexpr int BLOCK = 128;

struct RowArgs {
    const uint16_t *x;
    int64_t x_stride;
    int T, H;
    uint32_t blocks, part;  // blocks a row, and 2^24 / blocks rounded up
    uint8_t *q;
    float *scale;
};

// A CTA takes 64 blocks in a row (of one row of x after the other), four of each sixteen lanes, all loads first. Sixty-four times
// `blocks` of them are 64 rows, so CTA n starts n / blocks * 64 rows down, and what is left is
// below 64 * blocks <= 2^14 blocks: the product with the reciprocal, high by less than 2^-10 then, gives the same whole part as
// the division by up to 256.
constexpr int ROW_THREADS = 256, EACH = 4, GROUPS = ROW_THREADS / 16, TAKEN = GROUPS * EACH;
__global__ void __launch_bounds__(ROW_THREADS) quantize_rows_kernel(const RowArgs a) {
    const int lane = threadIdx.x & 15;
    const uint32_t whole = blockIdx.x / a.blocks, b0 = (blockIdx.x - whole * a.blocks) * TAKEN + (threadIdx.x >> 4);
    const int64_t row0 = (int64_t)whole * TAKEN;
    uint4 x[EACH];
    bool on[EACH];
    int64_t to[EACH];
    pdl_acquire();
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
        const uint32_t b = b0 + j * GROUPS, down = (uint32_t)(((uint64_t)b * a.part) >> 24);
        const int i = (int)(b - down * a.blocks) * BLOCK + lane * 8;
        on[j] = row0 + down < a.T && i < a.H;
        to[j] = (row0 + down) * a.H + i;
        x[j] = make_uint4(0, 0, 0, 0);
        if (on[j]) x[j] = *reinterpret_cast<const uint4 *>(a.x + (row0 + down) * a.x_stride + i);
    }
    uint32_t t[EACH];
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
        float f[8];
        unpack8(x[j], f);
        t[j] = top8(f);
    }
    float s, inv;
    block_scale(block_tops(t), s, inv);
    const int64_t u = row0 * a.blocks + b0 + lane * GROUPS;
    if (lane < EACH && u < (int64_t)a.T * a.blocks) a.scale[u] = s;
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
        const float sj = __shfl_sync(0xffffffffu, s, j, 16), ij = __shfl_sync(0xffffffffu, inv, j, 16);
        float f[8];
        unpack8(x[j], f);
        if (on[j]) *reinterpret_cast<uint2 *>(a.q + to[j]) = codes8_block(f, sj, ij);
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
    const fp8::RowArgs a{static_cast<const uint16_t *>(x), x_stride, T, H, (uint32_t)blocks, ((1u << 24) + blocks - 1) / blocks, q, scale};
    const int64_t ctas = ((int64_t)T * blocks + fp8::TAKEN - 1) / fp8::TAKEN;
    PQE_CHECK_ARG(ctas <= INT32_MAX);
    return launch_pdl(fp8::quantize_rows_kernel, dim3((unsigned)ctas), dim3(fp8::ROW_THREADS), 0, as_stream(stream), a);
}

int pqe_quantize_fp8_blocks(const float *w, int rows, int cols, uint8_t *q, float *scale, void *stream) {
    PQE_CHECK_ARG(w && q && scale && rows >= 1 && cols >= 1 && aligned(w, 4) && aligned(scale, 4));
    const int64_t rb = ((int64_t)rows + fp8::BLOCK - 1) / fp8::BLOCK, cb = ((int64_t)cols + fp8::BLOCK - 1) / fp8::BLOCK;
    PQE_CHECK_ARG(rb <= 65535 && cols <= INT32_MAX - (fp8::BLOCK - 1));  // the last tile's columns are ints too
    return launch_pdl(fp8::quantize_tiles_kernel, dim3((unsigned)cb, (unsigned)rb), dim3(256), 0, as_stream(stream), w, rows,
                      cols, q, scale);
}

}  // extern "C"
