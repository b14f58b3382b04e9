// fp8_matmul.cu -- fp8_block_matmul: argument checks, the choice of kernel, tensor maps.
//
// out[m, n] = sum_b xs[m, b] ws[n / 128, b] (sum over the block's k of x w). The scales change every 128 values of K, so each
// block is a product of its own in the tensor cores (exact products, fp32 sums), scaled and added outside them.
#include <atomic>

#include "fp8_matmul.cuh"

namespace pqe {
namespace fp8mm {

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                             const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeFn encode_fn() {
    static std::atomic<EncodeFn> fn{nullptr};
    EncodeFn f = fn.load(std::memory_order_acquire);
    if (!f) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn.store(f = reinterpret_cast<EncodeFn>(p), std::memory_order_release);
    }
    return f;
}

static bool encode(CUtensorMap *m, CUtensorMapDataType type, const void *base, uint64_t rows, uint64_t cols, uint64_t stride,
                   uint32_t box_rows, uint32_t box_cols, CUtensorMapSwizzle swizzle, CUtensorMapL2promotion promotion) {
    const EncodeFn f = encode_fn();
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {stride};
    const cuuint32_t box[2] = {box_cols, box_rows}, es[2] = {1, 1};
    return f && f(m, type, 2, const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promotion,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool map_codes(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols, uint64_t stride, uint32_t box_rows) {
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, rows, cols, stride, box_rows, BK, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

bool map_out(CUtensorMap *m, const Args &a, int cols) {
    const int size = a.fp32 ? 4 : 2;
    return encode(m, a.fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.out, (uint64_t)a.M, (uint64_t)cols,
                  (uint64_t)a.out_stride * size, 32, 64 / size, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

static std::atomic<int> g_kernel{0};      // pqe_test_set_matmul_kernel: tile << 16 | split, one word, so that no call sees parts of two
static std::atomic<int64_t> g_expiry{0};  // pqe_test_set_matmul_expiry: who << 32 | block

// whether out's rows lie as TMA needs them
static bool out_aligned(const Args &a) { return aligned(a.out, 16) && a.out_stride * (a.fp32 ? 4 : 2) % 16 == 0; }

// A store of a box that ends inside 16 bytes writes all of them, over what lies behind the row: where rows end so, only the boxes
// that lie wholly in them leave by TMA.
int tma_columns(const Args &a) {
    const int size = a.fp32 ? 4 : 2;
    return !out_aligned(a) ? 0 : (int64_t)a.N * size % 16 == 0 ? a.N : a.N / (64 / size) * (64 / size);
}

// Which kernel takes a call: the least of estimates in us, from measurements on one GB300 (K = 2048, bf16 out unless said).
//   few, 16 or 32 tokens a tile: 2.2 (2.3) to begin and end, 0.23 (0.29) a block of K and round of tiles; where SMs are left 2 to
//   8 CTAs share the blocks, for 0.8 (1 x 3584: 3.5 by four, 6.0 alone; 64 x 2048 x 2560: 5.0; 333 x 1003 x 1040 fp32: 5.4;
//   64 x 512 x 16384: 7.6 by eight, 41 alone)
//   many, 128 x 128 an SM: 2.7, 0.24 a block in a first round of tiles, 0.29 in several (128 x 3584: 7.0; 512 x 3584: 7.5)
//   many, 256 x 128 a pair: 3.2, 0.235, 0.27 (512 x 3584: 7.6; 4962 x 232 x 8112: 21; 29 with 256 x 256 and 26 to 30 with 128 x 128,
//   which takes it, the estimates being 0.2 apart)
//   many, 256 x 256 a pair: 4.1, 0.31, 0.44 (1024 x 3584: 10.0; the other two 12.1, 11.6. 4099 x 3584: 30; 35, 33.
//   16384 x 4096 x 2560: 120; 158, 146)
// and of no kernel less than the bytes at 6.2 TB/s (64 x 131072 fp32: 52 by 128 x 128 tiles, 55 by 32 tokens, 63, 66 by pairs;
// 16 x 131072: 44 by 16 tokens; 256 x 131072: 65, 70 by pairs, 100 by 128 x 128). The kernels for many rows store element by element
// where out's rows are not aligned to 16 bytes, 2 a round.
struct Choice {
    int rows, cols;  // few: tokens a tile, log2 of the CTAs that share one; many: 128 or 256 rows, columns
    double us;
};

static Choice least(const Call &c, int sms) {
    const int64_t M = c.a.M, N = c.a.N, kb = c.a.kb, tiles = (N + 127) / 128;
    const double bytes = ((double)M * c.K + (double)N * c.K + (double)M * N * (c.a.fp32 ? 4 : 2)) / 6.2e6;
    Choice best{0, 0, 1e30};
    auto offer = [&](int rows, int cols, double us) {
        us = (us > bytes ? us : bytes) + 0.1 * us;
        if (us < best.us) best = {rows, cols, us};
    };
    for (int tokens = 16; tokens <= 32; tokens *= 2) {
        const int64_t items = tiles * ((M + tokens - 1) / tokens);
        int log = 0;  // each CTA finishes four tokens at least
        while (tokens >> (log + 1) >= 4 && items << (log + 1) <= sms && kb >> (log + 1) >= 2) ++log;
        const int64_t rounds = ((items << log) + sms - 1) / sms, blocks = (kb + (1 << log) - 1) >> log;
        offer(tokens, log, (tokens == 16 ? 2.2 : 2.3) + (log ? 0.8 : 0) + (tokens == 16 ? 0.23 : 0.29) * rounds * blocks);
    }
    const double out = out_aligned(c.a) ? 0 : 2;
    auto rounds = [&](int64_t rows, int64_t cols, int64_t at_once) {
        return (double)(((M + rows - 1) / rows * ((N + cols - 1) / cols) + at_once - 1) / at_once);
    };
    const double ones = rounds(128, 128, sms), pairs = rounds(256, 128, sms / 2), wide = rounds(256, 256, sms / 2);
    offer(128, 128, 2.7 + ones * ((ones > 1 ? 0.29 : 0.24) * kb + out));
    offer(256, 128, 3.2 + pairs * ((pairs > 1 ? 0.27 : 0.235) * kb + out));
    offer(256, 256, 4.1 + wide * ((wide > 1 ? 0.44 : 0.31) * kb + 2 * out));
    return best;
}

static int run(const Call &c, int sms, cudaStream_t s) {
    const int kernel = g_kernel.load(std::memory_order_relaxed), tile = kernel >> 16, split = kernel & 0xFFFF;
    Choice use = least(c, sms);
    if (tile) {
        use = {tile, split, 0};
        if (tile < 128)
            while (use.cols && 1 << use.cols > c.a.kb) --use.cols;
    }
    return use.rows < 128 ? matmul_few(c, use.rows, use.cols, sms, s) : matmul_many(c, use.cols, use.rows / 128, sms, s);
}

}  // namespace fp8mm
}  // namespace pqe

using namespace pqe;

extern "C" {

int pqe_test_set_matmul_kernel(int tile, int split) {
    PQE_CHECK_ARG((tile == 0 && split == 0) || (tile == 16 && split >= 0 && split <= 2) || (tile == 32 && split >= 0 && split <= 3) ||
                  (tile == 128 && split == 128) || (tile == 256 && (split == 128 || split == 256)));
    fp8mm::g_kernel.store(tile << 16 | split, std::memory_order_relaxed);
    return PQE_OK;
}

int pqe_test_set_matmul_expiry(int who, int block) {
    PQE_CHECK_ARG(who >= fp8mm::EXPIRE_NONE && who <= fp8mm::EXPIRE_PARTS && block >= 0);
    fp8mm::g_expiry.store((int64_t)who << 32 | block, std::memory_order_relaxed);
    return PQE_OK;
}

int fp8_block_matmul(const uint8_t *x, int64_t x_stride, const float *x_scale, const uint8_t *w, const float *w_scale,
                     int M, int N, int K, void *out, int64_t out_stride, int out_fp32, int32_t *status, void *stream) {
    PQE_CHECK_ARG(M >= 0 && M <= 1 << 28 && N >= 1 && N <= 1 << 22 && K >= 16 && K <= 32768 && K % 16 == 0);
    if (M == 0) return PQE_OK;
    PQE_CHECK_ARG(x && x_scale && w && w_scale && out && status && x_stride >= K && x_stride % 16 == 0 && out_stride >= N);
    PQE_CHECK_ARG(aligned(x, 16) && aligned(w, 16) && aligned(x_scale, 4) && aligned(w_scale, 4) && aligned(status, 4) &&
                  aligned(out, out_fp32 ? 4 : 2));
    int dev = 0, sms = 0;
    const int rc = device_info(dev, sms);
    if (rc != PQE_OK) return rc;
    const int64_t expiry = fp8mm::g_expiry.load(std::memory_order_relaxed);
    const fp8mm::Call c{x, w, x_stride, K, {x_scale, w_scale, out, out_stride, M, N, (K + 127) / 128, out_fp32, status, wait_limit(),
                                            (int)(expiry >> 32), (int)(expiry & INT32_MAX)}};
    return fp8mm::run(c, sms, as_stream(stream));
}

}  // extern "C"
