// fp8_matmul.cuh -- what the kernels of fp8_block_matmul share (internal).
#pragma once

#include "f32x2.cuh"
#include "pqe_common.cuh"
#include "tc_ptx.cuh"

namespace pqe {
namespace fp8mm {
using namespace f32x2;
using ptx::cluster_rank;
using ptx::cluster_sync;
using ptx::map_rank;

constexpr int BK = 128;  // values (bytes) of K in a scale block, and in a stage
// polls of a wait for what the CTA itself has under way before it ends (some 20 ms: copies and MMAs take microseconds). Whatever
// limit other waits have, a CTA does not leave its shared memory and TMEM to them.
constexpr uint32_t DRAIN = 1u << 16;

// whose waits give up by pqe_test_set_matmul_expiry
enum Expiry { EXPIRE_NONE, EXPIRE_LOADS, EXPIRE_SECOND_LOADS, EXPIRE_MMA, EXPIRE_SCALES, EXPIRE_SUMS, EXPIRE_PARTS };

struct Args {
    const float *xs, *ws;  // scales [M, kb], [ceil(N / 128), kb]
    void *out;
    int64_t out_stride;
    int M, N, kb, fp32;
    int32_t *status;
    uint32_t wait_limit;
    int expire, expire_from;  // whose waits give up (none), and from which block of a CTA's on
    // polls of a wait of `who` for its CTA's block `it`
    __device__ __forceinline__ uint32_t polls(int who, int it) const { return expire == who && it >= expire_from ? 0 : wait_limit; }
};

struct Call {
    const uint8_t *x, *w;
    int64_t x_stride;
    int K;
    Args a;
};

// few rows: weight rows on the MMA's 128 lanes, `tokens` columns (16 or 32), the blocks of K shared by 2^parts_log CTAs
int matmul_few(const Call &c, int tokens, int parts_log, int sms, cudaStream_t s);
// many rows: 128 token rows on the lanes of an SM (ctas 1, cols 128) or 256 on those of a pair (2), `cols` weight rows (128 or 256)
int matmul_many(const Call &c, int cols, int ctas, int sms, cudaStream_t s);

// tensor map over bytes [rows, cols], rows `stride` apart, box [box_rows, 128], 128-byte swizzle; zeros outside
bool map_codes(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols, uint64_t stride, uint32_t box_rows);
// columns of the result, from the first on, that leave by TMA
int tma_columns(const Args &a);
// tensor map over the first `cols` columns of the result, box of 32 rows of 64 bytes, 64-byte swizzle
bool map_out(CUtensorMap *m, const Args &a, int cols);

// launch_pdl in clusters of `cluster` CTAs
template <typename... KArgs>
int launch_clusters(void (*kern)(KArgs...), unsigned grid, unsigned block, size_t smem, unsigned cluster, cudaStream_t s,
                    typename ident<KArgs>::type... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    PQE_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, args...));
    count_launch();
    return PQE_OK;
}

// ---- device ----

// takes bytes off what the barrier's phase still waits for
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// instruction descriptor, kind::f8f6f4: D fp32, A and B E4M3, both K-major
__host__ __device__ constexpr uint32_t idesc(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// waits for this thread's TMEM loads; the registers pass through it, so that nothing is computed from them before
template <int N>
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[N]) {
    static_assert(N == 16 || N == 32, "");
    if constexpr (N == 16)
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                       "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
    else
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                       "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                       "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                       "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[16]) { ptx::tmem_ld16(addr, r); }
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[32]) { ptx::tmem_ld32(addr, r); }

// One lane issues (`leader`), but its whole warp runs the code around it: descriptors then stay in uniform registers, where the
// instruction takes them from (inside a branch of one lane an MMA takes more than 100 clocks to issue). CTAS: 1, or 2 for a
// pair of SMs.
__device__ __forceinline__ uint32_t elect() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
template <int CTAS, bool ACCUM>
__device__ __forceinline__ void umma(uint32_t leader, uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t desc) {
    if constexpr (CTAS == 1)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t@q tcgen05.mma.cta_group::1.kind::f8f6f4 "
            "[%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(adesc), "l"(bdesc), "r"(desc), "n"(ACCUM ? 1 : 0), "r"(leader)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t@q tcgen05.mma.cta_group::2.kind::f8f6f4 "
            "[%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(adesc), "l"(bdesc), "r"(desc), "n"(ACCUM ? 1 : 0), "r"(leader)
            : "memory");
}
// one arrival on the barrier (of both CTAs of a pair) once the MMAs issued so far are done
template <int CTAS>
__device__ __forceinline__ void commit(uint32_t leader, uint32_t bar) {
    if constexpr (CTAS == 1)
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t@q "
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
            "r"(leader)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t@q "
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n\t}" ::"r"(bar),
            "r"(leader), "h"((uint16_t)3)
            : "memory");
}
// a block of 128 along K: D = A B^T of 128-byte rows
template <int CTAS>
__device__ __forceinline__ void umma_block(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t desc) {
    const uint64_t ad = ptx::sw128_desc(a), bd = ptx::sw128_desc(b);
    umma<CTAS, false>(leader, d, ad, bd, desc);
#pragma unroll
    for (int k = 1; k < BK / 32; ++k) umma<CTAS, true>(leader, d, ad + 2 * k, bd + 2 * k, desc);
}

// bounded wait for what other CTAs of the cluster wrote
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, uint32_t limit) {
    for (uint32_t i = 0; i < limit; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if (i > 32) __nanosleep(128);
    }
    return false;
}

}  // namespace fp8mm
}  // namespace pqe
