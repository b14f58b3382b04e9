// fp8_matmul_many.cu -- fp8_block_matmul for many rows of x: at the tensor cores' rate.
//
// A tile is 256 tokens by 256 or 128 weight rows on a pair of SMs (cta_group::2: each SM holds its own 128 tokens and half of
// the weight rows, the first CTA issues for both), or 128 by 128 on one. Each block of 128 along K is a product of its own into
// one of the TMEM accumulators (two of 256 columns, or four of 128). Eight warps an SM take it from there, a thread a token row
// and half of the columns, which lie in one 128-row block of W: one scale a thread and block, xs * ws, and a packed multiply-add
// for every two sums, held in registers over all of K.
//
// Persistent: a pair (or SM) takes every pairs-th tile. Warp 0 issues TMA, warp 1 the MMAs, warps 2 and 3 bring the scales to
// shared memory, warps 4-11 scale and add. Finished rows go through shared memory and leave as TMA stores (which cut what lies
// outside), or, where out is not aligned to 16 bytes or a row ends inside 16, element by element (the latter's last 64 bytes).
//
// In a replayed graph: 16384 x 4096 x 2560 120 us, 2.9 PFLOP/s (as calls in a row, where power lowers the clock, 135); 4099 x
// 3584 x 2048 30; 64 x 131072 x 2048 to fp32 52 (128 x 128 tiles, 5.8 TB/s of weights and results). What bounds the first: a
// block's product cannot be added to the next one's in the tensor core, so all of TMEM is read once a block. Without those reads
// (a copy of the kernel) the same loads and MMAs take 115 us, with accumulators enough never to wait 111; the two accumulators'
// round trip (MMA latency, commit, reading 128 columns, the arrival at the pair's first CTA) is what the rest is. A product with
// one scale for all of K, by the library, takes 96.
// Tried: 16 epilogue warps of 64 columns (154 us then against 135: TMEM reads at 221 bytes a clock, 294 with 8), two warps that
// issue in turn (137 against 135), scales read from global memory by each epilogue warp (32 lines a load: 135, 126 with the
// scale warps), the next barrier asked ahead (126 against 123), six stages (130 against 126), one SM a tile of 128 x 256 (136),
// tiles of a last round in halves where half of the pairs or more would be idle in it (127 against 118 to 122: the loops over K
// lose more by being there twice).
// Every wait is bounded. After one expires the roles stop, and before the CTAs end the first of them waits for every load that
// either has issued (each counts its own), and warp 1 for the MMAs.
#include <atomic>

#include "fp8_matmul.cuh"

namespace pqe {
namespace fp8mm {
using namespace ptx;

// Three warpgroups, 384 threads of 168 registers at launch (64512): the first gives its away, 2 * 128 * 216 + 128 * 72 as much.
constexpr int EPI_WARPS = 8, EPI_WARP0 = 4, SCALE_WARP0 = 2, MANY_THREADS = 128 + 32 * EPI_WARPS;
constexpr int EPI_REGS = 216, OTHER_REGS = 72;
static_assert(32 * EPI_WARPS * EPI_REGS + 128 * OTHER_REGS <= MANY_THREADS * 168, "registers of the launch");

template <int BN, int CTAS>
struct Many {
    static constexpr int A_BYTES = 128 * BK, B_ROWS = BN / CTAS, STAGE = A_BYTES + B_ROWS * BK;
    static constexpr int STAGES = BN == 256 || CTAS == 1 ? 4 : 6, NBUF = 512 / BN;
    static constexpr int CW = BN / 2;                            // columns of an epilogue warp
    static constexpr int BUF = 32 * 64, NOUT = 4;                // store buffers of a warp: 32 rows of 64 bytes
    static constexpr int OUT_OFF = STAGES * STAGE;
    // scales of a block: x's of the CTA's 128 rows, W's of the tile's two 128-row blocks. A slot is written anew when the block
    // NBUF before is full, and for that the epilogue warps have arrived too, once they had read the block NBUF before it. (Not a
    // barrier of the slots' own: a second poll a block in the scale warps took 13.0 us for 1024 x 3584 x 2048 in tiles of 256 x
    // 128, 11.6 without.)
    static constexpr int SLOTS = 2 * NBUF, SLOT = 128 + 4;
    static constexpr int SCALE_OFF = OUT_OFF + EPI_WARPS * NOUT * BUF;
    static constexpr int BAR_OFF = SCALE_OFF + SLOTS * SLOT * 4;
    static constexpr int TMEM_OFF = BAR_OFF + 8 * (2 * STAGES + 2 * NBUF + 1);
    static constexpr int SMEM = TMEM_OFF + 16;                   // TMEM's address, whether a role stopped, loads issued by each CTA
    static_assert(SMEM <= 227 * 1024, "shared memory of one CTA");
};

// a load into this CTA's shared memory; that of a pair counts on a barrier of the pair's first CTA
template <int CTAS>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t bar) {
    if constexpr (CTAS == 1) tma_load_2d(dst, map, c0, c1, bar);
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
            "[%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
}

// an arrival on a barrier of either CTA. It orders no memory of this thread's: what it says is that TMEM has been read, which
// the tcgen05 fences around it order (with release.cluster each arrival waited for the thread's earlier loads and stores: 57 us
// against 29 for 2048 x 4096 x 2560). That the block's scales have been read is said apart, inside the warp's CTA.
template <int CTAS>
__device__ __forceinline__ void arrive(uint32_t bar) {
    if constexpr (CTAS == 1) mbar_arrive_plain(bar);
    else asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <int BN, int CTAS, bool FP32>
__global__ void __launch_bounds__(MANY_THREADS, 1)
    matmul_many_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ CUtensorMap tmOut, const Args a, int n_tiles, int items, int tma_cols) {
    using L = Many<BN, CTAS>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint32_t sbase;  // in a register: as a constant it is put together anew for every descriptor (126 us against 122)
    asm volatile("mov.u32 %0, %1;" : "=r"(sbase) : "r"(smem_u32(smem)));
    const uint32_t bar_full = sbase + L::BAR_OFF, bar_empty = bar_full + 8 * L::STAGES;
    const uint32_t bar_tfull = bar_empty + 8 * L::STAGES, bar_tempty = bar_tfull + 8 * L::NBUF, bar_done = bar_tempty + 8 * L::NBUF;
    float *scales = reinterpret_cast<float *>(smem + L::SCALE_OFF);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::TMEM_OFF);
    volatile uint32_t *stopped = tmem_slot + 1, *issued = tmem_slot + 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CTAS == 2 ? cluster_rank() : 0;
    const int first = (int)blockIdx.x / CTAS, step = (int)gridDim.x / CTAS;

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::STAGES; ++s) {
            mbar_init(bar_full + 8 * s, 1);   // the first CTA's: its own arrival, and the bytes of both
            mbar_init(bar_empty + 8 * s, 1);  // each CTA's: the commit of the MMAs that read the stage
        }
        mbar_init(bar_done, 1);  // each CTA's: the last commit
        *stopped = 0;
        for (int b = 0; b < L::NBUF; ++b) {
            // each CTA's: the commit, its two scale warps, its epilogue warps when they are through with the buffer's last block
            mbar_init(bar_tfull + 8 * b, 3 + EPI_WARPS);
            mbar_init(bar_tempty + 8 * b, CTAS * EPI_WARPS);  // the first CTA's: the epilogue warps of both
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmX)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmW)) : "memory");
    }
    if (warp == 1) {
        if constexpr (CTAS == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512u)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512u)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if (CTAS == 2) cluster_sync();  // the other CTA's barriers are ready too
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_acquire();

    // (one lane, where loads may be left that no MMA has waited for) every CTA learns it
    auto stop = [&] {
        atomicOr(a.status, PQE_STATUS_TIMEOUT);
        for (int r = 0; r < CTAS; ++r) st_cluster(map_rank(smem_u32(tmem_slot + 1), r), 1);
    };
    if (warp < EPI_WARP0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
        if (warp == 0 && lane == 0) {
            const int who = rank == 0 ? EXPIRE_LOADS : EXPIRE_SECOND_LOADS;
            int it = 0;
            bool ok = true;
            for (int i = first; i < items && ok; i += step) {
                const int m0 = i / n_tiles * (128 * CTAS) + 128 * (int)rank, n0 = i % n_tiles * BN + L::B_ROWS * (int)rank;
                for (int kb = 0; kb < a.kb; ++kb, ++it) {
                    const int s = it % L::STAGES;
                    if (!(ok = mbar_wait(bar_empty + 8 * s, ((uint32_t)(it / L::STAGES) & 1u) ^ 1u, a.polls(who, it)))) break;
                    const uint32_t at = sbase + s * L::STAGE, bar = CTAS == 2 ? map_rank(bar_full + 8 * s, 0) : bar_full + 8 * s;
                    if (rank == 0) mbar_expect_tx(bar_full + 8 * s, CTAS * L::STAGE);
                    tma_load<CTAS>(at, &tmX, kb * BK, m0, bar);
                    tma_load<CTAS>(at + L::A_BYTES, &tmW, kb * BK, n0, bar);
                }
            }
            st_cluster(map_rank(smem_u32(tmem_slot + 2 + rank), 0), it);
            if (!ok) stop();
        }
        if (warp >= SCALE_WARP0) {
            // x's scales of 64 rows and one of W's, fetched a group of blocks ahead
            constexpr int G = 4;
            const int w = warp - SCALE_WARP0;
            float fx[G][2], fw[G];
            int it = 0;
            bool ok = true;
            auto fetch = [&](int i, int kb) {
                const int row = i / n_tiles * (128 * CTAS) + 128 * (int)rank + 64 * w + lane, col = i % n_tiles * BN + 128 * w;
                // rows and columns outside read the last one's; what they give is not stored
                const float *x0 = a.xs + (int64_t)min(row, a.M - 1) * a.kb, *x1 = a.xs + (int64_t)min(row + 32, a.M - 1) * a.kb;
                const float *ws = a.ws + (int64_t)(min(col, a.N - 1) / 128) * a.kb;
#pragma unroll
                for (int j = 0; j < G; ++j)
                    if (kb + j < a.kb) fx[j][0] = __ldg(x0 + kb + j), fx[j][1] = __ldg(x1 + kb + j), fw[j] = __ldg(ws + kb + j);
            };
            if (first < items) fetch(first, 0);
            for (int i = first; i < items && ok; i += step)
                for (int kb = 0; kb < a.kb && ok; kb += G) {
                    float vx[G][2], vw[G];
#pragma unroll
                    for (int j = 0; j < G; ++j) vx[j][0] = fx[j][0], vx[j][1] = fx[j][1], vw[j] = fw[j];
                    if (kb + G < a.kb) fetch(i, kb + G);
                    else if (i + step < items) fetch(i + step, 0);
#pragma unroll
                    for (int j = 0; j < G; ++j) {
                        if (kb + j >= a.kb || !ok) break;
                        const int b = it % L::NBUF;
                        ok = __all_sync(0xffffffffu, mbar_wait(bar_tfull + 8 * b, ((uint32_t)(it / L::NBUF) & 1u) ^ 1u, a.polls(EXPIRE_SCALES, it)));
                        if (!ok) break;
                        float *slot = scales + it % L::SLOTS * L::SLOT;
                        slot[64 * w + lane] = vx[j][0];
                        slot[64 * w + 32 + lane] = vx[j][1];
                        if (lane == 0) slot[128 + w] = vw[j];
                        __syncwarp();
                        if (lane == 0) mbar_arrive_plain(bar_tfull + 8 * b);
                        ++it;
                    }
                }
            if (!ok && lane == 0) atomicOr(a.status, PQE_STATUS_TIMEOUT);
        }
        if (warp == 1 && rank == 0) {
            const uint32_t one = elect();
            int it = 0;
            bool ok = true;
            for (int i = first; i < items && ok; i += step)
                for (int kb = 0; kb < a.kb; ++kb, ++it) {
                    const int s = it % L::STAGES, b = it % L::NBUF;
                    ok = mbar_wait(bar_full + 8 * s, (uint32_t)(it / L::STAGES) & 1u, a.polls(EXPIRE_MMA, it)) &&
                         mbar_wait(bar_tempty + 8 * b, ((uint32_t)(it / L::NBUF) & 1u) ^ 1u, a.wait_limit);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    tc_fence_after();
                    const uint32_t at = sbase + s * L::STAGE;
                    umma_block<CTAS>(one, tmem + b * BN, at, at + L::A_BYTES, idesc(128 * CTAS, BN));
                    commit<CTAS>(one, bar_empty + 8 * s);
                    commit<CTAS>(one, bar_tfull + 8 * b);
                }
            if (!ok && lane == 0) stop();
            commit<CTAS>(one, bar_done);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
        const int q = warp & 3, part = (warp - EPI_WARP0) >> 2;  // TMEM lane quarter, half of the columns
        uint8_t *buf = smem + L::OUT_OFF + (warp - EPI_WARP0) * L::NOUT * L::BUF;
        const uint32_t t0 = tmem + part * L::CW + ((uint32_t)(32 * q) << 16);
        const uint32_t tempty0 = CTAS == 2 ? map_rank(bar_tempty, 0) : bar_tempty;
        if (lane == 0)
            for (int b = 0; b < L::NBUF; ++b) mbar_arrive_plain(bar_tfull + 8 * b);
        int it = 0;
        bool ok = true;
        for (int i = first; i < items && ok; i += step) {
            uint64_t acc[L::CW / 2];
#pragma unroll
            for (int c = 0; c < L::CW / 2; ++c) acc[c] = 0;
            constexpr int LD = 4;  // loads under way at a time
            for (int kb = 0; kb < a.kb; ++kb, ++it) {
                const int b = it % L::NBUF;
                if (!__all_sync(0xffffffffu, mbar_wait(bar_tfull + 8 * b, (uint32_t)(it / L::NBUF) & 1u, a.polls(EXPIRE_SUMS, it)))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t t = t0 + b * BN;
                const float *slot = scales + it % L::SLOTS * L::SLOT;
                uint64_t s2;
#pragma unroll
                for (int c = 0; c < L::CW; c += 16 * LD) {
                    uint32_t d[LD][16];
#pragma unroll
                    for (int l = 0; l < LD; ++l) tmem_ld(t + c + 16 * l, d[l]);
                    if (c == 0) {
                        const float s = slot[32 * q + lane] * slot[128 + part * L::CW / 128];
                        s2 = pair(s, s);
                    }
#pragma unroll
                    for (int l = 0; l < LD; ++l) tmem_wait(d[l]);
#pragma unroll
                    for (int l = 0; l < LD; ++l)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            acc[c / 2 + 8 * l + e] = fma2(pair(d[l][2 * e], d[l][2 * e + 1]), s2, acc[c / 2 + 8 * l + e]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive<CTAS>(tempty0 + 8 * b), mbar_arrive_plain(bar_tfull + 8 * b);
            }
            if (!ok) {
                if (lane == 0) atomicOr(a.status, PQE_STATUS_TIMEOUT);
                break;
            }
            // 32 rows of CW values leave in pieces of 64 bytes a row, NOUT at a time
            constexpr int PER = FP32 ? 16 : 32, PIECES = L::CW / PER;
            const int row0 = i / n_tiles * (128 * CTAS) + 128 * (int)rank + 32 * q, col0 = i % n_tiles * BN + part * L::CW;
#pragma unroll
            for (int p0 = 0; p0 < PIECES; p0 += L::NOUT) {
                constexpr int N = PIECES < L::NOUT ? PIECES : L::NOUT;
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    uint8_t *mine = buf + j * L::BUF + lane * 64;
#pragma unroll
                    for (int v = 0; v < 4; ++v) {  // the output map's 64-byte swizzle
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if constexpr (FP32) {
                                const float2 f = unpair(acc[8 * (p0 + j) + 2 * v + e / 2]);
                                w[e] = __float_as_uint(e & 1 ? f.y : f.x);
                            } else {
                                const float2 f = unpair(acc[16 * (p0 + j) + 4 * v + e]);
                                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[e]) : "f"(f.y), "f"(f.x));
                            }
                        }
                        *reinterpret_cast<uint4 *>(mine + 16 * (v ^ ((lane >> 1) & 3))) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                if (tma_cols) {
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0 && row0 < a.M) {
#pragma unroll
                        for (int j = 0; j < N; ++j)
                            if (col0 + (p0 + j) * PER < tma_cols)
                                asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                                                 reinterpret_cast<uint64_t>(&tmOut)),
                                             "r"(col0 + (p0 + j) * PER), "r"(row0), "r"(smem_u32(buf + j * L::BUF))
                                             : "memory");
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                }
                if (tma_cols < a.N) {
                    __syncwarp();
                    constexpr int SIZE = FP32 ? 4 : 2;
                    const int c = lane % PER;
                    for (int j = max(0, (tma_cols - col0) / PER - p0); j < N; ++j)
                        for (int r = lane / PER; r < 32; r += 32 / PER) {
                            const int col = col0 + (p0 + j) * PER + c, row = row0 + r;
                            if (row >= a.M || col >= a.N) continue;
                            const uint8_t *from = buf + j * L::BUF + r * 64 + 16 * ((c * SIZE / 16) ^ ((r >> 1) & 3)) + c * SIZE % 16;
                            const int64_t at = (int64_t)row * a.out_stride + col;
                            if constexpr (FP32) static_cast<uint32_t *>(a.out)[at] = *reinterpret_cast<const uint32_t *>(from);
                            else static_cast<uint16_t *>(a.out)[at] = *reinterpret_cast<const uint16_t *>(from);
                        }
                    __syncwarp();
                }
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    __syncwarp();
    tc_fence_before();
    auto all = [] {
        if (CTAS == 1) __syncthreads();
        else cluster_sync();
    };
    all();  // neither CTA goes while the other's loads or arrivals may still reach it
    if (*stopped) {
        if (rank == 0 && threadIdx.x == 0) {
            // Loads of the last STAGES blocks may be under way: the MMAs waited for those before. A pair's count together, on the
            // first CTA's barrier of the stage, which that CTA armed for both with its own load.
            const int n0 = issued[0], n1 = issued[CTAS - 1], most = max(n0, n1);
            for (int j = max(0, most - L::STAGES); j < most; ++j) {
                const uint32_t bar = bar_full + 8 * (j % L::STAGES);
                if (j >= n0) mbar_expect_tx(bar, L::STAGE);
                else if (j >= n1) mbar_complete_tx(bar, L::STAGE);
                mbar_wait(bar, (uint32_t)(j / L::STAGES) & 1u, DRAIN);
            }
        }
        __syncwarp();
        all();
    }
    if (warp == 1) mbar_wait(bar_done, 0, DRAIN);  // nor before the MMAs are done, and have said so to both
    __syncwarp();
    if (warp == 1) {
        tc_fence_after();
        if constexpr (CTAS == 2)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

template <int BN, int CTAS, bool FP32>
static int launch(const Call &c, int sms, cudaStream_t s) {
    using L = Many<BN, CTAS>;
    static std::atomic<int> attr_set[PQE_MAX_DEVICES];
    int dev = 0, n = 0;
    const int rc = device_info(dev, n);
    if (rc != PQE_OK) return rc;
    if (!attr_set[dev].load(std::memory_order_relaxed)) {
        PQE_CUDA_TRY(cudaFuncSetAttribute(matmul_many_kernel<BN, CTAS, FP32>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM));
        attr_set[dev].store(1, std::memory_order_relaxed);
    }
    const int tma_cols = tma_columns(c.a);
    CUtensorMap mx, mw, mo = {};
    if (!map_codes(&mx, c.x, (uint64_t)c.a.M, (uint64_t)c.K, (uint64_t)c.x_stride, 128) ||
        !map_codes(&mw, c.w, (uint64_t)c.a.N, (uint64_t)c.K, (uint64_t)c.K, L::B_ROWS) || (tma_cols && !map_out(&mo, c.a, tma_cols)))
        return PQE_ERR_UNSUPPORTED;
    const int n_tiles = (c.a.N + BN - 1) / BN;
    const int64_t items = (int64_t)n_tiles * (((int64_t)c.a.M + 128 * CTAS - 1) / (128 * CTAS)), most = sms / CTAS;
    if (items > INT32_MAX / 8) return PQE_ERR_INVALID_ARG;
    return launch_clusters(matmul_many_kernel<BN, CTAS, FP32>, CTAS * (unsigned)(items < most ? items : most), MANY_THREADS, L::SMEM, CTAS, s, mx, mw, mo,
                           c.a, n_tiles, (int)items, tma_cols);
}

int matmul_many(const Call &c, int cols, int ctas, int sms, cudaStream_t s) {
    const bool f = c.a.fp32;
    if (ctas == 1) return f ? launch<128, 1, true>(c, sms, s) : launch<128, 1, false>(c, sms, s);
    if (cols == 128) return f ? launch<128, 2, true>(c, sms, s) : launch<128, 2, false>(c, sms, s);
    return f ? launch<256, 2, true>(c, sms, s) : launch<256, 2, false>(c, sms, s);
}

}  // namespace fp8mm
}  // namespace pqe
