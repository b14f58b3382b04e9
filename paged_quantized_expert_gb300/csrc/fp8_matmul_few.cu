// fp8_matmul_few.cu -- fp8_block_matmul for few rows of x: a stream of the weights.
//
// D[n, m] = W x^T: 128 rows of W are the MMA's M side, 16 or 32 tokens its N side, so a tile of W is read once and one scale of
// W holds for a whole tile and block. Each block of 128 along K is a product of its own into one of two TMEM accumulators; the
// epilogue adds it, times x's scale of that token and block and W's of the tile, to fp32 sums in registers (a thread holds a
// weight row's sums for every token).
//
// Where there are fewer tiles than SMs, a cluster of CTAs shares a tile's blocks of K: each sums its own and sends them, for
// each share of the tokens, to the CTA that finishes that share (stores into its shared memory that count on its barrier), and
// there they are added in the CTAs' order: the same result in every run, and no workspace.
//
// Warp 0 issues TMA (a ring of W and x stages), warp 1 the MMAs, warps 2-5 (one a TMEM lane quarter) scale and add. Two CTAs an
// SM: one's tile end, or the next call's set-up, beside the other's stream.
// 16 x 131072 x 2048: 44 us, 6.2 TB/s, the weights' bytes. 1 x 3584 x 2048: 3.5 us, 64 x 2048 x 2560: 5.0, of which set-up (TMEM,
// barriers), the first TMA and MMA, and the parts' way through the cluster are some 3: latency.
// Every wait is bounded. After one expires the roles stop waiting, and before the CTA ends its loads, its MMAs and the parts sent to
// it have come.
#include <atomic>

#include "fp8_matmul.cuh"

namespace pqe {
namespace fp8mm {
using namespace ptx;

template <int BN>
struct Few {
    static constexpr int W_BYTES = 128 * BK, X_BYTES = BN * BK, STAGE = W_BYTES + X_BYTES;
    static constexpr int STAGES = BN == 32 ? 4 : 5;
    static constexpr int GROUP = 4;                            // blocks whose scales are fetched together
    static constexpr uint32_t TMEM_COLS = 2 * BN;              // two accumulators
    static constexpr int PART_OFF = STAGES * STAGE;            // [column / 4][128 rows][4]: what the CTAs of a tile send
    static constexpr int SCALE_OFF = PART_OFF + 128 * BN * 4;  // [2][GROUP][BN]
    static constexpr int BAR_OFF = SCALE_OFF + 2 * GROUP * BN * 4;
    static constexpr int TMEM_OFF = BAR_OFF + 8 * (2 * STAGES + 6);
    static constexpr int SMEM = TMEM_OFF + 16 + 1024;          // + room to align to 1024
    static_assert(SMEM <= 113 * 1024, "shared memory of two CTAs");
};

constexpr int FEW_EPI = 128, FEW_THREADS = 64 + FEW_EPI;

// the first n of four neighbouring columns of D: out at one weight row of n tokens
__device__ __forceinline__ void put4(const Args &a, int64_t at, int n, const float4 &v) {
    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < n) {
            if (a.fp32) static_cast<float *>(a.out)[at + j * a.out_stride] = f[j];
            else static_cast<uint16_t *>(a.out)[at + j * a.out_stride] = f32_to_bf16_rn(f[j]);
        }
}

__device__ __forceinline__ float4 quad(uint64_t a, uint64_t b) {
    const float2 x = unpair(a), y = unpair(b);
    return make_float4(x.x, x.y, y.x, y.y);
}

template <int BN>
__global__ void __launch_bounds__(FEW_THREADS, 2)
    matmul_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Args a, int m_tiles,
                      int items, int parts_log) {
    using L = Few<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar_full = sbase + L::BAR_OFF, bar_empty = bar_full + 8 * L::STAGES;
    const uint32_t bar_tfull = bar_empty + 8 * L::STAGES, bar_tempty = bar_tfull + 16, bar_parts = bar_tempty + 16, bar_done = bar_parts + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::TMEM_OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // a cluster of 2^parts_log CTAs an item, or (one) items one after another; items of one weight tile are neighbours
    const int parts = 1 << parts_log, own_log = __ffs(BN) - 1 - parts_log, own = 1 << own_log;
    const int rank = (int)blockIdx.x & (parts - 1), first = (int)blockIdx.x >> parts_log, step = (int)gridDim.x >> parts_log;
    const int k0 = (int)((int64_t)a.kb * rank / parts), k1 = (int)((int64_t)a.kb * (rank + 1) / parts);

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::STAGES; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_tfull + 8 * b, 1);
            mbar_init(bar_tempty + 8 * b, FEW_EPI / 32);
        }
        mbar_init(bar_done, 1);
        mbar_init(bar_parts, 1);
        mbar_expect_tx(bar_parts, BN * 512);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmW)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmX)) : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(L::TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    if (parts_log) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // waited for where the first part is sent
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_acquire();

    bool late = false;
    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int i = first; i < items && ok; i += step) {
                const int nt = i / m_tiles, mt = i % m_tiles;
                for (int kb = k0; kb < k1; ++kb, ++it) {
                    const int s = it % L::STAGES;
                    if (!(ok = mbar_wait(bar_empty + 8 * s, ((uint32_t)(it / L::STAGES) & 1u) ^ 1u, a.polls(EXPIRE_LOADS, it)))) break;
                    const uint32_t at = sbase + s * L::STAGE;
                    mbar_expect_tx(bar_full + 8 * s, L::STAGE);
                    tma_load_2d(at, &tmW, kb * BK, nt * 128, bar_full + 8 * s);
                    tma_load_2d(at + L::W_BYTES, &tmX, kb * BK, mt * BN, bar_full + 8 * s);
                }
            }
            if (!ok) atomicOr(a.status, PQE_STATUS_TIMEOUT);
            for (int j = it > L::STAGES ? it - L::STAGES : 0; j < it; ++j)  // what was issued last has landed
                mbar_wait(bar_full + 8 * (j % L::STAGES), (uint32_t)(j / L::STAGES) & 1u, DRAIN);
        }
    } else if (warp == 1) {
        const uint32_t one = elect();
        int it = 0;
        bool ok = true;
        for (int i = first; i < items && ok; i += step)
            for (int kb = k0; kb < k1; ++kb, ++it) {
                const int s = it % L::STAGES, b = it & 1;
                ok = mbar_wait(bar_tempty + 8 * b, ((uint32_t)(it >> 1) & 1u) ^ 1u, a.polls(EXPIRE_MMA, it)) &&
                     mbar_wait(bar_full + 8 * s, (uint32_t)(it / L::STAGES) & 1u, a.wait_limit);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                tc_fence_after();
                const uint32_t at = sbase + s * L::STAGE;
                umma_block<1>(one, tmem + b * BN, at, at + L::W_BYTES, idesc(128, BN));
                commit<1>(one, bar_empty + 8 * s);
                commit<1>(one, bar_tfull + 8 * b);
            }
        if (!ok && lane == 0) atomicOr(a.status, PQE_STATUS_TIMEOUT);
        commit<1>(one, bar_done);  // the MMAs are done before TMEM goes
        mbar_wait(bar_done, 0, DRAIN);
    } else {
        const int q = warp & 3, n_at = 32 * q + lane, et = threadIdx.x - 64;
        float *scales = reinterpret_cast<float *>(smem + L::SCALE_OFF);
        float4 *mine = reinterpret_cast<float4 *>(smem + L::PART_OFF) + n_at;
        uint32_t limit = a.wait_limit;
        int it = 0, group = 0;
        for (int i = first; i < items; i += step) {
            const int nt = i / m_tiles, mt = i % m_tiles, m0 = mt * BN, nk = k1 - k0;
            const float *xs = a.xs + (int64_t)min(m0 + et, a.M - 1) * a.kb + k0, *ws = a.ws + (int64_t)nt * a.kb + k0;
            float fx[L::GROUP], fw[L::GROUP];
            auto fetch = [&](int at) {
#pragma unroll
                for (int j = 0; j < L::GROUP; ++j)
                    if (et < BN && at + j < nk) fx[j] = __ldg(xs + at + j), fw[j] = __ldg(ws + at + j);
            };
            fetch(0);
            uint64_t acc[BN / 2];
#pragma unroll
            for (int c = 0; c < BN / 2; ++c) acc[c] = 0;
            for (int at = 0; at < nk; at += L::GROUP, ++group) {
                float *sc = scales + (group & 1) * L::GROUP * BN;
                if (et < BN)
#pragma unroll
                    for (int j = 0; j < L::GROUP; ++j)
                        if (at + j < nk) sc[j * BN + et] = fx[j] * fw[j];
                // the readers of this half two groups ago were through at the last barrier
                asm volatile("bar.sync 1, %0;" ::"n"(FEW_EPI) : "memory");
                fetch(at + L::GROUP);
                for (int j = 0; j < L::GROUP && at + j < nk; ++j, ++it) {
                    const int b = it & 1;
                    if (!mbar_wait(bar_tfull + 8 * b, (uint32_t)(it >> 1) & 1u, min(limit, a.polls(EXPIRE_SUMS, it)))) {
                        limit = 1;  // the others keep to their barriers: go on without waiting
                        atomicOr(a.status, PQE_STATUS_TIMEOUT);
                    }
                    __syncwarp();
                    tc_fence_after();
                    const uint32_t t = tmem + b * BN + ((uint32_t)(32 * q) << 16);
                    const float4 *s4 = reinterpret_cast<const float4 *>(sc + j * BN);
                    uint32_t d[BN / 16][16];
#pragma unroll
                    for (int l = 0; l < BN / 16; ++l) tmem_ld16(t + 16 * l, d[l]);
#pragma unroll
                    for (int l = 0; l < BN / 16; ++l) {
                        tmem_wait(d[l]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 s = s4[4 * l + e];
                            uint64_t *o = acc + 8 * l + 2 * e;
                            o[0] = fma2(pair(d[l][4 * e], d[l][4 * e + 1]), pair(s.x, s.y), o[0]);
                            o[1] = fma2(pair(d[l][4 * e + 2], d[l][4 * e + 3]), pair(s.z, s.w), o[1]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_plain(bar_tempty + 8 * b);
                }
            }
            const int n = nt * 128 + n_at;
            if (parts_log == 0) {
                int64_t at = (int64_t)m0 * a.out_stride + n;
#pragma unroll
                for (int c = 0; c < BN / 4; ++c) {
                    const int left = a.M - m0 - 4 * c;
                    if (left <= 0) break;  // (code past it is not even fetched)
                    if (n < a.N) put4(a, at, min(4, left), quad(acc[2 * c], acc[2 * c + 1]));
                    at += 4 * a.out_stride;
                }
                continue;
            }
            // columns [r * own, (r + 1) * own) go to CTA r, which counts the bytes as they come
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // it has begun, and its barrier stands
#pragma unroll
            for (int c = 0; c < BN / 4; ++c) {
                const int to = c >> (own_log - 2), place = (rank << (own_log - 2)) + (c & (own / 4 - 1));
                const float4 v = quad(acc[2 * c], acc[2 * c + 1]);
                asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                                 map_rank(smem_u32(mine + place * 128), to)),
                             "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(map_rank(bar_parts, to))
                             : "memory");
            }
            // (every CTA sends its parts, also one whose waits expired: none leaves before all have come)
            if (!mbar_wait_cluster(bar_parts, 0, a.polls(EXPIRE_PARTS, rank) ? max(a.wait_limit, DRAIN) : 0)) {
                late = true;
                atomicOr(a.status, PQE_STATUS_TIMEOUT);
            }
            const int m1 = m0 + rank * own;
            for (int c = 0; c < own && m1 + c < a.M; c += 4) {
                float4 v = mine[c / 4 * 128];
                for (int r = 1; r < parts; ++r) {
                    const float4 o = mine[(r * own + c) / 4 * 128];
                    v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
                }
                if (n < a.N) put4(a, (int64_t)(m1 + c) * a.out_stride + n, min(4, a.M - m1 - c), v);
            }
        }
    }
    __syncwarp();
    if (parts_log && warp < 2) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    tc_fence_before();
    const bool any_late = __syncthreads_or(late);
    if (parts_log && any_late) {  // what the others send may still come
        cluster_sync();           // all of it has been sent (a CTA that is through is gone and does not count)
        if (threadIdx.x == 0) mbar_wait_cluster(bar_parts, 0, DRAIN);
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::TMEM_COLS) : "memory");
    }
}

template <int BN>
static int launch(const Call &c, int parts_log, int sms, cudaStream_t s) {
    using L = Few<BN>;
    static std::atomic<int> attr_set[PQE_MAX_DEVICES];
    int dev = 0, n = 0;
    const int rc = device_info(dev, n);
    if (rc != PQE_OK) return rc;
    if (!attr_set[dev].load(std::memory_order_relaxed)) {
        PQE_CUDA_TRY(cudaFuncSetAttribute(matmul_few_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM));
        attr_set[dev].store(1, std::memory_order_relaxed);
    }
    CUtensorMap mw, mx;
    if (!map_codes(&mw, c.w, (uint64_t)c.a.N, (uint64_t)c.K, (uint64_t)c.K, 128) ||
        !map_codes(&mx, c.x, (uint64_t)c.a.M, (uint64_t)c.K, (uint64_t)c.x_stride, BN))
        return PQE_ERR_UNSUPPORTED;
    const int m_tiles = (int)(((int64_t)c.a.M + BN - 1) / BN);
    const int64_t items = (int64_t)m_tiles * ((c.a.N + 127) / 128);
    if (items > INT32_MAX / 8) return PQE_ERR_INVALID_ARG;
    const unsigned grid = parts_log ? (unsigned)items << parts_log : (unsigned)(items < 2 * sms ? items : 2 * sms);
    return launch_clusters(matmul_few_kernel<BN>, grid, FEW_THREADS, L::SMEM, 1u << parts_log, s, mw, mx, c.a, m_tiles, (int)items,
                           parts_log);
}

int matmul_few(const Call &c, int tokens, int parts_log, int sms, cudaStream_t s) {
    return tokens == 16 ? launch<16>(c, parts_log, sms, s) : launch<32>(c, parts_log, sms, s);
}

}  // namespace fp8mm
}  // namespace pqe
