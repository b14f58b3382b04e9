// kv_attn_prompt.cu -- attention over the 4-bit paged cache for many query rows
// (prompt chunks) on the 5th-generation tensor cores.
//
// For one sequence and KV head the m * group query rows are cut into tiles of
// 128; a CTA takes two of them and walks the tokens that they see, 128 at a
// time. Per step and tile:
//   S = Q . K^T       tcgen05 kind::f16, M = 128 rows, N = 128 tokens, into TMEM
//   p = 2^(c S - ref + 8)   a row per thread, from TMEM to TMEM (f16, in S's place
//                     where the head size leaves no other room)
//   O += P . V        A from TMEM, N = d channels, fp32 in TMEM
// The two tiles alternate, so that the tensor pipe works on one while the other's
// softmax runs. The reference `ref` of a row follows its maximum only when
// that has grown by 7 or more (p stays under 2^15, inside f16); O and the sum are
// scaled then.
//
// Four warps turn codes into f16 in shared memory (128-byte swizzle, K-major
// both): K as it lies, V transposed on the way, its tokens in the order in which
// the cache's bytes hold them, which is the order P is written in. Codes are
// multiplied by 2^(scale - top + 13) with top the largest scale that the CTA's
// tokens have: exact while a scale is within 27 of it. Both tiles use what is
// converted once. Where some row sees scales far above what another row sees, the
// CTA's rows are summed one by one in fp32 instead.
//
// Where the tiles are fewer than SMs, each is cut along the cache into equal
// parts for several CTAs, which leave theirs in the workspace for a second kernel
// to join.
//
// Two chunks of 2048 tokens over 5000 to 8192 (16 heads, 4 KV heads of 128): 194.2
// us, 929 TFLOP/s of counted work. A step of both tiles takes some 3650 clocks an
// SM: 32 MMAs take 2050 at their peak and about 2600 here, beside the shared
// memory's own 2050 clocks for their operands and the converted tiles; a tile's
// chain is 1400 of softmax, two products and the waits between them; the four
// converting warps need about 3000. None of them is idle for long, and what runs on
// the issue slots of one runs against the others. Prompts of 17 to 701 tokens
// (heads of 64): 37.5 us, where a CTA's begin and end (tiles found, scales scanned,
// Q, the first conversion, the rows out) are 7 of its 12 us.
#include <math.h>

#include "kv_attn_plain.cuh"
#include "tc_ptx.cuh"

namespace pqe {
namespace kv {
namespace prompt {
using namespace ptx;

constexpr int BM = 128;           // rows of a tile
constexpr int TILES = 2;          // tiles of a CTA
constexpr int BK = 128;           // tokens of a step
constexpr int SOFT_WARPS = 8;     // four per tile
constexpr int CONV_WARPS = 4;
constexpr int MMA_WARP = SOFT_WARPS + CONV_WARPS;
constexpr int THREADS = 32 * (MMA_WARP + 4);  // the last warpgroup holds the MMA warp alone
// registers a thread, by warpgroup: the softmax warps take what the others give up of the 128 each that 512 threads are
// launched with
constexpr int LAUNCH_REGS = 128, SOFT_REGS = 168, CONV_REGS = 112, MMA_REGS = 64;
static_assert((2 * SOFT_REGS + CONV_REGS + MMA_REGS) * 128 <= LAUNCH_REGS * THREADS, "above the launch's total");
constexpr int CHUNK = 128 * 128;  // bytes of 128 rows of 64 f16
constexpr float LAZY = 7.f;       // growth of a maximum that its reference does not follow
// Exponents of two (a score and its reference) above which c s - c ref is not taken as one fma: the product of the reference, once
// rounded, would be off by a part of its own size, which is all of p's exponent from 2^27 or so on.
constexpr float FAR = 1 << 20;

// TMEM columns
__device__ __forceinline__ constexpr uint32_t s_col(int tile) { return 128 * tile; }
__device__ __forceinline__ constexpr uint32_t o_col(int tile) { return 256 + 128 * tile; }
template <int D>
__device__ __forceinline__ constexpr uint32_t p_col(int tile) {  // P: half a column per token
    return D == 128 ? s_col(tile) : o_col(tile) + 64;
}

template <int N>
struct Find {  // find_tiles()'s scratch
    static_assert(N % 32 == 0, "whole warps");
    int scan[N / 32];
    int2 found;
};

template <int D>
struct Smem {
    alignas(1024) uint8_t q[TILES][D / 64][CHUNK];  // [128-byte rows of 64 channels]
    uint8_t k[2][D / 64][CHUNK];
    uint8_t v[2][2][D * 128];  // V^T: D rows of 64 tokens, two a step
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full[2], drained;
    uint32_t tmem;
    Find<THREADS> find;
    alignas(16) uint2 tops[THREADS / 32];  // what each warp found of the scales: K's in the low halves, V's in the high ones
    int k_nan, v_nan;
    // of a step's 16-token blocks, two bits from each converting warp: those that are there. Four steps' worth: a
    // step's is rewritten only once the softmax of the step three before has ended.
    alignas(4) uint8_t have[4][CONV_WARPS];
};

// One lane issues (`leader`), but all of its warp runs the code around it: descriptors then stay in uniform registers,
// where the instruction takes them from. (With the loop inside a branch of one lane an MMA took some 130 clocks to issue.)
template <bool ACCUM>
__device__ __forceinline__ void umma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t@q tcgen05.mma.cta_group::1.kind::f16 "
        "[%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "n"(ACCUM ? 1 : 0), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t@q tcgen05.mma.cta_group::1.kind::f16 "
        "[%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accum), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 "
        "[%0];\n\t}" ::"r"(bar),
        "r"(leader)
        : "memory");
}
__device__ __forceinline__ uint32_t elect() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// two fp32 operations in one instruction
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float &x, float &y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// for the softmax and MMA warpgroups; the converting warps begin beside the loads of Q
__device__ __forceinline__ void q_barrier() {
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS - 32 * CONV_WARPS) : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Bits of the 32 tokens from j on that lie in [lo, hi) and in one of the two blocks of `have` (a bit each).
__device__ __forceinline__ uint32_t seen(int j, int lo, int hi, uint32_t have) {
    const int from = min(max(lo - j, 0), 32), to = min(max(hi - j, 0), 32);
    const uint32_t below = to < 32 ? (1u << to) - 1u : 0xFFFFFFFFu, before = from < 32 ? (1u << from) - 1u : 0xFFFFFFFFu;
    return below & ~before & ((have & 1u ? 0x0000FFFFu : 0u) | (have & 2u ? 0xFFFF0000u : 0u));
}

// f16 pair of 2^(x - top + 13) for the E8M0 bytes x <= top in the halves of `two` (times a code, 6 at most, still inside f16);
// zero from 28 below top on
struct Weights {
    uint32_t least, add;
    __device__ __forceinline__ explicit Weights(int top)
        : least((uint32_t)max(top - 28, 0) * 0x10001u), add((uint32_t)(28 - top) * (1024u * 0x10001u)) {}
    __device__ __forceinline__ uint32_t operator()(uint32_t two) const { return __vmaxu2(two, least) * 1024u + add; }
};

// 2^(top - 140): what a product with a weighted value lacks to the value's own
__device__ __forceinline__ float unweight(int top) {
    return __uint_as_float(top > 13 ? (uint32_t)(top - 13) << 23 : 1u << (top + 9));
}
// Scales further apart than this, between the largest that some row of a CTA sees and what another row sees, leave the CTA's rows
// to plain_rows(). What is 15 below the largest that a row sees then still has its weight.
constexpr int APART = 12;

// The sequence and tile pair of place `at` in the line of all sequences' tile pairs, counted from its end (the last of a
// sequence see the most tokens, and go first); .x < 0 past its beginning. For all N threads of a block.
template <int N>
__device__ __forceinline__ int2 find_tiles(const AttnArgs &a, int at, Find<N> &sm) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = a.n_q / a.c.n_kv;
    const int per = (a.B + N - 1) / N, b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    auto tiles_of = [&](int b) {
        int first, m, len;
        sequence_of(a, b, first, m, len);
        if (!is_ours(a, m)) return 0;
        return (int)(((int64_t)m * group + BM * TILES - 1) / (BM * TILES));
    };
    if (tid == 0) sm.found = make_int2(-1, 0);
    int mine = 0;
    for (int b = b0; b < b1; ++b) mine += tiles_of(b);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) sm.scan[warp] = incl;
    __syncthreads();
    int total = 0, before = incl - mine;
#pragma unroll
    for (int w = 0; w < N / 32; ++w) {
        if (w < warp) before += sm.scan[w];
        total += sm.scan[w];
    }
    const int want = total - 1 - at;
    if (want >= before && want < before + mine)
        for (int b = b0; b < b1; ++b) {
            const int n = per > 1 ? tiles_of(b) : mine;
            if (want < before + n) {
                sm.found = make_int2(b, want - before);
                break;
            }
            before += n;
        }
    __syncthreads();
    return sm.found;
}

// A part's result for its 256 rows: O as [D / 4][row][4], then m and l of the rows, fp32
constexpr int ROWS = BM * TILES;
__host__ __device__ constexpr int part_floats(int d) { return ROWS * (d + 2); }

// A CTA's rows one by one from the cache, over tokens [from, to): a warp each
template <int D, bool SPLIT>
__device__ __noinline__ void plain_rows(const AttnArgs a, int b, int kv_head, int first, int m, int len, int row0, int from, int to,
                                        float *parts) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, group = a.n_q / a.c.n_kv;
    for (int r = threadIdx.x >> 5; r < ROWS && row0 + r < m * group; r += THREADS / 32) {
        const int i = (row0 + r) / group, head = kv_head * group + (row0 + r) % group;
        int lo, hi;
        visible(a, i, m, len, lo, hi);
        const PlainRow<D> x = plain_row<D>(a.c, a.block_table + (size_t)b * a.max_pages, kv_head,
                                           a.q + (int64_t)(first + i) * a.q_stride + head * D, a.scale, max(lo, from), min(hi, to));
        const int64_t row = (int64_t)(first + i) * a.n_q + head;
        if constexpr (SPLIT) {  // in units of 2^-8, as the others' parts
            float *part = parts + (size_t)blockIdx.x * part_floats(D);
#pragma unroll
            for (int e = 0; e < E; ++e) part[((lane * E + e) / 4 * ROWS + r) * 4 + (lane * E + e) % 4] = 256.f * x.o[e];
            if (lane == 0) {
                part[ROWS * D + r] = x.m;
                part[ROWS * D + ROWS + r] = 256.f * x.l;
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) a.out[row * D + lane * E + e] = f32_to_bf16_rn(x.l == 0.f ? 0.f : x.o[e] / x.l);
            if (lane == 0 && a.lse) a.lse[row] = x.l == 0.f ? -INFINITY : (x.m + log2f(x.l)) * 0.693147180559945309f;
        }
    }
}

// SPLIT: of `splits` CTAs of a tile pair each leaves a part (a kernel of its own, so that the other has its registers).
template <int D, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1) attn_prompt_kernel(const AttnArgs a, int n_splits, float *parts) {
    const int splits = SPLIT ? n_splits : 1;
    extern __shared__ uint8_t smem_raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = a.n_q / a.c.n_kv, part_no = blockIdx.x % splits, head = blockIdx.x / splits % a.c.n_kv;
    constexpr uint32_t IDESC_S = (1u << 4) | ((uint32_t)(BK >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
    constexpr uint32_t IDESC_O = (1u << 4) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sm.k_full[i]), CONV_WARPS);
            mbar_init(smem_u32(&sm.v_full[i]), CONV_WARPS);
            mbar_init(smem_u32(&sm.k_empty[i]), 1);
            mbar_init(smem_u32(&sm.v_empty[i]), 1);
            mbar_init(smem_u32(&sm.s_full[i]), 1);
            mbar_init(smem_u32(&sm.p_full[i]), 4);
            mbar_init(smem_u32(&sm.o_full[i]), 1);
        }
        mbar_init(smem_u32(&sm.drained), 1);
        sm.k_nan = sm.v_nan = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    pdl_acquire();

    // ---- this CTA's sequence and rows ----
    const int2 found = find_tiles<THREADS>(a, (int)(blockIdx.x / ((uint32_t)splits * a.c.n_kv)), sm.find);
    const int b = found.x;
    if (b < 0) return;
    int first, m, len;
    sequence_of(a, b, first, m, len);
    if (a.kv_lens[b] > len && tid == 0) atomicOr(a.status, PQE_STATUS_BAD_PAGE);
    const int row0 = found.y * (BM * TILES), n_rows = m * group;
    const int tiles = row0 + BM < n_rows ? 2 : 1;
    // the tokens that some row of the CTA sees
    int lo, hi, lo_last, hi_last;  // of the first row, and of the last
    visible(a, row0 / group, m, len, lo, hi);
    visible(a, (min(row0 + BM * TILES, n_rows) - 1) / group, m, len, lo_last, hi_last);
    int k_first = lo / BK * BK, k_end = max(hi_last, 0);
    int steps = k_end > k_first ? (k_end - k_first + BK - 1) / BK : 0;
    if constexpr (SPLIT) {
        // this part's steps of them
        const int from = (int)((int64_t)steps * part_no / splits), to = (int)((int64_t)steps * (part_no + 1) / splits);
        k_end = min(k_end, k_first + to * BK);
        k_first += from * BK;
        steps = to - from;
    }
    const int32_t *table = a.block_table + (size_t)b * a.max_pages;
    const int page_mask = (1 << a.c.page_shift) - 1;

    // ---- the largest K and V scales among those tokens, and whether every row sees some near them ----
    // Each row sees the tokens that all see, of which there may be whole blocks: then their largest counts. Else it sees one of
    // the tokens at least: then the token counts whose largest block is the smallest (as 255 less, so that it is a maximum too).
    const bool same = lo == lo_last && hi == hi_last;  // all rows see the same
    const int all_lo = max(lo_last, k_first), all_hi = min(hi, k_end);
    const bool common = (all_lo + BLOCK - 1) / BLOCK * BLOCK + BLOCK <= all_hi;
    {
        int kt = 0, vt = 0, ka = 0, va = 0, nan = 0;
        constexpr int PIECES = D / 16;  // 16-byte pieces of a block's scales: K's, then V's
        const int n_pieces = (k_end - k_first + BLOCK - 1) / BLOCK * PIECES;
        constexpr int AHEAD = 4;  // loads in flight: table entries, then scales
        for (int i0 = tid; i0 < n_pieces; i0 += AHEAD * THREADS) {
            int page[AHEAD];
            uint4 u[AHEAD];
#pragma unroll
            for (int y = 0; y < AHEAD; ++y) {
                const int i = i0 + y * THREADS, j = k_first + i / PIECES * BLOCK;
                // before the window a page may be gone
                page[y] = i < n_pieces && j + BLOCK > lo ? max(table[j >> a.c.page_shift], -1) : -2;
            }
#pragma unroll
            for (int y = 0; y < AHEAD; ++y) {
                const int i = i0 + y * THREADS, j = k_first + i / PIECES * BLOCK;
                u[y] = make_uint4(0, 0, 0, 0);
                if (page[y] >= 0 && page[y] < a.c.n_pages)
                    u[y] = *reinterpret_cast<const uint4 *>(block_of<D>(a.c, page[y], j & page_mask, head) + 16 * D +
                                                            16 * (i % PIECES));
                else if (page[y] != -2)
                    atomicOr(a.status, PQE_STATUS_BAD_PAGE);
            }
#pragma unroll
            for (int y = 0; y < AHEAD; ++y) {
                if (page[y] == -2) continue;
                const int i = i0 + y * THREADS, j = k_first + i / PIECES * BLOCK, piece = i % PIECES;
                uint32_t w[4] = {u[y].x, u[y].y, u[y].z, u[y].w};
                const bool is_v = piece >= PIECES / 2;
                const int at = piece % (PIECES / 2), left = k_end - j, skip = lo - j;
                auto largest = [&] {
                    uint32_t two = 0;
#pragma unroll
                    for (int x = 0; x < 4; ++x) two = __vmaxu2(two, __vmaxu2(w[x] & 0x00FF00FFu, (w[x] >> 8) & 0x00FF00FFu));
                    return (int)max(two & 0xFFFFu, two >> 16);
                };
                int top = largest(), all = j >= all_lo && j + BLOCK <= all_hi ? top : 0;
                if (top == 255 || left < BLOCK || skip > 0 || !(common || same)) {
                    // some blocks are NaN, or of tokens that are not there or that no row sees: K [token][G], V [t][G][j]
                    int near = 0;
                    uint32_t m = 0;  // V: the largest byte of each of four tokens
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        uint32_t keep = 0;
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const int tok = is_v ? 2 * (D == 128 ? at : 2 * at + (x >> 1)) + (z & 1) + 8 * (z >> 1)
                                                 : at * (512 / D) + (4 * x + z) / (D / 32);
                            keep |= tok >= skip && tok < left ? 0xFFu << (8 * z) : 0u;
                        }
                        const uint32_t bad = __vcmpeq4(w[x], 0xFFFFFFFFu) & keep;
                        if (bad) nan |= is_v ? 1 : 2;
                        w[x] &= keep & ~bad;
                        if (!is_v) {
                            m = __vmaxu4(w[x], w[x] >> 8);
                            if (D == 128) m = __vmaxu4(m, m >> 16);
                            m &= D == 128 ? 0xFFu : 0x00FF00FFu;
                        } else {
                            m = x % (D / 32) == 0 ? w[x] : __vmaxu4(m, w[x]);
                        }
                        if (!is_v || x % (D / 32) == D / 32 - 1) {
                            const uint32_t n = ~m & ~__vcmpeq4(m, 0);  // 255 less each that is not zero
                            near = max(near, (int)max(max(n & 0xFFu, n >> 8 & 0xFFu), max(n >> 16 & 0xFFu, n >> 24)));
                        }
                    }
                    top = largest();
                    all = !common ? near : all ? top : 0;
                }
                if (is_v)
                    vt = max(vt, top), va = max(va, all);
                else
                    kt = max(kt, top), ka = max(ka, all);
            }
        }
        kt = __reduce_max_sync(0xffffffffu, kt);
        vt = __reduce_max_sync(0xffffffffu, vt);
        ka = __reduce_max_sync(0xffffffffu, ka);
        va = __reduce_max_sync(0xffffffffu, va);
        nan = __reduce_or_sync(0xffffffffu, nan);
        if (lane == 0) {
            sm.tops[warp] = make_uint2((uint32_t)(kt | vt << 16), (uint32_t)(ka | va << 16));
            if (nan & 1) atomicOr(&sm.v_nan, 1);
            if (nan & 2) atomicOr(&sm.k_nan, 1);
        }
    }
    if (warp == MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    uint32_t tops = 0, alls = 0;
#pragma unroll
    for (int x = 0; x < THREADS / 32; ++x) {
        const uint2 u = sm.tops[x];
        tops = __vmaxu2(tops, u.x);
        alls = __vmaxu2(alls, u.y);
    }
    if (!common) alls = 0x00FF00FFu - alls;
    const int k_top = (int)(tops & 0xFFFFu), v_top = (int)(tops >> 16);

    if (!same && max(k_top - (int)(alls & 0xFFFFu), v_top - (int)(alls >> 16)) > APART) {
        plain_rows<D, SPLIT>(a, b, head, first, m, len, row0, k_first, k_end, parts);
    } else if (warp < SOFT_WARPS) {
        more_registers<SOFT_REGS>();
        // ================= softmax: a row per thread =================
        const int tile = warp >> 2, r = tid & (BM - 1), row = row0 + tile * BM + r;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const bool valid = row < n_rows;
        const int64_t out_row = (int64_t)(first + row / group) * a.n_q + head * group + row % group;
        int my_lo = 0, my_hi = 0;
        float c = 1.f;
        if (tile < tiles) {
            // the row to f16, scaled by a power of two
            uint4 raw[D / 8];
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) raw[i] = make_uint4(0, 0, 0, 0);
            if (valid) {
                visible(a, row / group, m, len, my_lo, my_hi);
                const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (int64_t)(first + row / group) * a.q_stride +
                                                                   (head * group + row % group) * D);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) raw[i] = src[i];
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                for (int x = 0; x < 4; ++x) top = max(top, max(w[x] & 0x7FFFu, w[x] >> 16 & 0x7FFFu));
            }
            float f, inv;
            q_factor(top, f, inv);
            c = fabsf(a.scale) * inv * unweight(k_top);
            if (a.scale < 0.f) f = -f;
            if (c == 0.f) c = 1e-38f;                             // scores of (next to) zero, and no 0 * infinity
            if (top >= 0x7F80u) f = __uint_as_float(0x7FC00000u);  // a row that is not finite: scores of NaN
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                uint32_t o[4];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    o[x] = pack_f16(__uint_as_float(w[x] << 16) * f, __uint_as_float(w[x] & 0xFFFF0000u) * f);
                *reinterpret_cast<uint4 *>(&sm.q[tile][i >> 3][r * 128 + (((i & 7) ^ (r & 7)) << 4)]) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
        fence_async();
        q_barrier();  // Q is there
        if (tile < tiles) {
            float ref = -INFINITY, l = 0.f;  // ref: of S, c times it an exponent of two; l: 2^8 times the sum
            bool ok = true;
            for (int it = 0; it < steps; ++it) {
                if (!mbar_wait(smem_u32(&sm.s_full[tile]), it & 1, a.wait_limit)) ok = false;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const int k0 = k_first + it * BK;
                const uint32_t s_at = tmem + lanes + s_col(tile), p_at = tmem + lanes + p_col<D>(tile);
                const uint32_t have = *reinterpret_cast<const volatile uint32_t *>(sm.have[it & 3]);
                const bool all = __all_sync(0xffffffffu, !valid || (k0 + BK <= my_hi && k0 >= my_lo)) && have == 0x03030303u;
                bool done = false;
                if (all && __all_sync(0xffffffffu, fabsf(ref * c) < FAR)) {
                    // Every token is seen, and the reference will most likely stand: one pass, the probabilities held
                    // back until the maximum is known.
                    uint32_t p[BK / 2], s[2][32];
                    const float base = fmaf(-ref, c, 8.f);
                    const uint64_t c2 = pair(c, c), base2 = pair(base, base);
                    uint64_t sum2[2] = {0, 0};
                    float top0 = -INFINITY, top1 = -INFINITY;
                    tmem_ld32(s_at, s[0]);
#pragma unroll
                    for (int ch = 0; ch < BK / 32; ++ch) {
                        tmem_ld_wait();
                        if (ch + 1 < BK / 32) tmem_ld32(s_at + 32 * (ch + 1), s[(ch + 1) & 1]);
                        const uint32_t(&u)[32] = s[ch & 1];
                        float e[32];
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float s0 = __uint_as_float(u[i]), s1 = __uint_as_float(u[i + 1]);
                            const float s2 = __uint_as_float(u[i + 2]), s3 = __uint_as_float(u[i + 3]);
                            top0 = max3(top0, s0, s1);
                            top1 = max3(top1, s2, s3);
                            unpair(fma2(pair(s0, s1), c2, base2), e[i], e[i + 1]);
                            unpair(fma2(pair(s2, s3), c2, base2), e[i + 2], e[i + 3]);
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) e[i] = exp2_approx(e[i]);
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            sum2[0] = add2(sum2[0], pair(e[i], e[i + 1]));
                            sum2[1] = add2(sum2[1], pair(e[i + 2], e[i + 3]));
                        }
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            const int j = (x >> 1 & 1) * 16 + (x & 1) * 8 + (x >> 2) * 2;
                            p[16 * ch + x] = pack_f16(e[j], e[j + 1]);
                        }
                    }
                    if (!__any_sync(0xffffffffu, (fmaxf(top0, top1) - ref) * c > LAZY)) {
                        tmem_st32(p_at, *reinterpret_cast<const uint32_t(*)[32]>(p));
                        tmem_st32(p_at + 32, *reinterpret_cast<const uint32_t(*)[32]>(p + 32));
                        float x, y;
                        unpair(add2(sum2[0], sum2[1]), x, y);
                        l += x + y;
                        done = true;
                    }
                }
                if (!done) {
                    // pass 1: the maximum
                    float top = -INFINITY;
#pragma unroll 1
                    for (int ch = 0; ch < BK / 32; ++ch) {
                        uint32_t s[32];
                        tmem_ld32(s_at + 32 * ch, s);
                        tmem_ld_wait();
                        if (all) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) top = fmaxf(top, __uint_as_float(s[i]));
                        } else {
                            const uint32_t sees = seen(k0 + 32 * ch, my_lo, my_hi, have >> (8 * ch));
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (sees >> i & 1) top = fmaxf(top, __uint_as_float(s[i]));
                        }
                    }
                    // the reference follows a maximum that has outgrown it; O and the sum with it
                    const bool grow = (top - ref) * c > LAZY;  // (nothing seen yet: NaN, or infinity)
                    if (__any_sync(0xffffffffu, grow)) {
                        const float keep = grow ? exp2_approx((ref - top) * c) : 1.f;
                        if (grow) ref = top;
                        l *= keep;
                        if (it > 0) {
#pragma unroll 1
                            for (int ch = 0; ch < D / 32; ++ch) {
                                uint32_t o[32];
                                tmem_ld32(tmem + lanes + o_col(tile) + 32 * ch, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
                                tmem_st32(tmem + lanes + o_col(tile) + 32 * ch, o);
                            }
                            tmem_st_wait();
                        }
                    }
                    // pass 2: the probabilities
                    const float base = ref == -INFINITY ? 0.f : ref;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                    for (int ch = 0; ch < BK / 32; ++ch) {
                        uint32_t s[32];
                        tmem_ld32(s_at + 32 * ch, s);
                        tmem_ld_wait();
                        float p[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) p[i] = exp2_approx(fmaf(__uint_as_float(s[i]) - base, c, 8.f));
                        if (!all) {
                            const uint32_t sees = seen(k0 + 32 * ch, my_lo, my_hi, have >> (8 * ch));
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!(sees >> i & 1)) p[i] = 0.f;
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) sum[i & 3] += p[i];
                        // in the order of V^T's columns: t, block of the pair, tokens 2t, 2t+1, 2t+8, 2t+9
                        uint32_t o[16];
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            const int j = (x >> 1 & 1) * 16 + (x & 1) * 8 + (x >> 2) * 2;
                            o[x] = pack_f16(p[j], p[j + 1]);
                        }
                        tmem_st16(p_at + 16 * ch, o);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_plain(smem_u32(&sm.p_full[tile]));
            }
            // ---- the rows' results ----
            if (ok && steps > 0) {
                if (!mbar_wait(smem_u32(&sm.o_full[tile]), 0, a.wait_limit)) ok = false;
                ok = __all_sync(0xffffffffu, ok);
            }
            if (!ok) {
                if (lane == 0) atomicOr(a.status, PQE_STATUS_TIMEOUT);
            } else {
                tc_fence_after();
                uint32_t nan = 0;  // blocks of channels where the row sees a NaN
                if (sm.v_nan && valid) {
                    for (int j = max(my_lo, k_first); j < min(my_hi, k_end); ++j) {
                        const int page = table[j >> a.c.page_shift];
                        if (page < 0 || page >= a.c.n_pages) continue;
                        const uint8_t *blk = block_of<D>(a.c, page, j & page_mask, head);
#pragma unroll
                        for (int G = 0; G < D / 32; ++G) nan |= (blk[v_scale<D>(j & 15, G)] == 255 ? 1u : 0u) << G;
                    }
                }
                const float inv = SPLIT ? unweight(v_top) : l == 0.f ? 0.f : unweight(v_top) / l;
#pragma unroll
                for (int ch = 0; ch < D / 32; ++ch) {
                    uint32_t o[32];
                    if (steps > 0) {
                        tmem_ld32(tmem + lanes + o_col(tile) + 32 * ch, o);
                        tmem_ld_wait();
                    }
                    if constexpr (SPLIT) {
                        float4 *part = reinterpret_cast<float4 *>(parts + (size_t)blockIdx.x * part_floats(D));
                        const float f = nan >> ch & 1 ? __uint_as_float(0x7FC00000u) : inv;
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            float v[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) v[y] = l == 0.f ? 0.f : __uint_as_float(o[4 * x + y]) * f;
                            part[(8 * ch + x) * ROWS + tile * BM + r] = make_float4(v[0], v[1], v[2], v[3]);
                        }
                    } else if (valid) {
                        const float f = nan >> ch & 1 ? __uint_as_float(0x7FC00000u) : inv;
                        uint4 *dst = reinterpret_cast<uint4 *>(a.out + out_row * D + 32 * ch);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            uint32_t u[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const int i = 8 * x + 2 * y;
                                const float v0 = l == 0.f ? 0.f : __uint_as_float(o[i]) * f;
                                const float v1 = l == 0.f ? 0.f : __uint_as_float(o[i + 1]) * f;
                                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[y]) : "f"(v1), "f"(v0));
                            }
                            dst[x] = make_uint4(u[0], u[1], u[2], u[3]);
                        }
                    }
                }
                if constexpr (SPLIT) {
                    float *ml = parts + (size_t)blockIdx.x * part_floats(D) + ROWS * D + tile * BM + r;
                    ml[0] = ref * c;
                    ml[ROWS] = l;
                } else if (valid && a.lse) {
                    a.lse[out_row] = l == 0.f ? -INFINITY : (ref * c + log2f(l) - 8.f) * 0.693147180559945309f;
                }
            }
        }
    } else if (warp < MMA_WARP) {
        fewer_registers<CONV_REGS>();
        // ================= conversion: warp w takes a step's blocks 2w and 2w + 1 =================
        const int w = warp - SOFT_WARPS;
        constexpr int NK = D / 32;  // 16-byte pieces of K a thread takes
        constexpr int NV = D / 64;  // planes of V
        uint4 kr[NK], vr[NV][2];
        uint32_t ks[NK], vs[NV][2][2];
        int pages[2];
        auto look = [&](int it) {  // table entries of the warp's two blocks
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = k_first + it * BK + (2 * w + i) * BLOCK;
                pages[i] = j < k_end && j + BLOCK > lo ? table[j >> a.c.page_shift] : -1;
            }
        };
        // a K piece's token: rows 0..7 of a block to a warp's lanes so that a quarter warp's stores meet eight banks
        const int g = lane >> 2, t = lane & 3;
        const int tok8 = ((lane >> 2) & 1) * 4 + (lane >> 3);  // D = 128: 8 tokens x 4 pieces of 16 bytes
        const int tok16 = ((lane >> 1) & 1) * 4 + ((lane >> 2) & 3) + (lane >> 4) * 8;  // D = 64: 16 tokens x 2 pieces
        auto load = [&](int it) -> uint32_t {
            uint32_t have = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = k_first + it * BK + (2 * w + i) * BLOCK;
                const bool in = pages[i] >= 0 && pages[i] < a.c.n_pages;
                if (in) have |= 1u << i;
                const uint8_t *blk = block_of<D>(a.c, in ? pages[i] : 0, in ? j & page_mask : 0, head);
                const int left = k_end - j, skip = lo - j;  // tokens of the block that count: from skip on, below left
                if constexpr (D == 128) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int tok = tok8 + 8 * h;
                        kr[2 * i + h] = *reinterpret_cast<const uint4 *>(blk + tok * 64 + t * 16);
                        ks[2 * i + h] = *reinterpret_cast<const uint32_t *>(blk + 16 * D + tok * 4);
                    }
                } else {
                    kr[i] = *reinterpret_cast<const uint4 *>(blk + tok16 * 32 + (lane & 1) * 16);
                    ks[i] = *reinterpret_cast<const uint16_t *>(blk + 16 * D + tok16 * 2);
                }
#pragma unroll
                for (int q2 = 0; q2 < NV; ++q2) {
                    vr[q2][i] = *reinterpret_cast<const uint4 *>(blk + 8 * D + q2 * 512 + lane * 16);
                    const uint2 s = *reinterpret_cast<const uint2 *>(blk + 16 * D + D / 2 + t * (D / 8) + q2 * 8);
                    vs[q2][i][0] = s.x;
                    vs[q2][i][1] = s.y;
                }
                if (!in || left < BLOCK || skip > 0) {
                    // tokens that are not there, or that no row sees (their scales may be above the largest): K of scale
                    // byte 0, V of zero (bytes of scale 0, codes 0)
                    if constexpr (D == 128) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (!in || tok8 + 8 * h >= left || tok8 + 8 * h < skip) ks[2 * i + h] = 0;
                    } else {
                        if (!in || tok16 >= left || tok16 < skip) ks[i] = 0;
                    }
                    const uint32_t tk[4] = {2u * t, 2u * t + 1, 2u * t + 8, 2u * t + 9};
                    uint32_t keep = 0;
#pragma unroll
                    for (int x = 0; x < 4; ++x) keep |= (in && (int)tk[x] < left && (int)tk[x] >= skip ? 0xFFu : 0u) << (8 * x);
#pragma unroll
                    for (int q2 = 0; q2 < NV; ++q2) {
                        vs[q2][i][0] &= keep;
                        vs[q2][i][1] &= keep;
                        uint4 &v = vr[q2][i];
                        v = make_uint4(keep & 1u ? v.x : 0u, keep & 0x100u ? v.y : 0u, keep & 0x10000u ? v.z : 0u,
                                       keep & 0x1000000u ? v.w : 0u);
                    }
                }
            }
            return have;
        };
        const Weights k_weight(k_top), v_weight(v_top);
        const bool k_nan = sm.k_nan, v_nan = sm.v_nan;
        bool ok = true;
        uint32_t have = 0;
        if (steps > 0) {
            look(0);
            have = load(0);
            if (steps > 1) look(1);
        }
        for (int it = 0; it < steps; ++it) {
            const int s = it & 1;
            const uint32_t parity = ((uint32_t)(it >> 1) & 1u) ^ 1u;
            if (!mbar_wait(smem_u32(&sm.k_empty[s]), parity, a.wait_limit)) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            // K: eight codes of a word are 16 bytes of a row
#pragma unroll
            for (int p = 0; p < NK; ++p) {
                const uint32_t wd[4] = {kr[p].x, kr[p].y, kr[p].z, kr[p].w};
                const int tok = D == 128 ? (2 * w + (p >> 1)) * BLOCK + tok8 + 8 * (p & 1) : (2 * w + p) * BLOCK + tok16;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int G = D == 128 ? x : x & 1, piece = D == 128 ? t : 2 * (lane & 1) + (x >> 1);
                    uint32_t f = k_weight(__byte_perm(ks[p], 0, 0x4040 | G * 0x0101));
                    if (k_nan && (ks[p] >> (8 * G) & 255u) == 255u) f = 0x7E007E00u;
                    uint32_t h[4];
                    e2m1x8_to_f16(wd[x], h);
                    *reinterpret_cast<uint4 *>(&sm.k[s][G >> 1][tok * 128 + ((((G & 1) * 4 + piece) ^ (tok & 7)) << 4)]) =
                        make_uint4(mul_f16x2(h[0], f), mul_f16x2(h[1], f), mul_f16x2(h[2], f), mul_f16x2(h[3], f));
                }
            }
            fence_async();
            __syncwarp();
            if (lane == 0) {
                *(volatile uint8_t *)&sm.have[it & 3][w] = (uint8_t)have;
                mbar_arrive_plain(smem_u32(&sm.k_full[s]));
            }
            if (!mbar_wait(smem_u32(&sm.v_empty[s]), parity, a.wait_limit)) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (v_nan) {  // a block that is not a number counts as zero here; its rows are found at the end
#pragma unroll
                for (int q2 = 0; q2 < NV; ++q2)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) vs[q2][i][h] &= ~__vcmpeq4(vs[q2][i][h], 0xFFFFFFFFu);
            }
            // V: four tokens a block and eight channels a thread; two blocks make 16 bytes of a channel's row
#pragma unroll
            for (int q2 = 0; q2 < NV; ++q2) {
                uint32_t c0[2][4], c1[2][4], c2[2][4], c3[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 v = vr[q2][i];
                    e2m1x8_to_f16((v.x & 0x0F0F0F0Fu) | ((v.y << 4) & 0xF0F0F0F0u), c0[i]);
                    e2m1x8_to_f16(((v.x >> 4) & 0x0F0F0F0Fu) | (v.y & 0xF0F0F0F0u), c1[i]);
                    e2m1x8_to_f16((v.z & 0x0F0F0F0Fu) | ((v.w << 4) & 0xF0F0F0F0u), c2[i]);
                    e2m1x8_to_f16(((v.z >> 4) & 0x0F0F0F0Fu) | (v.w & 0xF0F0F0F0u), c3[i]);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t f[2][2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t x = vs[q2][i][h];
                        f[i][0] = v_weight(__byte_perm(x, 0, 0x4140));
                        f[i][1] = v_weight(__byte_perm(x, 0, 0x4342));
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int d = 64 * q2 + 32 * h + 4 * g + e, x = 2 * h + (e >> 1);
                        const uint4 o = make_uint4(
                            mul_f16x2(e & 1 ? c1[0][x] : c0[0][x], f[0][0]), mul_f16x2(e & 1 ? c3[0][x] : c2[0][x], f[0][1]),
                            mul_f16x2(e & 1 ? c1[1][x] : c0[1][x], f[1][0]), mul_f16x2(e & 1 ? c3[1][x] : c2[1][x], f[1][1]));
                        *reinterpret_cast<uint4 *>(&sm.v[s][w >> 1][d * 128 + ((((w & 1) * 4 + t) ^ (d & 7)) << 4)]) = o;
                    }
                }
            }
            if (it + 1 < steps) {
                have = load(it + 1);
                if (it + 2 < steps) look(it + 2);
            }
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive_plain(smem_u32(&sm.v_full[s]));
        }
        if (!ok && lane == 0) atomicOr(a.status, PQE_STATUS_TIMEOUT);
    } else {
        fewer_registers<MMA_REGS>();
        // ================= MMA =================
        q_barrier();
        if (warp == MMA_WARP && steps > 0) {
            tc_fence_after();
            const uint32_t one = elect();
            bool ok = true;
            auto wait = [&](uint32_t bar, uint32_t parity) {
                if (!mbar_wait(bar, parity, a.wait_limit)) ok = false;
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
                return ok;
            };
            const uint64_t q_desc = sw128_desc(smem_u32(sm.q[0][0])), k_desc = sw128_desc(smem_u32(sm.k[0][0])),
                           v_desc = sw128_desc(smem_u32(sm.v[0][0]));
            constexpr uint64_t QK_STAGE = sizeof(sm.k[0]) / 16, V_STAGE = sizeof(sm.v[0]) / 16;  // a tile of Q is as large
            const uint32_t k_full = smem_u32(&sm.k_full[0]), k_empty = smem_u32(&sm.k_empty[0]);
            const uint32_t v_full = smem_u32(&sm.v_full[0]), v_empty = smem_u32(&sm.v_empty[0]);
            const uint32_t s_full = smem_u32(&sm.s_full[0]), p_full = smem_u32(&sm.p_full[0]), o_full = smem_u32(&sm.o_full[0]);
            auto scores = [&](int tile, uint64_t k) {
                const uint64_t q = q_desc + tile * QK_STAGE;
                umma_ss<false>(one, tmem + s_col(tile), q, k, IDESC_S);
#pragma unroll
                for (int x = 1; x < D / 16; ++x) {
                    const uint64_t at = (x >> 2) * (CHUNK / 16) + (x & 3) * 2;
                    umma_ss<true>(one, tmem + s_col(tile), q + at, k + at, IDESC_S);
                }
                commit(one, s_full + 8 * tile);
            };
            if (wait(k_full, 0)) {
                scores(0, k_desc);
                if (tiles > 1) scores(1, k_desc);
                commit(one, k_empty);
            }
            for (int it = 0; it < steps && ok; ++it) {
                const int s = it & 1;
                const bool more = it + 1 < steps;
                const uint64_t v = v_desc + s * V_STAGE, k = k_desc + (s ^ 1) * QK_STAGE;
                if (!wait(v_full + 8 * s, (uint32_t)(it >> 1) & 1u)) break;
                if (more && !wait(k_full + 8 * (s ^ 1), (uint32_t)((it + 1) >> 1) & 1u)) break;
#pragma unroll
                for (int tile = 0; tile < TILES; ++tile) {
                    if (tile >= tiles) break;
                    if (!wait(p_full + 8 * tile, it & 1)) break;
#pragma unroll
                    for (int x = 0; x < BK / 16; ++x)
                        umma_ts(one, tmem + o_col(tile), tmem + p_col<D>(tile) + 8 * x,
                                v + (x >> 2) * (D * 128 / 16) + (x & 3) * 2, IDESC_O, x == 0 ? it != 0 : 1);
                    if (more)
                        scores(tile, k);
                    else
                        commit(one, o_full + 8 * tile);
                }
                if (!ok) break;
                commit(one, v_empty + 8 * s);
                if (more) commit(one, k_empty + 8 * (s ^ 1));
            }
            // every MMA has finished before TMEM is released
            commit(one, smem_u32(&sm.drained));
            if (!mbar_wait(smem_u32(&sm.drained), 0, DEFAULT_WAIT_LIMIT)) ok = false;  // whatever the limit of the others is
            if (!ok && lane == 0) atomicOr(a.status, PQE_STATUS_TIMEOUT);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// Joins the parts of a tile pair, 32 rows a CTA: a row per lane and an eighth of the channels per warp, then through shared
// memory so that rows go out whole.
template <int D>
__global__ void __launch_bounds__(256) prompt_join_kernel(const AttnArgs a, int splits, const float *parts) {
    constexpr int C4 = D / 32;  // groups of four channels that a warp takes
    __shared__ Find<256> find;
    __shared__ __align__(16) uint2 rows[32][D / 4 + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = a.n_q / a.c.n_kv;
    const int pair = blockIdx.x / a.c.n_kv, head = blockIdx.x % a.c.n_kv;
    // the call's own inputs were complete before the first kernel let this one start
    const int2 found = find_tiles<256>(a, pair, find);
    pdl_acquire();
    if (found.x < 0) return;
    int first, m, len;
    sequence_of(a, found.x, first, m, len);
    const int r0 = blockIdx.y * 32, row0 = found.y * ROWS + r0, n_rows = m * group;
    if (row0 >= n_rows) return;
    const float *p = parts + (size_t)blockIdx.x * splits * part_floats(D);
    float top = -INFINITY, l = 0.f;
    float4 o[C4];
#pragma unroll
    for (int x = 0; x < C4; ++x) o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < splits; ++s) top = fmaxf(top, p[(size_t)s * part_floats(D) + ROWS * D + r0 + lane]);
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
        const float *q = p + (size_t)s * part_floats(D);
        const float f = exp2_approx(q[ROWS * D + r0 + lane] - base);
        l = fmaf(q[ROWS * D + ROWS + r0 + lane], f, l);
#pragma unroll
        for (int x = 0; x < C4; ++x) {
            const float4 v = reinterpret_cast<const float4 *>(q)[(warp * C4 + x) * ROWS + r0 + lane];
            o[x].x = fmaf(v.x, f, o[x].x), o[x].y = fmaf(v.y, f, o[x].y);
            o[x].z = fmaf(v.z, f, o[x].z), o[x].w = fmaf(v.w, f, o[x].w);
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int x = 0; x < C4; ++x) {
        uint2 u;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.x) : "f"(o[x].y * inv), "f"(o[x].x * inv));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.y) : "f"(o[x].w * inv), "f"(o[x].z * inv));
        rows[lane][warp * C4 + x] = u;
    }
    if (warp == 0 && a.lse && row0 + lane < n_rows) {
        const int row = row0 + lane;
        a.lse[(int64_t)(first + row / group) * a.n_q + head * group + row % group] =
            l == 0.f ? -INFINITY : (top + log2f(l) - 8.f) * 0.693147180559945309f;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * (D / 4); i += 256) {
        const int row = row0 + i / (D / 4), c = i % (D / 4);
        if (row < n_rows)
            reinterpret_cast<uint2 *>(a.out + ((int64_t)(first + row / group) * a.n_q + head * group + row % group) * D)[c] =
                rows[i / (D / 4)][c];
    }
}

// No sequence has more tile pairs than its rows fill, and one that they do not: a bound that needs no lengths.
int64_t pairs_bound(int B, int total_q, int n_q, int n_kv) {
    return ((int64_t)total_q * (n_q / n_kv) / ROWS + B) * n_kv;
}

template <int D, bool SPLIT>
int launch(const AttnArgs &a, int splits, void *ws, cudaStream_t s) {
    static bool set[PQE_MAX_DEVICES] = {};
    int dev = 0, n = 0;
    int rc = device_info(dev, n);
    if (rc != PQE_OK) return rc;
    constexpr int smem = (int)sizeof(Smem<D>) + 1024;
    if (!set[dev]) {
        // the split of the registers waits forever where the block is launched with fewer than it counts on
        cudaFuncAttributes at;
        PQE_CUDA_TRY(cudaFuncGetAttributes(&at, attn_prompt_kernel<D, SPLIT>));
        if (at.numRegs != LAUNCH_REGS) return PQE_ERR_UNSUPPORTED;
        PQE_CUDA_TRY(cudaFuncSetAttribute(attn_prompt_kernel<D, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
        set[dev] = true;
    }
    const int64_t ctas = pairs_bound(a.B, a.total_q, a.n_q, a.c.n_kv);
    PQE_CHECK_ARG(ctas * splits <= INT32_MAX);
    rc = launch_pdl(attn_prompt_kernel<D, SPLIT>, dim3((unsigned)(ctas * splits)), dim3(THREADS), smem, s, a, splits,
                    static_cast<float *>(ws));
    if (rc != PQE_OK || !SPLIT) return rc;
    return launch_pdl(prompt_join_kernel<D>, dim3((unsigned)ctas, ROWS / 32), dim3(256), 0, s, a, splits,
                      static_cast<const float *>(ws));
}

}  // namespace prompt

// Parts that a tile pair is cut into: so many that all of them have an SM, of three steps or more at the longest cache.
int prompt_splits(int B, int total_q, int n_q, int n_kv, int64_t tokens, int sms) {
    const int64_t pairs = prompt::pairs_bound(B, total_q, n_q, n_kv), by_steps = tokens / (3 * prompt::BK);
    int64_t n = pairs > 0 ? sms / pairs : 1;
    if (n > by_steps) n = by_steps;
    return n < 1 ? 1 : n > 16 ? 16 : (int)n;
}

size_t attn_prompt_ws(int B, int total_q, int n_q, int n_kv, int d, int sms) {
    const int splits = prompt_splits(B, total_q, n_q, n_kv, INT64_MAX, sms);
    if (splits == 1) return 256;
    return (size_t)prompt::pairs_bound(B, total_q, n_q, n_kv) * splits * prompt::part_floats(d) * sizeof(float);
}

int attn_prompt(const pqe_kv_cache *cache, const AttnArgs &a, int splits, void *ws, cudaStream_t s) {
    if (cache->d == 128) return splits > 1 ? prompt::launch<128, true>(a, splits, ws, s) : prompt::launch<128, false>(a, 1, ws, s);
    return splits > 1 ? prompt::launch<64, true>(a, splits, ws, s) : prompt::launch<64, false>(a, 1, ws, s);
}

}  // namespace kv
}  // namespace pqe
