// kv_attn_split.cu -- attention over the 4-bit paged cache for few query rows
// (single tokens, a few tokens at once), split along the cache.
//
// For one sequence and KV head the R = m * group query rows form the N side of
// mma.sync m16n8k16 (f16 in, fp32 sums): S^T[token, row] = K . Q^T with 16
// tokens as M, then O^T[d, row] = V^T . P^T with 16 channels as M, so 8 rows
// fill a tile that 16-row forms would leave half empty. Per tile of 64 tokens:
//   S[j, r]  = sum_G 2^(ks[j, G]) * (codes of block G . q)   K scales in fp32,
//              after each 32-channel block's two MMAs: codes enter as they are
//   p        = 2^(c_r (S - m_r) + 8), running maximum m_r, sum l_r
//   O[d, r] += code[j, d] * (p * 2^(vs[j, G] - top + 7)), top the largest V scale
//              of the tiles so far: p and the factor stay inside f16, O in fp32
// and O is scaled when a maximum or top has grown, which is rare after the
// first tiles. (top is common to the rows of a set. Where some of them see a V
// far above what the others see, the set's rows are summed one by one in fp32.)
// P^T's fragments come from S^T's by movmatrix, with no trip through memory.
//
// The cache is read once. Work is (sequence, KV head, 8 * NT rows, tile); all of
// it in one line is cut into equal shares, one per warp of the grid, whatever
// the lengths are (they are read on the device). A warp fetches its tiles
// with bulk copies into its own ring of shared memory, two ahead; it meets no
// other warp. A (sequence, head, rows) that lies in one share
// goes straight out; of one that shares divide between them each leaves a
// partial in the workspace, two at most, and a second kernel joins them in the
// order of the cache.
//
// Bound by the cache's bytes when there are many (4.25 bits a value), by latency
// when there are few. 64 sequences of 1 to 8192 tokens (4 KV heads of 128, 16
// query heads, 146 MB): 39.8 us, 3.7 TB/s; 3 of 60001 to 131071 (20 heads): 42.6 us,
// 3.7 TB/s; one of 517: 8.4 us. Of the 42: 1.5 to set up, 5 until a warp has its
// first tile, 24.5 of walking them (a warp's share takes 20 to 29), 5 for the join,
// the rest launches and tails. Within the walk no pipe is full (issue 47%, ALU 45%,
// MMA 24%): a warp's tile is a chain of some 2 us, and registers leave room for 12
// to 16 warps an SM.
#include <math.h>

#include "kv_attn_plain.cuh"
#include "tc_ptx.cuh"

namespace pqe {
namespace kv {
namespace split {
using namespace ptx;

constexpr int WARPS = 4;
constexpr int STAGES = 2;
constexpr int TB = TILE / BLOCK;  // blocks of a tile
constexpr uint32_t ALL = (1u << TB) - 1;

template <int D>
constexpr int tile_bytes() {
    return TILE / BLOCK * block_bytes(D);
}
// CTAs an SM: what the registers of a warp leave room for. (Heads of 64, one row tile, 4 against 3: 64 sequences of 4000: 39.4
// us, 40.3; 16 of 1000: 8.7, 10.3. Heads of 128 spill 32 bytes at 3, and 160 at 4.)
__host__ __device__ constexpr int ctas(int d, int nt) { return nt == 1 ? (d == 64 ? 4 : 3) : 2; }
// one partial result: O [rows][D], m [rows], l [rows], all fp32
__host__ __device__ constexpr int part_floats(int d, int rows) { return rows * (d + 2); }

// Beginning and ending a (sequence, head, rows) costs about as much as two tiles: it counts as two in the line of work, before
// its first tile. (64 sequences of 1 to 8192 tokens: 40.4 us with one, 39.3 with two; five rows of four heads over windows of
// 1024: 24.5 and 22.3 us.)
constexpr int OPEN = 2;

// a sequence's part of the line of work
struct Seq {
    int first, m, len, lo, t0, T, nrc;  // lo: the first token that any of its queries sees
    __device__ __forceinline__ int64_t units(int n_kv) const { return T > 0 ? (int64_t)(T + OPEN) * nrc * n_kv : 0; }
};
template <int NT>
__device__ __forceinline__ Seq load_seq(const AttnArgs &a, int b, int group) {
    Seq s;
    sequence_of(a, b, s.first, s.m, s.len);
    s.nrc = (s.m * group + 8 * NT - 1) / (8 * NT);
    int hi;
    visible(a, 0, s.m, s.len, s.lo, hi);
    s.t0 = min(s.lo, s.len) / TILE;
    s.T = is_ours(a, s.m) ? (s.len + TILE - 1) / TILE - s.t0 : 0;
    return s;
}

struct Cursor {
    int b, head, chunk, tile;  // tile counts from the sequence's t0
    Seq s;
};
template <int NT>
__device__ __forceinline__ void next_rows(const AttnArgs &a, Cursor &c, int group) {
    c.tile = 0;
    if (++c.chunk < c.s.nrc) return;
    c.chunk = 0;
    if (++c.head < a.c.n_kv) return;
    c.head = 0;
    while (++c.b < a.B) {
        c.s = load_seq<NT>(a, c.b, group);
        if (c.s.T > 0) return;
    }
}

// Exponents of two (c m of a row) above which p's, c S - c m, is not right as one fma: c m, rounded, is off by a part of its own
// size, which from 2^27 or so on is all of p's exponent. A set of rows with such scores is left to plain_rows().
constexpr float FAR = 1 << 20;

// what a tile's scale bytes become for the MMAs' lanes
template <int D>
struct alignas(16) Factors {
    float k[TILE][D / 32];        // [token][block]: 2^(scale - 127)
    uint32_t v[TB][4][D / 32][2];  // [16 tokens][t][block]: f16 pairs for tokens 2t, 2t+1 and 2t+8, 2t+9
    uint32_t far;                  // not 0: some row's maximum was above FAR
};

template <int D, int NT>
struct Smem {
    alignas(16) uint8_t ring[WARPS][STAGES][tile_bytes<D>()];
    alignas(16) Factors<D> fac[WARPS];
    alignas(8) uint64_t full[WARPS][STAGES];
    Cursor at[WARPS], ahead[WARPS];  // the rows at hand, and those that tiles are fetched for
    int64_t scan[WARPS];
    int64_t share[WARPS + 1];  // units at which the warps' shares begin
    int64_t first[WARPS];      // unit at which the sequence begins that a share begins in
};

static_assert(sizeof(Factors<64>) % 16 == 0 && sizeof(Factors<128>) % 16 == 0, "a warp's factors are read 16 bytes at a time");

// shares that `total` units are cut into: at least one unit each
__host__ __device__ __forceinline__ int64_t shares(int64_t total, int ctas) {
    const int64_t most = (int64_t)ctas * WARPS;
    return total < most ? (total > 0 ? total : 1) : most;
}
// unit at which share i of n begins, of `total` units
__device__ __forceinline__ int64_t share_start(int64_t i, int64_t n, int64_t total) { return i * total / n; }
// the share that unit u falls into
__device__ __forceinline__ int64_t share_of(int64_t u, int64_t n, int64_t total) { return ((u + 1) * n - 1) / total; }

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the same into zeros
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// What fetching needs of a cursor (the rest of it waits in shared memory), and of the lane: lane i of the first few copies the
// blocks from blk on, of one page.
struct Feed {
    const int32_t *table;  // the sequence's
    const uint8_t *head;   // the head's part of page 0
    int j, len, lo;        // j: the first token that the lane copies; of a lane that copies none, below zero, however far it goes
};
__device__ __forceinline__ int blocks_shift(const AttnArgs &a) { return min(a.c.page_shift - 4, TB == 4 ? 2 : 1); }
template <int D>
__device__ __forceinline__ Feed feed_of(const AttnArgs &a, const Cursor &c, int lane) {
    const int blk = lane << blocks_shift(a);
    return {a.block_table + (size_t)c.b * a.max_pages, block_of<D>(a.c, 0, 0, c.head),
            blk < TB ? (c.s.t0 + c.tile) * TILE + blk * BLOCK : INT32_MIN, c.s.len, c.s.lo};
}

// The table entry that this lane's copy of the tile needs. Asked for a tile early, so that fetch() does not wait.
__device__ __forceinline__ int table_entry(const AttnArgs &a, const Feed &f) {
    if ((uint32_t)f.j >= (uint32_t)f.len) return -3;           // no tokens, or not a lane that copies
    if (f.j + (BLOCK << blocks_shift(a)) <= f.lo) return -2;  // before the window: the page may be gone
    return max(f.table[f.j >> a.c.page_shift], -1);
}

// Starts the copies of a tile into a stage; returns the bit mask of its 16-token
// blocks that the stage will hold (a block of a bad page, or past the end, is
// not there).
template <int D>
__device__ __forceinline__ uint32_t fetch(const AttnArgs &a, const Feed &f, int page, uint32_t dst, uint32_t bar, int lane) {
    const int sh = blocks_shift(a), copies = TB >> sh;  // lanes that copy
    const bool good = (uint32_t)page < (uint32_t)a.c.n_pages;
    const uint8_t *src = f.head + (size_t)(uint32_t)page * a.c.page_stride +
                         ((f.j & ((1 << a.c.page_shift) - 1)) >> 4) * block_bytes(D);
    dst += (lane << sh) * block_bytes(D);
    if (__all_sync(0xffffffffu, lane >= copies || (good && f.j + (BLOCK << sh) <= f.len))) {
        if (lane == 0) mbar_expect_tx(bar, TB * block_bytes(D));
        __syncwarp();
        if (lane < copies) bulk_copy(dst, src, block_bytes(D) << sh, bar);
        return ALL;
    }
    uint32_t n = 0;  // blocks that this lane copies
    if (good)
        n = min(1 << sh, (f.len - f.j + BLOCK - 1) / BLOCK);
    else if (page == -1 || page >= a.c.n_pages)
        atomicOr(a.status, PQE_STATUS_BAD_PAGE);
    const uint32_t mask = __reduce_or_sync(0xffffffffu, n ? ((1u << n) - 1) << (lane << sh) : 0u);
    if (lane == 0) mbar_expect_tx(bar, __popc(mask) * block_bytes(D));
    __syncwarp();
    if (n) bulk_copy(dst, src, n * block_bytes(D), bar);
    return mask;
}

// row r of a (sequence, head, chunk): its place in q, out and lse
__device__ __forceinline__ int64_t row_index(const AttnArgs &a, const Seq &s, int head, int group, int r) {
    return (int64_t)(s.first + r / group) * a.n_q + head * group + r % group;
}

// Bits of the 32 tokens from j on that lie in [lo, hi).
__device__ __forceinline__ uint32_t tokens_in(int j, int lo, int hi) {
    const int from = min(max(lo - j, 0), 32), to = min(max(hi - j, 0), 32);
    return (to < 32 ? (1u << to) - 1u : 0xFFFFFFFFu) & ~(from < 32 ? (1u << from) - 1u : 0xFFFFFFFFu);
}

// The rows of one (sequence, KV head, chunk) while its tiles pass.
template <int D, int NT>
struct Rows {
    uint32_t q[NT][D / 32][4];  // B fragments: row 8 * nt + g, channels 32 * G + 8 * t ..
    float c[NT][2];             // of rows 8 * nt + 2 * t, + 1: the factor (above 0) from S to an exponent of two
    int lo[NT][2], hi[NT][2];   // and the tokens they see
    int min_lo, max_lo, min_hi, max_hi;
    float m[NT][2], l[NT][2];   // m: of S; l: this lane's tokens only
    uint32_t top;               // the E8M0 byte that o is in units of (2^-15 more): the largest that some row sees
    uint32_t all, least;        // the largest among tokens that all rows see; the smallest token's that only some see
    float o[D / 32][2][NT][4];  // O^T: block G, channels 4g + {0, 1} and 4g + {2, 3}
};

template <int D, int NT>
__device__ __forceinline__ void begin_rows(const AttnArgs &a, const Cursor &c, int group, int lane, Rows<D, NT> &R) {
    const int g = lane >> 2, t = lane & 3;
    const int head = c.head, r0 = c.chunk * 8 * NT, n = c.s.m * group;
    R.top = R.all = 0;
    R.least = 255;
    R.min_lo = R.min_hi = INT32_MAX;
    R.max_lo = R.max_hi = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = r0 + 8 * nt + g;
        uint4 raw[D / 32];
        uint32_t top = 0;
        int lo = 0, hi = 0;
        if (r < n) {
            const uint16_t *row = a.q + (int64_t)(c.s.first + r / group) * a.q_stride + (head * group + r % group) * D;
            visible(a, r / group, c.s.m, c.s.len, lo, hi);
#pragma unroll
            for (int G = 0; G < D / 32; ++G) raw[G] = *reinterpret_cast<const uint4 *>(row + 32 * G + 8 * t);
            R.min_lo = min(R.min_lo, lo);
            R.max_lo = max(R.max_lo, lo);
            R.min_hi = min(R.min_hi, hi);
            R.max_hi = max(R.max_hi, hi);
        } else {
#pragma unroll
            for (int G = 0; G < D / 32; ++G) raw[G] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int G = 0; G < D / 32; ++G) {
            const uint32_t w[4] = {raw[G].x, raw[G].y, raw[G].z, raw[G].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float f, inv;
        q_factor(top, f, inv);
        inv *= fabsf(a.scale);
        if (a.scale < 0.f) f = -f;
        if (inv == 0.f) f = 0.f, inv = 1.f;                       // scores of zero
        if (top >= 0x7F80u) f = __uint_as_float(0x7FC00000u);  // a row that is not finite: scores of NaN
#pragma unroll
        for (int G = 0; G < D / 32; ++G) {
            const uint32_t w[4] = {raw[G].x, raw[G].y, raw[G].z, raw[G].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                R.q[nt][G][i] = pack_f16(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xFFFF0000u) * f);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int src = (2 * t + i) * 4;  // a lane that holds row 8 * nt + 2 * t + i
            R.c[nt][i] = __shfl_sync(0xffffffffu, inv, src);
            R.lo[nt][i] = __shfl_sync(0xffffffffu, lo, src);
            R.hi[nt][i] = __shfl_sync(0xffffffffu, hi, src);
            R.m[nt][i] = -INFINITY;
            R.l[nt][i] = 0.f;
        }
    }
    R.min_lo = __reduce_min_sync(0xffffffffu, R.min_lo);
    R.max_lo = __reduce_max_sync(0xffffffffu, R.max_lo);
    R.min_hi = __reduce_min_sync(0xffffffffu, R.min_hi);
    R.max_hi = __reduce_max_sync(0xffffffffu, R.max_hi);
#pragma unroll
    for (int G = 0; G < D / 32; ++G)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) R.o[G][h][nt][i] = 0.f;
}

// O of the rows that see a token whose V block is not a number turns to NaN in that block's channels, whatever weight the
// token has, and stays it. (Bytes of tokens that are not there, or that no row sees, are 0 by now.)
template <int D, int NT>
__device__ __forceinline__ void add_nans(const uint8_t *tile, int j0, int lane, Rows<D, NT> &R) {
#pragma unroll
    for (int G = 0; G < D / 32; ++G)
#pragma unroll
        for (int h = 0; h < TILE; h += 32) {
            const uint32_t bad =
                __ballot_sync(0xffffffffu, tile[((h + lane) >> 4) * block_bytes(D) + v_scale<D>(lane & 15, G)] == 255);
            if (!bad) continue;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (bad & tokens_in(j0 + h, R.lo[nt][i], R.hi[nt][i]))
                        R.o[G][0][nt][i] = R.o[G][0][nt][i + 2] = R.o[G][1][nt][i] = R.o[G][1][nt][i + 2] =
                            __uint_as_float(0x7FC00000u);
        }
}

// O += codes . (p * factors) of one tile
template <int D, int NT>
__device__ __forceinline__ void add_values(const uint8_t *tile, const Factors<D> &fac, int lane,
                                           const uint32_t (&p)[TB][NT][2], Rows<D, NT> &R) {
    const int t = lane & 3;
#pragma unroll
    for (int q2 = 0; q2 < D / 64; ++q2) {
#pragma unroll
        for (int mt = 0; mt < TB; ++mt) {
            // four tokens (2t, 2t+1, 2t+8, 2t+9) x channels 4g.. of two blocks
            const uint4 w = *reinterpret_cast<const uint4 *>(tile + mt * block_bytes(D) + 8 * D + q2 * 512 + lane * 16);
            const uint4 vf = *reinterpret_cast<const uint4 *>(fac.v[mt][t][2 * q2]);
            uint32_t a0[4], a1[4], a2[4], a3[4];
            e2m1x8_to_f16((w.x & 0x0F0F0F0Fu) | ((w.y << 4) & 0xF0F0F0F0u), a0);  // token pairs of the even channels
            e2m1x8_to_f16(((w.x >> 4) & 0x0F0F0F0Fu) | (w.y & 0xF0F0F0F0u), a1);  // and of the odd ones
            e2m1x8_to_f16((w.z & 0x0F0F0F0Fu) | ((w.w << 4) & 0xF0F0F0F0u), a2);
            e2m1x8_to_f16(((w.z >> 4) & 0x0F0F0F0Fu) | (w.w & 0xF0F0F0F0u), a3);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t f0 = h ? vf.z : vf.x, f1 = h ? vf.w : vf.y;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint32_t b0 = mul_f16x2(p[mt][nt][0], f0), b1 = mul_f16x2(p[mt][nt][1], f1);
                    mma_f16(R.o[2 * q2 + h][0][nt], a0[2 * h], a1[2 * h], a2[2 * h], a3[2 * h], b0, b1);
                    mma_f16(R.o[2 * q2 + h][1][nt], a0[2 * h + 1], a1[2 * h + 1], a2[2 * h + 1], a3[2 * h + 1], b0, b1);
                }
            }
        }
    }
}

// One tile: scores, softmax step, values. have: the 16-token blocks that are there.
template <int D, int NT>
__device__ __forceinline__ void add_tile(uint8_t *tile, Factors<D> &fac, int j0, uint32_t have, int lane, Rows<D, NT> &R) {
    const int g = lane >> 2, t = lane & 3;
    const bool part = have != ALL || j0 + TILE > R.min_hi || j0 < R.max_lo;  // some row does not see all of it
    if (part) {
        // V of tokens that no row sees may hold anything: scale bytes of zero
        uint32_t all = 0, least = 255;
#pragma unroll 1
        for (int i = lane; i < TILE; i += 32) {
            const int j = j0 + i;
            const bool seen = have >> (i >> 4) & 1 && j < R.max_hi && j >= R.min_lo;
            uint32_t most = 0;
#pragma unroll
            for (int G = 0; G < D / 32; ++G) {
                uint8_t &x = tile[(i >> 4) * block_bytes(D) + v_scale<D>(i & 15, G)];
                if (!seen) x = 0;
                most = max(most, x == 255 ? 0u : (uint32_t)x);
            }
            if (j >= R.max_lo && j < R.min_hi)
                all = max(all, most);
            else if (most)
                least = min(least, most);
        }
        R.all = max(R.all, __reduce_max_sync(0xffffffffu, all));
        R.least = min(R.least, __reduce_min_sync(0xffffffffu, least));
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the next copy into this stage
        __syncwarp();
    }
    // The scale bytes as the factors that the lanes take. Each would otherwise be made by the four lanes (K) or eight
    // (V) that use it, on the integer pipe that the code conversions fill.
    uint32_t top = 0;
    bool nans;
    {
#pragma unroll
        for (int h = 0; h < TILE / 32; ++h) {
            // of tokens lane and lane + 32
            const uint8_t *at = tile + ((lane >> 4) + 2 * h) * block_bytes(D) + 16 * D + (lane & 15) * (D / 32);
            const uint32_t w = D == 128 ? *reinterpret_cast<const uint32_t *>(at) : *reinterpret_cast<const uint16_t *>(at);
            float f[D / 32];
            // byte into the exponent; 0 gives 0
#pragma unroll
            for (int G = 0; G < D / 32; ++G) f[G] = __uint_as_float(w << (G < 3 ? 23 - 8 * G : 0) >> (G < 3 ? 0 : 1) & 0x7F800000u);
            if (w & 0x80808080u & ((w & 0x7F7F7F7Fu) + 0x01010101u))  // some byte is 255
#pragma unroll
                for (int G = 0; G < D / 32; ++G)
                    if ((w >> (8 * G) & 255u) == 255u) f[G] = __uint_as_float(0x7FC00000u);
            if constexpr (D == 128)
                *reinterpret_cast<float4 *>(fac.k[lane + 32 * h]) = make_float4(f[0], f[1], f[2], f[3]);
            else
                *reinterpret_cast<float2 *>(fac.k[lane + 32 * h]) = make_float2(f[0], f[1]);
        }
        // V: words [16 tokens][t][block] of four tokens' scales, WORDS a lane
        constexpr int WORDS = TB * (D / 32) / 8;
        uint32_t w[WORDS], two = 0;
        const uint8_t *vs = tile + lane * WORDS / (D / 8) * block_bytes(D) + 16 * D + D / 2 + lane * WORDS % (D / 8) * 4;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            w[i] = *reinterpret_cast<const uint32_t *>(vs + 4 * i);
            two = __vmaxu2(two, __vmaxu2(w[i] & 0x00FF00FFu, (w[i] >> 8) & 0x00FF00FFu));
        }
        top = __reduce_max_sync(0xffffffffu, max(two & 0xFFFFu, two >> 16));
        nans = top == 255;
        if (nans) {  // a block that is not a number counts as one of zeros; its rows are found below
            top = 0;
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                w[i] &= ~__vcmpeq4(w[i], 0xFFFFFFFFu);
#pragma unroll
                for (int j = 0; j < 32; j += 8) top = max(top, w[i] >> j & 255u);
            }
            top = __reduce_max_sync(0xffffffffu, top);
        }
        if (!part) R.all = max(R.all, top);
        top = max(top, R.top);
        // f16 pairs of 2^(scale - top + 7): 0 from 22 below top on
        const uint32_t least = (uint32_t)max((int)top - 22, 0) * 0x10001u, off = (uint32_t)((int)top - 22) * (1024u * 0x10001u);
        uint32_t o[2 * WORDS];
#pragma unroll
        for (int i = 0; i < 2 * WORDS; ++i)
            o[i] = __vmaxu2(__byte_perm(w[i >> 1], 0, i & 1 ? 0x4342 : 0x4140), least) * 1024u - off;
        uint32_t *vf = &fac.v[0][0][0][0] + lane * 2 * WORDS;
        if constexpr (WORDS == 2)
            *reinterpret_cast<uint4 *>(vf) = make_uint4(o[0], o[1], o[2], o[3]);
        else
            *reinterpret_cast<uint2 *>(vf) = make_uint2(o[0], o[1]);
    }
    __syncwarp();
    float x[TB][NT][4];  // S^T, then exponents, then p: tokens 16 * mt + g (+ 8), rows 8 * nt + 2t (+ 1)
#pragma unroll
    for (int mt = 0; mt < TB; ++mt) {
        const uint8_t *blk = tile + mt * block_bytes(D);
        uint32_t k0[D / 32], k1[D / 32];
        float f0[D / 32], f1[D / 32];
        if constexpr (D == 128) {
            const uint4 u = *reinterpret_cast<const uint4 *>(blk + g * 64 + t * 16);
            const uint4 v = *reinterpret_cast<const uint4 *>(blk + (g + 8) * 64 + t * 16);
            k0[0] = u.x, k0[1] = u.y, k0[2] = u.z, k0[3] = u.w;
            k1[0] = v.x, k1[1] = v.y, k1[2] = v.z, k1[3] = v.w;
            const float4 a = *reinterpret_cast<const float4 *>(fac.k[16 * mt + g]);
            const float4 b = *reinterpret_cast<const float4 *>(fac.k[16 * mt + g + 8]);
            f0[0] = a.x, f0[1] = a.y, f0[2] = a.z, f0[3] = a.w;
            f1[0] = b.x, f1[1] = b.y, f1[2] = b.z, f1[3] = b.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(blk + g * 32 + t * 8);
            const uint2 v = *reinterpret_cast<const uint2 *>(blk + (g + 8) * 32 + t * 8);
            k0[0] = u.x, k0[1] = u.y;
            k1[0] = v.x, k1[1] = v.y;
            const float2 a = *reinterpret_cast<const float2 *>(fac.k[16 * mt + g]);
            const float2 b = *reinterpret_cast<const float2 *>(fac.k[16 * mt + g + 8]);
            f0[0] = a.x, f0[1] = a.y;
            f1[0] = b.x, f1[1] = b.y;
        }
#pragma unroll
        for (int G = 0; G < D / 32; ++G) {
            uint32_t a[4], b[4];
            e2m1x8_to_f16(k0[G], a);
            e2m1x8_to_f16(k1[G], b);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float d[4];
                mma_f16_first(d, a[0], b[0], a[1], b[1], R.q[nt][G][0], R.q[nt][G][1]);
                mma_f16(d, a[2], b[2], a[3], b[3], R.q[nt][G][2], R.q[nt][G][3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = i < 2 ? f0[G] : f1[G];
                    x[mt][nt][i] = G == 0 ? d[i] * f : fmaf(d[i], f, x[mt][nt][i]);
                }
            }
        }
    }
    if (part) {
#pragma unroll
        for (int mt = 0; mt < TB; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = j0 + 16 * mt + g + 8 * (i >> 1);
                    if (!(have >> mt & 1) || j >= R.hi[nt][i & 1] || j < R.lo[nt][i & 1]) x[mt][nt][i] = -INFINITY;
                }
    }
    // the running maximum; rows' values lie in the eight lanes of equal t
    float keep[NT][2];
    bool moved = top != R.top;
    const float shrink = moved ? exp2_approx((float)(int)(R.top - top)) : 1.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float m = R.m[nt][i];
#pragma unroll
            for (int mt = 0; mt < TB; ++mt) m = fmaxf(m, fmaxf(x[mt][nt][i], x[mt][nt][i + 2]));
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float c = R.c[nt][i], base = m == -INFINITY ? -8.f : fmaf(m, c, -8.f);
            const float k = m == R.m[nt][i] ? 1.f : exp2_approx((R.m[nt][i] - m) * c);
            moved |= k != 1.f;
            keep[nt][i] = k * shrink;
            R.m[nt][i] = m;
            float sum = 0.f;
#pragma unroll
            for (int mt = 0; mt < TB; ++mt)
#pragma unroll
                for (int h = 0; h < 4; h += 2) {
                    const float p = exp2_approx(fmaf(x[mt][nt][i + h], c, -base));
                    x[mt][nt][i + h] = p;
                    sum += p;
                }
            R.l[nt][i] = fmaf(R.l[nt][i], k, sum);
        }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int G = 0; G < D / 32; ++G)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) R.o[G][e][nt][i] *= keep[nt][i & 1];
        R.top = top;
        bool far = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) far |= R.m[nt][i] != -INFINITY && fabsf(R.m[nt][i] * R.c[nt][i]) > FAR;
        if (far) fac.far = 1;
    }
    uint32_t p[TB][NT][2];
#pragma unroll
    for (int mt = 0; mt < TB; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            p[mt][nt][0] = transpose8x8(pack_f16(x[mt][nt][0], x[mt][nt][1]));
            p[mt][nt][1] = transpose8x8(pack_f16(x[mt][nt][2], x[mt][nt][3]));
        }
    add_values<D, NT>(tile, fac, lane, p, R);
    if (nans) add_nans<D, NT>(tile, j0, lane, R);
    __syncwarp();  // before the factors of the next tile
}

// four channels of a row's result, and its lse
__device__ __forceinline__ void store_out(const AttnArgs &a, int64_t row, int D, int d, const float4 &o, float m, float l) {
    const float inv = l == 0.f ? 0.f : 256.f / l;
    uint2 u;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.x) : "f"(o.y * inv), "f"(o.x * inv));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.y) : "f"(o.w * inv), "f"(o.z * inv));
    *reinterpret_cast<uint2 *>(a.out + row * D + d) = u;
    if (a.lse && d == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l) - 8.f) * 0.693147180559945309f;
}

// The end of a piece: l summed over the lanes; the rows go out if the piece was all of them, else into a partial.
template <int D, int NT>
__device__ __forceinline__ void end_rows(const AttnArgs &a, const Cursor &c, int group, int lane, Rows<D, NT> &R,
                                         bool whole, float *part) {
    const int g = lane >> 2, t = lane & 3;
    const int head = c.head, r0 = c.chunk * 8 * NT, n = c.s.m * group;
    const float back = v_factor(R.top);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float m = R.m[nt][i] == -INFINITY ? -INFINITY : R.m[nt][i] * R.c[nt][i];
            float l = R.l[nt][i];
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            const int r = 8 * nt + 2 * t + i;
            if (whole && r0 + r >= n) continue;
            const int64_t row = whole ? row_index(a, c.s, head, group, r0 + r) : 0;
#pragma unroll
            for (int G = 0; G < D / 32; ++G) {
                const float4 o = make_float4(R.o[G][0][nt][i] * back, R.o[G][0][nt][i + 2] * back,
                                             R.o[G][1][nt][i] * back, R.o[G][1][nt][i + 2] * back);
                if (whole)
                    store_out(a, row, D, 32 * G + 4 * g, o, m, l);
                else
                    *reinterpret_cast<float4 *>(part + r * D + 32 * G + 4 * g) = o;
            }
            if (!whole && g == 0) {
                part[8 * NT * D + r] = m;
                part[8 * NT * D + 8 * NT + r] = l;
            }
        }
}

// V scales further apart than this, between what some row of a set sees and what another does, are left to plain_rows() (five
// rows over a window of 1024: 23.0 us with the test for it, 22.4 without; single tokens: no difference). The
// products of p and V's factors then hold 2^-32 of a row's largest p, and V blocks 13 below the largest that the row sees.
constexpr uint32_t APART = 8;
// Whether every row of the piece over tokens [from, to) sees a V scale near the largest of all: each sees the tokens that all see,
// if there are any, else one of the others at least.
template <int D, int NT>
__device__ __forceinline__ bool alike(const Rows<D, NT> &R, int from, int to) {
    if (R.min_lo == R.max_lo && R.min_hi == R.max_hi) return true;  // they see the same tokens
    return R.top <= (max(R.max_lo, from) < min(R.min_hi, to) ? R.all : R.least) + APART;
}

// end_rows() for rows that are not: each by itself, from the cache
template <int D, int NT>
__device__ __noinline__ void plain_rows(const AttnArgs a, const Cursor c, int from, int to, bool whole, float *part) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, group = a.n_q / a.c.n_kv, r0 = c.chunk * 8 * NT;
    for (int r = 0; r < 8 * NT && r0 + r < c.s.m * group; ++r) {
        int lo, hi;
        visible(a, (r0 + r) / group, c.s.m, c.s.len, lo, hi);
        const int head = c.head * group + (r0 + r) % group;
        const PlainRow<D> x = plain_row<D>(a.c, a.block_table + (size_t)c.b * a.max_pages, c.head,
                                           a.q + (int64_t)(c.s.first + (r0 + r) / group) * a.q_stride + head * D, a.scale,
                                           max(lo, from), min(hi, to));
        const int64_t row = whole ? row_index(a, c.s, c.head, group, r0 + r) : 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (whole)
                a.out[row * D + lane * E + e] = f32_to_bf16_rn(x.l == 0.f ? 0.f : x.o[e] / x.l);
            else
                part[r * D + lane * E + e] = x.o[e];
        }
        if (lane == 0) {  // l in units of 2^-8, as the rows' own
            if (!whole) {
                part[8 * NT * D + r] = x.m;
                part[8 * NT * D + 8 * NT + r] = x.l * 256.f;
            } else if (a.lse) {
                a.lse[row] = x.l == 0.f ? -INFINITY : (x.m + log2f(x.l)) * 0.693147180559945309f;
            }
        }
    }
}

// Workspace: prefix [B + 1] of the sequences' units, then two partials per warp
__host__ __device__ inline size_t prefix_bytes(int B) { return round_up(((size_t)B + 1) * 8, 256); }

template <int D, int NT>
__global__ void __launch_bounds__(WARPS * 32, ctas(D, NT)) attn_split_kernel(const AttnArgs a, uint8_t *ws) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    auto &sm = *reinterpret_cast<Smem<D, NT> *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = a.n_q / a.c.n_kv;
    constexpr int PART = part_floats(D, 8 * NT);
    int64_t *prefix = reinterpret_cast<int64_t *>(ws);
    float *parts = reinterpret_cast<float *>(ws + prefix_bytes(a.B));

    if (lane == 0)
        for (int s = 0; s < STAGES; ++s) mbar_init(smem_u32(&sm.full[warp][s]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    pdl_acquire();

    // ---- the line of work: each thread a run of sequences, then a scan over the threads ----
    const int per = (a.B + WARPS * 32 - 1) / (WARPS * 32);
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    int64_t mine = 0;
    Cursor c = {};  // the sequence at hand: with one a thread it is not read again below
    for (int b = b0; b < b1; ++b) {
        c.s = load_seq<NT>(a, b, group);
        mine += c.s.units(a.c.n_kv);
        if (blockIdx.x == 0 && a.kv_lens[b] > c.s.len) atomicOr(a.status, PQE_STATUS_BAD_PAGE);
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) sm.scan[warp] = incl;
    __syncthreads();
    int64_t total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += sm.scan[w];
        total += sm.scan[w];
    }
    before += incl - mine;
    const int64_t nw = shares(total, gridDim.x);
    if (tid <= WARPS) sm.share[tid] = share_start(min((int64_t)blockIdx.x * WARPS + tid, nw), nw, total);
    __syncthreads();
    int64_t at = before;
    for (int b = b0; b < b1; ++b) {
        if (per > 1) c.s = load_seq<NT>(a, b, group);
        const int64_t n = c.s.units(a.c.n_kv);
        c.b = b;
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            if (sm.share[w] >= at && sm.share[w] < at + n) {
                sm.at[w] = c;
                sm.first[w] = at;
            }
        if (blockIdx.x == 0) prefix[b] = at;
        at += n;
    }
    if (blockIdx.x == 0 && tid == 0) prefix[a.B] = total;
    __syncthreads();

    // ---- this warp's share ----
    const int64_t u0 = sm.share[warp], u1 = sm.share[warp + 1];
    if (u0 < u1) {
        int left = (int)(u1 - u0), ahead = 0;  // units to do, and to fetch: from a tile on, never from one of OPEN
        int rows_end = 0;                      // what is left to fetch when the rows' last tile has been
        Feed f;
        {
            Cursor c = sm.at[warp];
            const uint32_t per_rows = c.s.T + OPEN;
            const int64_t off = u0 - sm.first[warp];
            const int nth = off >> 32 ? (int)(off / per_rows) : (int)((uint32_t)off / per_rows);
            const int skip = (int)(off - (int64_t)nth * per_rows) - OPEN;
            c.head = nth / c.s.nrc;
            c.chunk = nth % c.s.nrc;
            c.tile = max(skip, 0);
            left += min(skip, 0);
            ahead = left;
            rows_end = left - (c.s.T - c.tile);
            f = feed_of<D>(a, c, lane);
            __syncwarp();
            if (lane == 0) sm.at[warp] = sm.ahead[warp] = c;
            __syncwarp();
        }
        const uint32_t ring = smem_u32(sm.ring[warp][0]), bar = smem_u32(&sm.full[warp][0]);
        uint32_t have[STAGES] = {};
        int page = ahead > 0 ? table_entry(a, f) : -1;
        uint32_t fetched = 0;
        auto fetch_next = [&](int s) {
            ++fetched;
            const uint32_t h = fetch<D>(a, f, page, ring + s * tile_bytes<D>(), bar + 8 * s, lane);
            f.j += TILE;
            if (--ahead == rows_end && ahead > 0) {
                ahead -= OPEN;
                Cursor c = sm.ahead[warp];
                if (ahead > 0) next_rows<NT>(a, c, group);
                f = feed_of<D>(a, c, lane);
                rows_end = ahead - c.s.T;
                __syncwarp();
                if (lane == 0) sm.ahead[warp] = c;
                __syncwarp();
            }
            if (ahead > 0) page = table_entry(a, f);
            return h;
        };
        if (ahead > 0) have[0] = fetch_next(0);
        if (ahead > 0) have[1] = fetch_next(1);
        Rows<D, NT> R;
        bool ok = true;
        uint32_t it = 0;
        while (left > 0 && ok) {
            // the tiles of one (sequence, head, rows)
            int j0, j_end, j_start, tiles;
            {
                const Cursor c = sm.at[warp];
                begin_rows<D, NT>(a, c, group, lane, R);
                if (lane == 0) sm.fac[warp].far = 0;
                __syncwarp();
                tiles = min(c.s.T - c.tile, left);
                j0 = j_start = (c.s.t0 + c.tile) * TILE;
                j_end = j0 + tiles * TILE;
            }
            for (; j0 < j_end; j0 += TILE, ++it) {
                const int s = it & 1;
                if (!mbar_wait(bar + 8 * s, it >> 1 & 1u, a.wait_limit)) ok = false;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (j0 < R.max_hi)  // else no row of the chunk sees it
                    add_tile<D, NT>(sm.ring[warp][s], sm.fac[warp], j0, s ? have[1] : have[0], lane, R);
                if (ahead > 0) {
                    const uint32_t h = fetch_next(s);
                    if (s)
                        have[1] = h;
                    else
                        have[0] = h;
                }
            }
            Cursor c = sm.at[warp];
            const int from = c.tile, to = from + tiles;
            const int64_t seg_start = u1 - left - from - OPEN;
            left -= tiles;
            const bool ended = to == c.s.T, whole = from == 0 && ended;
            if (ended) left -= OPEN;
            // the share's first piece in the first partial, one that begins inside it in the second
            float *part = parts + ((size_t)2 * (blockIdx.x * WARPS + warp) + (seg_start > u0 ? 1 : 0)) * PART;
            if (ok) {
                if (alike(R, j_start, j_end) && !sm.fac[warp].far)
                    end_rows<D, NT>(a, c, group, lane, R, whole, part);
                else
                    plain_rows<D, NT>(a, c, j_start, j_end, whole, part);
            }
            if (left > 0) {
                next_rows<NT>(a, c, group);
                __syncwarp();
                if (lane == 0) sm.at[warp] = c;
                __syncwarp();
            }
        }
        if (!ok) {
            // the copies in flight land before the block ends (bounded, whatever the limit of the other waits is)
#pragma unroll
            for (int s = 0; s < STAGES; ++s) {
                const uint32_t n = (fetched + STAGES - 1 - s) / STAGES;  // copies into this stage
                if (n) mbar_wait(bar + 8 * s, (n - 1) & 1u, DEFAULT_WAIT_LIMIT);
            }
            if (lane == 0) atomicOr(a.status, PQE_STATUS_TIMEOUT);
        }
    }
}

// Joins the partials of the (sequence, KV head, rows) that more than one share
// took part in, and writes the rows of sequences with no token to see. A CTA
// has some rows of one of them (blockIdx.x; rows blockIdx.y * blockDim.z on),
// W = blockDim.y warps a row: each takes every W-th partial, JOIN_AHEAD loads at
// a time, and their results are joined in order. (The partials are fresh from
// other SMs: a round of loads takes some 2 us, and so few of them is what counts.)
constexpr int JOIN_WARPS = 16, JOIN_AHEAD = 6;
template <int D, int NT>
__global__ void __launch_bounds__(32 * JOIN_WARPS)
    attn_join_kernel(const AttnArgs a, const uint8_t *ws, int split_ctas, int chunks) {
    constexpr int PART = part_floats(D, 8 * NT), E = D / 32;
    __shared__ float sh_m[JOIN_WARPS], sh_l[JOIN_WARPS];
    __shared__ __align__(16) float sh_o[JOIN_WARPS][D];
    const int lane = threadIdx.x, warp = threadIdx.y, W = blockDim.y, group = a.n_q / a.c.n_kv;
    const int r = blockIdx.y * blockDim.z + threadIdx.z;  // of the 8 * NT
    const int b = blockIdx.x / (a.c.n_kv * chunks), head = blockIdx.x / chunks % a.c.n_kv;
    // the call's own inputs were complete before the split kernel let this one start
    const Seq s = load_seq<NT>(a, b, group);
    pdl_acquire();
    const int n = is_ours(a, s.m) ? s.m * group : 0;
    // (one chunk, unless a sequence has more queries than the call said)
    for (int r0 = (int)(blockIdx.x % chunks) * 8 * NT; r0 < n; r0 += chunks * 8 * NT) {
        const bool mine = r < 8 * NT && r0 + r < n;
        const int64_t row = mine ? row_index(a, s, head, group, r0 + r) : 0;
        if (s.T == 0) {
            if (mine && warp == 0 && lane < D / 4)
                store_out(a, row, D, lane * 4, make_float4(0.f, 0.f, 0.f, 0.f), 0.f, 0.f);
            continue;
        }
        const int64_t *prefix = reinterpret_cast<const int64_t *>(ws);
        const float *parts = reinterpret_cast<const float *>(ws + prefix_bytes(a.B));
        const int64_t total = prefix[a.B], nw = shares(total, split_ctas);
        const int64_t s0 = prefix[b] + ((int64_t)head * s.nrc + r0 / (8 * NT)) * (s.T + OPEN);
        const int w0 = (int)share_of(s0 + OPEN, nw, total), w1 = (int)share_of(s0 + OPEN + s.T - 1, nw, total);
        if (w0 == w1) continue;  // that share's warp wrote it
        // the first share's partial is its second one if the row begins inside it
        const bool inside = s0 > share_start(w0, nw, total);
        float m = -INFINITY, l = 0.f, o[E] = {};
        for (int w = w0 + warp; mine && w <= w1; w += W * JOIN_AHEAD) {
            float pm[JOIN_AHEAD], pl[JOIN_AHEAD], po[JOIN_AHEAD][E];
#pragma unroll
            for (int y = 0; y < JOIN_AHEAD; ++y) {
                const int x = w + y * W;
                const float *p = parts + ((size_t)2 * x + (x == w0 && inside ? 1 : 0)) * PART;
                pm[y] = x <= w1 ? p[8 * NT * D + r] : -INFINITY;
                pl[y] = x <= w1 ? p[8 * NT * D + 8 * NT + r] : 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) po[y][e] = 0.f;
                if (x <= w1) {
                    if constexpr (E == 4)
                        *reinterpret_cast<float4 *>(po[y]) = *reinterpret_cast<const float4 *>(p + r * D + lane * E);
                    else
                        *reinterpret_cast<float2 *>(po[y]) = *reinterpret_cast<const float2 *>(p + r * D + lane * E);
                }
            }
            float now = m;
#pragma unroll
            for (int y = 0; y < JOIN_AHEAD; ++y) now = fmaxf(now, pm[y]);
            const float base = now == -INFINITY ? 0.f : now, keep = exp2_approx(m - base);
            l *= keep;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] *= keep;
#pragma unroll
            for (int y = 0; y < JOIN_AHEAD; ++y) {
                const float f = exp2_approx(pm[y] - base);
                l = fmaf(pl[y], f, l);
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = fmaf(po[y][e], f, o[e]);
            }
            m = now;
        }
        const int slot = threadIdx.z * W;
#pragma unroll
        for (int e = 0; e < E; ++e) sh_o[slot + warp][lane * E + e] = o[e];
        if (lane == 0) {
            sh_m[slot + warp] = m;
            sh_l[slot + warp] = l;
        }
        __syncthreads();
        if (mine && warp == 0 && lane < D / 4) {
            m = -INFINITY;
            for (int w = 0; w < W; ++w) m = fmaxf(m, sh_m[slot + w]);
            const float base = m == -INFINITY ? 0.f : m;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            l = 0.f;
            for (int w = 0; w < W; ++w) {
                const float f = exp2_approx(sh_m[slot + w] - base);
                const float4 v = *reinterpret_cast<const float4 *>(&sh_o[slot + w][lane * 4]);
                sum.x = fmaf(v.x, f, sum.x), sum.y = fmaf(v.y, f, sum.y), sum.z = fmaf(v.z, f, sum.z), sum.w = fmaf(v.w, f, sum.w);
                l = fmaf(sh_l[slot + w], f, l);
            }
            store_out(a, row, D, lane * 4, sum, m, l);
        }
        __syncthreads();
    }
}

template <int D, int NT>
int launch(const AttnArgs &a, int max_q, int sms, void *ws, cudaStream_t s) {
    // as many CTAs as fit, or as the longest sequences that the table can describe give work for
    const int group = a.n_q / a.c.n_kv;
    const int64_t nrc = ((int64_t)max_q * group + 8 * NT - 1) / (8 * NT);
    const int64_t tiles = (((int64_t)a.max_pages << a.c.page_shift) + TILE - 1) / TILE;
    const double most = (double)a.B * a.c.n_kv * nrc * (tiles + OPEN) / WARPS + 1;
    const int64_t units = (int64_t)a.B * a.c.n_kv * nrc;
    PQE_CHECK_ARG(units <= INT32_MAX);
    int grid = sms * ctas(D, NT);
    if (most < grid) grid = (int)most;
    static bool set[PQE_MAX_DEVICES] = {};
    int dev = 0, n = 0;
    int rc = device_info(dev, n);
    if (rc != PQE_OK) return rc;
    constexpr int smem = (int)sizeof(Smem<D, NT>);
    if (!set[dev]) {
        PQE_CUDA_TRY(cudaFuncSetAttribute(attn_split_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
        set[dev] = true;
    }
    rc = launch_pdl(attn_split_kernel<D, NT>, dim3((unsigned)grid), dim3(WARPS * 32), smem, s, a,
                    static_cast<uint8_t *>(ws));
    if (rc != PQE_OK) return rc;
    // as few warps a row as take a mean number of partials in one round; eight warps a CTA, or one row's
    const int64_t per_row = (int64_t)grid * WARPS / units + 1;
    const int W = (int)(per_row < 5 * JOIN_WARPS ? (per_row + 4) / 5 : JOIN_WARPS), rows = W < 8 ? 8 / W : 1;
    return launch_pdl(attn_join_kernel<D, NT>, dim3((unsigned)units, (unsigned)((8 * NT + rows - 1) / rows)), dim3(32, W, rows),
                      0, s, a, static_cast<const uint8_t *>(ws), grid, (int)nrc);
}

}  // namespace split

// Rows of a KV head taken together, in eights: as few as hold a step's, and what registers allow. A sequence's cache is read
// once for each such set of its rows.
static int eights(int max_q, int group, int d) {
    const int64_t rows = (int64_t)max_q * group;
    return rows <= 8 ? 1 : rows <= 16 || d == 128 ? 2 : rows <= 24 ? 3 : 2;
}

size_t attn_split_ws(int B, int max_q, int group, int d) {
    const int NT = eights(max_q, group, d);
    int dev = 0, sms = 0;
    if (device_info(dev, sms) != PQE_OK) sms = 160;  // without a device: an upper bound
    return split::prefix_bytes(B) +
           (size_t)sms * split::ctas(d, NT) * 2 * split::WARPS * split::part_floats(d, 8 * NT) * sizeof(float);
}

int attn_split(const pqe_kv_cache *cache, const AttnArgs &a, int max_q, int sms, void *ws, cudaStream_t s) {
    const int NT = eights(max_q, a.n_q / a.c.n_kv, cache->d);
    if (cache->d == 128) return NT == 1 ? split::launch<128, 1>(a, max_q, sms, ws, s) : split::launch<128, 2>(a, max_q, sms, ws, s);
    return NT == 1   ? split::launch<64, 1>(a, max_q, sms, ws, s)
           : NT == 2 ? split::launch<64, 2>(a, max_q, sms, ws, s)
                     : split::launch<64, 3>(a, max_q, sms, ws, s);
}

}  // namespace kv
}  // namespace pqe
