// kv_cache.cu -- writing K and V rows into the 4-bit paged cache, and reading
// them back.
//
// Per block of 32 values along d: amax, X = 2^(floor(log2 amax) - 2), codes
// RNE_e2m1(v / X). X is a power of two, so v / X is exact in fp32 and the only
// rounding is the code's own. The lanes' shares are those of the cache's byte
// order, so that what a warp writes or reads of a block is contiguous: K by rows,
// V by places.
//
// Bound by memory once there are many tokens, with the conversions close behind
// (an instruction for every two values each of expanding, scaling and coding), by
// latency below. 16384 tokens of 8 heads of 128, 85 MB: write 18.1 us (4.7 TB/s),
// read 15.7 us (5.4 TB/s), on three sets of tensors in turn (on one, partly in L2:
// 16.6 and 14.4); 65537 of 4 heads: read 28.4 us (6.0 TB/s); 64 tokens of 8 heads:
// 1.7 us each.
#include "kv_layout.cuh"

namespace pqe {
namespace kv {

// bits of |v| of two bf16: they order as the values do; a NaN or an infinity ends at or above 0x7F80
__device__ __forceinline__ uint32_t top_of(uint32_t a, uint32_t b) { return __vmaxu2(a & 0x7FFF7FFFu, b & 0x7FFF7FFFu); }
__device__ __forceinline__ uint32_t top_of(uint32_t two) { return max(two & 0xFFFFu, two >> 16); }

// E8M0 byte of a block of 32 with largest |v| `top` (bf16 bits), and 1 / X; 255 and 0 for one that is not finite
__device__ __forceinline__ uint32_t block_scale(uint32_t top, float &inv) {
    // floor(log2 amax) + 127 is the exponent field; subnormal values end at byte 0
    const uint32_t s = (uint32_t)max((int)(top >> 7) - 2, 0);
    inv = __uint_as_float((254u - s) << 23);  // 2^(127 - s): s is at most 252 for finite values
    if (top >= 0x7F80u) {
        inv = 0.f;
        return 255;
    }
    return s;
}

// eight bf16 to their codes, the first in the lowest nibble; zero where inv is (they may then be NaN)
__device__ __forceinline__ uint32_t codes8(const uint4 &v, float inv) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        lo[i] = __uint_as_float(w[i] << 16) * inv;
        hi[i] = __uint_as_float(w[i] & 0xFFFF0000u) * inv;
    }
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(lo[0]), "f"(hi[0]), "f"(lo[1]), "f"(hi[1]), "f"(lo[2]), "f"(hi[2]), "f"(lo[3]), "f"(hi[3]));
    return inv == 0.f ? 0u : r;
}

// What the values of scale byte x come to as bf16 pairs. The bits of an f16 one, shifted to bf16's places, are those of
// 2^-112 times the value; 2^(x - 15) is left, in two factors where x is above 142. NaN for 255.
struct Factor {
    uint32_t a, b;
};
__device__ __forceinline__ Factor factor_of(uint32_t x) {
    Factor f;
    f.a = x == 255u ? 0x7FC07FC0u : (min(x, 142u) + 112u) * (128u * 0x10001u);
    f.b = (max(x, 142u) - 15u) * (128u * 0x10001u);
    return f;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// eight codes to bf16: four of one block, four of another
__device__ __forceinline__ uint4 values8(uint32_t codes, const Factor &x, const Factor &y) {
    uint32_t h[4];
    e2m1x8_to_f16(codes, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const Factor &f = i < 2 ? x : y;
        h[i] = mul_bf16x2(mul_bf16x2((h[i] >> 3 & 0x0FFF0FFFu) | (h[i] & 0x80008000u), f.a), f.b);
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}

// ---- few tokens: a thread per eight values, the shortest way from a row to its bytes ----

// Token, head, first channel and K or V of eight values; 2 * n_kv * D / 8 threads a token, K before V, four neighbouring
// lanes for a block of 32.
struct Eight {
    int tok, head, e;
    bool is_v, in;
};
template <int D>
__device__ __forceinline__ Eight eight_of(const Cache &c, int n) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x, per = 2 * c.n_kv * (D / 8);
    Eight x;
    x.tok = (int)(i / per);
    x.in = x.tok < n;
    const uint32_t r = i % per;
    x.is_v = r >= per / 2;
    const uint32_t rr = x.is_v ? r - per / 2 : r;
    x.head = (int)(rr / (D / 8));
    x.e = (int)(rr % (D / 8)) * 8;
    return x;
}
// the token's slot, -1 if it has none
__device__ __forceinline__ int64_t slot_of(const Cache &c, const int64_t *slots, const Eight &x, int32_t *status) {
    if (!x.in) return -1;
    const int64_t slot = slots[x.tok];
    if (slot >> c.page_shift < c.n_pages) return slot;
    if (!x.is_v && x.head == 0 && x.e == 0) atomicOr(status, PQE_STATUS_BAD_PAGE);
    return -1;
}

template <int D>
__global__ void __launch_bounds__(256) kv_write_few_kernel(const Cache c, const uint16_t *__restrict__ k,
                                                           const uint16_t *__restrict__ v, int64_t k_stride,
                                                           int64_t v_stride, const int64_t *__restrict__ slots, int n,
                                                           int32_t *status) {
    pdl_acquire();
    const Eight x = eight_of<D>(c, n);
    // the row is asked for beside its slot
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (x.in) raw = *reinterpret_cast<const uint4 *>((x.is_v ? v + x.tok * v_stride : k + x.tok * k_stride) + x.head * D + x.e);
    const int64_t slot = slot_of(c, slots, x, status);
    uint32_t top = top_of(__vmaxu2(top_of(raw.x, raw.y), top_of(raw.z, raw.w)));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    float inv;
    const uint32_t scale = block_scale(top, inv);
    const uint32_t word = codes8(raw, inv);
    if (slot < 0) return;
    const int at = (int)(slot & ((1 << c.page_shift) - 1)), t = at & 15;
    uint8_t *b = block_of<D>(c, slot >> c.page_shift, at, x.head);
    if (!x.is_v) {
        *reinterpret_cast<uint32_t *>(b + k_code<D>(t, x.e)) = word;
        if (x.e % 32 == 0) b[k_scale<D>(t, x.e / 32)] = (uint8_t)scale;
    } else {
        *reinterpret_cast<uint16_t *>(b + v_code<D>(t, x.e)) = (uint16_t)word;
        *reinterpret_cast<uint16_t *>(b + v_code<D>(t, x.e + 4)) = (uint16_t)(word >> 16);
        if (x.e % 32 == 0) b[v_scale<D>(t, x.e / 32)] = (uint8_t)scale;
    }
}

template <int D>
__global__ void __launch_bounds__(256) kv_read_few_kernel(const Cache c, const int64_t *__restrict__ slots, int n,
                                                          uint16_t *k, uint16_t *v, int32_t *status) {
    pdl_acquire();
    const Eight x = eight_of<D>(c, n);
    const int64_t slot = slot_of(c, slots, x, status);
    uint16_t *out = x.is_v ? v : k;
    if (!x.in || !out) return;
    uint32_t word = 0, s = 0;
    if (slot >= 0) {
        const int at = (int)(slot & ((1 << c.page_shift) - 1)), t = at & 15;
        const uint8_t *b = block_of<D>(c, slot >> c.page_shift, at, x.head);
        if (!x.is_v) {
            word = *reinterpret_cast<const uint32_t *>(b + k_code<D>(t, x.e));
            s = b[k_scale<D>(t, x.e / 32)];
        } else {
            word = (uint32_t)*reinterpret_cast<const uint16_t *>(b + v_code<D>(t, x.e)) |
                   (uint32_t)*reinterpret_cast<const uint16_t *>(b + v_code<D>(t, x.e + 4)) << 16;
            s = b[v_scale<D>(t, x.e / 32)];
        }
    }
    const Factor f = factor_of(s);
    *reinterpret_cast<uint4 *>(out + ((size_t)x.tok * c.n_kv + x.head) * D + x.e) = values8(word, f, f);
}

// ---- many tokens ----

constexpr int WARPS = 8;
// Groups an SM below which a thread for each eight values is faster. (Write and read of a run of 1024 tokens of 8 heads of
// 128, 7 groups an SM: 3.2 + 2.9 us that way, 3.0 + 3.1 by groups; 3000 of 4 heads, 10: 3.8 + 3.3 and 4.0 + 3.7; 2048 of 8, 13:
// 4.6 + 4.0 and 4.1 + 3.8; 512: 2.3 + 2.1 and 2.9 + 3.0; 16384: 24.7 + 23.5 and 16.6 + 14.4.)
constexpr int FEW_WARPS = 12;

// The 16 rows that a warp takes of one head of K or V: consecutive rows of the
// call. Where they go is told per row, so they may lie in 16 blocks; a prompt's
// rows lie in one block, or in two when the call begins inside one.
struct Group {
    const uint8_t *blk[16];  // the row's block in the cache (of this head), NULL: no row, or one that is skipped
    int8_t tok[16];          // its place in the block
    int8_t row[16];          // V: the row that the lanes of place p take. Where the rows' places are all different, that is
                             // the row of place p, and a lane's four rows then lie side by side in a block's bytes
};

template <int D>
__device__ __forceinline__ void group_of(const Cache &c, const int64_t *__restrict__ slots, int n, int first, int head,
                                         int lane, Group &g, int32_t *status, bool report) {
    const int r = lane & 15;
    int64_t slot = first + r < n ? slots[first + r] : -1;
    if (slot >> c.page_shift >= c.n_pages) {
        if (report && lane < 16) atomicOr(status, PQE_STATUS_BAD_PAGE);
        slot = -1;
    }
    const int at = (int)(slot & ((1 << c.page_shift) - 1)), tok = at & 15;
    const uint32_t place = slot >= 0 ? 1u << tok : 0u;
    // all places different: as many bits as rows
    const uint32_t places = __reduce_or_sync(0xffffffffu, place);
    const bool apart = __popc(places) == __popc(__ballot_sync(0xffffffffu, slot >= 0) & 0xFFFFu);
    if (lane < 16) {
        g.blk[r] = slot >= 0 ? block_of<D>(c, slot >> c.page_shift, at, head) : nullptr;
        g.tok[r] = (int8_t)tok;
        if (!apart || !(places >> r & 1)) g.row[r] = apart ? (int8_t)-1 : (int8_t)r;
    }
    __syncwarp();
    if (lane < 16 && apart && slot >= 0) g.row[tok] = (int8_t)r;
    __syncwarp();
}

// K and V of one group and head by one warp each: four lanes a row, eight channels of each block a lane. A K row's bytes go
// out as they are; those of V, which lie two by two among the other tokens' of their block, meet in shared memory first where
// the rows fill a block, and go out as the block's bytes do. (16384 tokens of 8 heads of 128:
// 16.6 us, two bytes at a time 20.5.)
template <int D>
__global__ void __launch_bounds__(32 * WARPS) kv_write_kernel(const Cache c, const uint16_t *__restrict__ k,
                                                              const uint16_t *__restrict__ v, int64_t k_stride,
                                                              int64_t v_stride, const int64_t *__restrict__ slots, int n,
                                                              int32_t *status) {
    __shared__ Group groups[WARPS];
    __shared__ __align__(16) uint8_t staged[WARPS][8 * D + D / 2];  // a block's V codes and V scales
    constexpr int NB = D / 32, CODES = 8 * D;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane & 3;
    const uint32_t unit = blockIdx.x * WARPS + warp, per = 2 * c.n_kv, which = unit % per;
    const int first = (int)(unit / per) * 16, head = which >> 1;
    const bool is_v = which & 1;
    pdl_acquire();
    if (first >= n) return;
    Group &G = groups[warp];
    group_of<D>(c, slots, n, first, head, lane, G, status, which == 0);
    uint4 raw[2][NB];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = (lane >> 2) + 8 * h;
        const uint16_t *row = (is_v ? v + (first + r) * v_stride : k + (first + r) * k_stride) + head * D + 8 * t;
#pragma unroll
        for (int b = 0; b < NB; ++b)
            raw[h][b] = G.blk[r] ? *reinterpret_cast<const uint4 *>(row + 32 * b) : make_uint4(0, 0, 0, 0);
    }
    // V: do the 16 rows fill all the places of one block? (Two rows of one slot leave a place without a row.)
    const uint8_t *blk0 = G.blk[0];
    const bool side = __all_sync(0xffffffffu, blk0 && G.blk[lane & 15] == blk0);
    const bool whole = is_v && side && __reduce_or_sync(0xffffffffu, 1u << G.tok[lane & 15]) == 0xFFFFu;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = (lane >> 2) + 8 * h;
        uint8_t *blk = const_cast<uint8_t *>(G.blk[r]);
        uint32_t word[NB], scales = 0;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint4 &u = raw[h][b];
            uint32_t top = top_of(__vmaxu2(top_of(u.x, u.y), top_of(u.z, u.w)));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            float inv;
            scales |= block_scale(top, inv) << (8 * b);
            word[b] = codes8(u, inv);
        }
        if (!blk) continue;
        const int tok = G.tok[r];
        if (!is_v) {
            if constexpr (D == 128) {
                *reinterpret_cast<uint4 *>(blk + tok * 64 + t * 16) = make_uint4(word[0], word[1], word[2], word[3]);
                if (t == 0) *reinterpret_cast<uint32_t *>(blk + 16 * D + tok * 4) = scales;
            } else {
                *reinterpret_cast<uint2 *>(blk + tok * 32 + t * 8) = make_uint2(word[0], word[1]);
                if (t == 0) *reinterpret_cast<uint16_t *>(blk + 16 * D + tok * 2) = (uint16_t)scales;
            }
            continue;
        }
        uint8_t *codes = whole ? staged[warp] : blk + CODES, *sc = whole ? staged[warp] + CODES : blk + 16 * D + D / 2;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            // channels 8t .. 8t+3 are lane 2t's of the attention's fragments, the next four lane 2t+1's
            const int at = v_code<D>(tok, 32 * b + 8 * t) - CODES;
            *reinterpret_cast<uint16_t *>(codes + at) = (uint16_t)word[b];
            *reinterpret_cast<uint16_t *>(codes + at + 64) = (uint16_t)(word[b] >> 16);
            if (t == b) sc[v_scale<D>(tok, b) - 16 * D - D / 2] = (uint8_t)(scales >> (8 * b));
        }
    }
    if (!whole) return;
    __syncwarp();
    uint8_t *dst = const_cast<uint8_t *>(blk0);
#pragma unroll
    for (int i = 0; i < CODES / 512; ++i)
        *reinterpret_cast<uint4 *>(dst + CODES + 512 * i + 16 * lane) =
            *reinterpret_cast<const uint4 *>(staged[warp] + 512 * i + 16 * lane);
    if (lane < D / 32)
        *reinterpret_cast<uint4 *>(dst + 16 * D + D / 2 + 16 * lane) =
            *reinterpret_cast<const uint4 *>(staged[warp] + CODES + 16 * lane);
}

// The same shares as the write's: a group, a head, K or V a warp.
template <int D>
__global__ void __launch_bounds__(32 * WARPS) kv_read_kernel(const Cache c, const int64_t *__restrict__ slots, int n,
                                                             uint16_t *k, uint16_t *v, int32_t *status) {
    __shared__ Group groups[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t unit = blockIdx.x * WARPS + warp, per = 2 * c.n_kv, which = unit % per;
    const int first = (int)(unit / per) * 16, head = which >> 1;
    pdl_acquire();
    if (first >= n) return;
    Group &G = groups[warp];
    group_of<D>(c, slots, n, first, head, lane, G, status, which == 0);
    constexpr int NB = D / 32;
    if (!(which & 1)) {
        if (!k) return;
        const int t = lane & 3;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = (lane >> 2) + 8 * h;
            if (first + r >= n) continue;
            uint32_t word[NB] = {}, scales = 0;
            if (const uint8_t *blk = G.blk[r]) {
                const int tok = G.tok[r];
                if constexpr (D == 128) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(blk + tok * 64 + t * 16);
                    word[0] = u.x, word[1] = u.y, word[2] = u.z, word[3] = u.w;
                    scales = *reinterpret_cast<const uint32_t *>(blk + 16 * D + tok * 4);
                } else {
                    const uint2 u = *reinterpret_cast<const uint2 *>(blk + tok * 32 + t * 8);
                    word[0] = u.x, word[1] = u.y;
                    scales = *reinterpret_cast<const uint16_t *>(blk + 16 * D + tok * 2);
                }
            }
            uint16_t *out = k + ((size_t)(first + r) * c.n_kv + head) * D + 8 * t;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const Factor f = factor_of(scales >> (8 * b) & 255u);
                *reinterpret_cast<uint4 *>(out + 32 * b) = values8(word[b], f, f);
            }
        }
    } else {
        if (!v) return;
        const int g = lane >> 2, t = lane & 3;
        int row[4];
        const uint8_t *blk[4];
        bool together = true;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int place = 2 * t + (j & 1) + 8 * (j >> 1);
            row[j] = G.row[place];
            blk[j] = row[j] >= 0 ? G.blk[row[j]] : nullptr;
            together = together && blk[j] && blk[j] == blk[0] && G.tok[row[j]] == place;
        }
        uint32_t word[NB / 2][4] = {}, scales[NB] = {};
        if (together) {
#pragma unroll
            for (int q = 0; q < NB / 2; ++q) {
                const uint4 u = *reinterpret_cast<const uint4 *>(blk[0] + 8 * D + q * 512 + lane * 16);
                word[q][0] = u.x, word[q][1] = u.y, word[q][2] = u.z, word[q][3] = u.w;
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
                scales[b] = *reinterpret_cast<const uint32_t *>(blk[0] + 16 * D + D / 2 + t * (D / 8) + b * 4);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (!blk[j]) continue;
                const int tok = G.tok[row[j]];
#pragma unroll
                for (int q = 0; q < NB / 2; ++q)
                    word[q][j] = *reinterpret_cast<const uint32_t *>(blk[j] + v_code<D>(tok, 64 * q + 4 * g));
#pragma unroll
                for (int b = 0; b < NB; ++b) scales[b] |= (uint32_t)blk[j][v_scale<D>(tok, b)] << (8 * j);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (row[j] < 0 || first + row[j] >= n) continue;
            uint16_t *out = v + ((size_t)(first + row[j]) * c.n_kv + head) * D + 4 * g;
#pragma unroll
            for (int b = 0; b < NB; b += 2) {
                const uint4 u = values8(word[b >> 1][j], factor_of(scales[b] >> (8 * j) & 255u), factor_of(scales[b + 1] >> (8 * j) & 255u));
                *reinterpret_cast<uint2 *>(out + 32 * b) = make_uint2(u.x, u.y);
                *reinterpret_cast<uint2 *>(out + 32 * b + 32) = make_uint2(u.z, u.w);
            }
        }
        // rows that are skipped: nobody's place where the others' are all different
        if (lane < 16 && first + lane < n && !G.blk[lane]) {
            bool mine = false;
            for (int p = 0; p < 16; ++p) mine = mine || G.row[p] == lane;
            if (!mine)
                for (int d = 0; d < D; d += 8)
                    *reinterpret_cast<uint4 *>(v + ((size_t)(first + lane) * c.n_kv + head) * D + d) = make_uint4(0, 0, 0, 0);
        }
    }
}

// a warp for each 16 rows, head, and K or V
static int64_t group_units(int n, int n_kv) { return (((int64_t)n + 15) / 16) * 2 * n_kv; }

template <typename... KArgs>
static int launch_groups(void (*few)(KArgs...), void (*many)(KArgs...), int n, int n_kv, int d, cudaStream_t s,
                         typename ident<KArgs>::type... args) {
    int dev = 0, sms = 0;
    const int rc = device_info(dev, sms);
    if (rc != PQE_OK) return rc;
    const int64_t units = group_units(n, n_kv);
    if (units < FEW_WARPS * sms)
        return launch_pdl(few, dim3((unsigned)(((int64_t)n * 2 * n_kv * d / 8 + 255) / 256)), dim3(256), 0, s, args...);
    return launch_pdl(many, dim3((unsigned)((units + WARPS - 1) / WARPS)), dim3(32 * WARPS), 0, s, args...);
}

}  // namespace kv
}  // namespace pqe

using namespace pqe;

extern "C" {

size_t pqe_kv_page_bytes(int page_size, int n_kv, int d) {
    if (!kv::cache_shape_ok(page_size, n_kv, d)) return 0;
    return (size_t)n_kv * (page_size / kv::BLOCK) * kv::block_bytes(d);
}

int kv_cache_write(const pqe_kv_cache *cache, const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                   const int64_t *slots, int n, int32_t *status, void *stream) {
    PQE_CHECK_ARG(kv::cache_ok(cache) && n >= 0);
    if (n == 0) return PQE_OK;
    const int64_t row = (int64_t)cache->n_kv * cache->d;
    PQE_CHECK_ARG(k && v && slots && status && aligned(k, 16) && aligned(v, 16) && aligned(slots, 8));
    PQE_CHECK_ARG(k_stride >= row && v_stride >= row && k_stride % 8 == 0 && v_stride % 8 == 0);
    const kv::Cache c = kv::cache_of(cache);
    const uint16_t *kp = static_cast<const uint16_t *>(k), *vp = static_cast<const uint16_t *>(v);
    if (cache->d == 128)
        return kv::launch_groups(kv::kv_write_few_kernel<128>, kv::kv_write_kernel<128>, n, cache->n_kv, 128,
                                 as_stream(stream), c, kp, vp, k_stride, v_stride, slots, n, status);
    return kv::launch_groups(kv::kv_write_few_kernel<64>, kv::kv_write_kernel<64>, n, cache->n_kv, 64, as_stream(stream), c,
                             kp, vp, k_stride, v_stride, slots, n, status);
}

int kv_cache_read(const pqe_kv_cache *cache, const int64_t *slots, int n, void *k, void *v, int32_t *status,
                  void *stream) {
    PQE_CHECK_ARG(kv::cache_ok(cache) && n >= 0);
    if (n == 0) return PQE_OK;
    PQE_CHECK_ARG((k || v) && slots && status && aligned(k, 16) && aligned(v, 16) && aligned(slots, 8));
    const kv::Cache c = kv::cache_of(cache);
    uint16_t *kp = static_cast<uint16_t *>(k), *vp = static_cast<uint16_t *>(v);
    if (cache->d == 128)
        return kv::launch_groups(kv::kv_read_few_kernel<128>, kv::kv_read_kernel<128>, n, cache->n_kv, 128, as_stream(stream),
                                 c, slots, n, kp, vp, status);
    return kv::launch_groups(kv::kv_read_few_kernel<64>, kv::kv_read_kernel<64>, n, cache->n_kv, 64, as_stream(stream), c,
                             slots, n, kp, vp, status);
}

}  // extern "C"
