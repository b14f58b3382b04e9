// sample.cu -- sample_tokens: the next token of each row of logits.
//
// What is kept of a row is a beginning of its order (logits descending, lower index first), and the token is where the sum of
// the kept weights, in index order, passes u times their total. A row lies in the shared memory of a cluster of 1 to 8 CTAs, so
// logits are read once; sums are whole numbers (weights times 2^43), the same in any order.
//
//   all kept (no top_k, no top_p)  a sum for each thread's part of a warp's stretch of the row, a scan, and the warp whose stretch u
//                                  falls into walks it.
//   a top_k of FEW_K at most       the largest logits of GROUPS groups of lanes: what is not below the top_k-th of them holds the
//                                  first top_k and is hardly more. Up to RANKED candidates go to a list, where the first CTA
//                                  compares each with each and finishes.
//   another border                 a histogram of the logits, 32 bins for each factor of two of the weights: counts, and for
//                                  top_p sums. The bins are merged in slices, a CTA each; the CTA whose slice the border falls
//                                  into finds the bin. Where what lies above the border's bin and in it is RANKED at most, it
//                                  is listed and finished in the same way. Otherwise the bin alone goes to a list (LIST at most)
//                                  that the first CTA sorts, which gives the border's value and how many of its equals are kept,
//                                  and the row is walked as above.
//   more than that in one bin      (thousands of equal logits, or nearly) bisection on the values' bits.
//
// Weights: with P = 32 log2(e) (max - l) / t, n a whole number near it and below, f the rest, w = 2^(-n / 32) 2^(-f / 32): the
// first factor from a table of all n, the second from five terms of its series. P is held in two floats: w is within 2^-28 of
// itself (the roundings of f ln(2) / 32, of its series and their product, by an emulation 2^-28.07 at worst) and 2^-44 of the
// largest, sums of thousands of them within far less. u of 24 bits falls so near a border of two tokens that it matters about
// once in a million rows of 10^5 nearly equal tokens.
//
// Rows of 131072 fp32: one 8.7 us (all kept), 7.6 (top_k), 20.5 (top_p); 64 of them 31.7, 41, 65, 51 with settings of each kind,
// 14 greedy. 512 rows of 32000, all kept: 54 us; reading them takes 10. What bounds it is a CTA's chain (begin, loads, maximum
// through the cluster, weights, sums through the cluster, the walk) with two CTAs an SM to overlap: without the weights those
// rows take 39 us, and a barrier of the cluster is 1000 to 1400 clocks. Then issue slots: 58 instructions for 32 logits a pass
// (41% of them used).
// Tried: weights from a table made for the row, fewer fp32 operations but as many instructions (53 us; top_p 65), a cluster that
// is through takes over a waiting one (clusterlaunchcontrol: 63 against 54; the loop around a row costs registers).
#include <math.h>

#include <atomic>
#include <type_traits>

#include "f32x2.cuh"
#include "pqe_common.cuh"
#include "tc_ptx.cuh"

namespace pqe {
namespace sampling {
using namespace ptx;
using namespace f32x2;
typedef unsigned long long u64;

struct Args {
    const void *logits;
    int64_t stride;
    int V;
    const float *temperature, *top_p, *min_p, *u;
    const int32_t *top_k;
    int32_t *tokens, *status;
    float *logprobs;
};

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int OCTAVE = 32;                   // bins for a factor of two
constexpr int FAR = 44 * OCTAVE + 1;         // what falls into this bin weighs less than 2^-44: nothing
constexpr int BINS = 1440;                   // FAR and a little, in slices for up to MAX_PARTS CTAs
constexpr int LIST = 2 * THREADS;            // elements of a bin that one CTA sorts, two a thread
constexpr int GROUPS = 128, FEW_K = 100;     // groups of lanes whose largest logits are compared; up to this top_k by them alone
constexpr int RANKED = 256;                  // candidates of a row that it ranks by comparing each with each
constexpr int MAX_PARTS = 8;
constexpr int SCALE = 43;                    // the largest logit's weight: 2^43; 2^18.6 of them fit 63 bits
constexpr int CHUNK_MAX = 46080;             // logits of a CTA; sums of a bin's 13-bit parts stay below 2^32
static_assert((int64_t)CHUNK_MAX << 13 < (int64_t)1 << 32, "");

// 2^SCALE 2^(-i / 32)
__device__ const u64 TABLE[OCTAVE] = {
    8796093022208ull, 8607610887057ull, 8423167535396ull, 8242676424423ull, 8066052865769ull, 7893213985764ull, 7724078686549ull, 7558567608024ull,
    7396603090613ull, 7238109138825ull, 7083011385596ull, 6931237057393ull, 6782714940072ull, 6637375345460ull, 6495150078656ull, 6355972406040ull,
    6219777023951ull, 6086500028053ull, 5956078883349ull, 5828452394836ull, 5703560678795ull, 5581345134690ull, 5461748417677ull, 5344714411690ull,
    5230188203118ull, 5118116055032ull, 5008445381977ull, 4901124725294ull, 4796103728980ull, 4693333116055ull, 4592764665442ull, 4494351189345ull};
constexpr int SLACK = 65536;                 // of 2^30: a weight is less than that under its bin's lower end (0.001 of P, and roundings)

// Whole numbers that order as the values do (-0 as +0), NaN below -infinity's or above +infinity's.
constexpr uint32_t KEY_NEG_INF = 0x007FFFFFu, KEY_INF = 0xFF800000u;
__device__ __forceinline__ uint32_t key_of(float l) {
    const uint32_t b = __float_as_uint(l + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

struct Found {         // where a border falls
    int bin;           // the bin, or -1
    uint32_t count;    // elements in the bins above it, and in it
    uint32_t in;
    u64 mass;          // sum of weights above it
};

struct Shared {
    union {                           // of block scans
        struct {
            u64 part[WARPS];
            uint32_t count_part[WARPS];
        };
        struct {
            u64 mass, far_mass;
            uint32_t count, far_count;
        } parts[WARPS];
    };
    u64 swap[3][MAX_PARTS][4];        // of the cluster's exchanges, three in turn
    u64 weight[FAR + 1];              // of the upper ends of the bins: bin b holds P from b - 1 on
    uint32_t listed[4];               // entries of each list gathered
    double min_drop;                  // t ln(min_p)
    Found found;
    uint32_t tops[GROUPS];            // the groups' largest logits
    float floor;                      // no smaller logit is among the first top_k
    u64 list[LIST];
    union {
        struct {
            uint32_t count[BINS];     // merged in place: counts, and sums of weights as (low, high) words
            uint32_t lo[BINS], hi[BINS];
        };
        u64 spare[RANKED];            // at the end
    };
};

static_assert(BINS > FAR && BINS % MAX_PARTS == 0, "");
constexpr size_t HEAD = (sizeof(Shared) + 127) / 128 * 128 + 64;  // + room to align the pieces
static_assert(HEAD + CHUNK_MAX * sizeof(float) <= 227 * 1024, "shared memory of one CTA");
// the most logits of a CTA with which two fit on an SM: of its 228 KB the system takes 1 KB a CTA (64 rows of 152064, 19008 a CTA:
// all kept 39 us, 52 with one CTA an SM; top_p 93, 140)
constexpr int CHUNK_TWO = (int)((114 * 1024 - 1024 - HEAD) / sizeof(float));
static_assert(2 * (HEAD + CHUNK_TWO * sizeof(float) + 1024) <= 228 * 1024, "");
static_assert(MAX_PARTS * CHUNK_TWO >= 152064, "a usual vocabulary keeps two CTAs an SM");

// What a row's weights go by.
constexpr float MAGIC = 12582912.f;  // 1.5 * 2^23: a number added to it is rounded to a whole one
struct Scale {
    float half_max, c_hi, c_lo;  // max / 2, and 64 log2(e) / t in two parts (values enter halved: their difference does not overflow)
    // MAGIC + the whole part of P of a logit, less what keeps the rest positive: rises as l falls
    __device__ __forceinline__ float spot(float l) const {
        return (fminf((half_max - 0.5f * l) * c_hi, (float)FAR) - 0.501f) + MAGIC;
    }
    __device__ __forceinline__ static int bin(float spot) { return __float_as_int(spot) - (0x4B400000 - 1); }
    __device__ __forceinline__ static float spot_of(int bin) { return MAGIC + (float)(bin - 1); }
    // the bins and weights of four logits
    __device__ __forceinline__ void weigh(const u64 *weight, const float (&l)[4], int (&b)[4], u64 (&w)[4]) const {
#pragma unroll
        for (int h = 0; h < 4; h += 2) {
            const u64 x = pair(l[h], l[h + 1]), hm = pair(half_max), c = pair(c_hi), minus = pair(-1.f);
            const u64 a = mul2(x, pair(0.5f)), s = fma2(x, pair(-0.5f), hm);  // s + e = half_max - a: what rounding took
            const u64 v = add2(s, pair(-half_max)), e = fma2(add2(a, v), minus, fma2(fma2(v, minus, s), minus, hm));
            const u64 np = mul2(s, pair(-c_hi));  // -P, and what P lacks
            const u64 lack = fma2(e, c, fma2(s, pair(c_lo), fma2(s, c, np)));
            const float2 q = unpair(np);
            const u64 at = add2(add2(pair(fminf(-q.x, (float)FAR), fminf(-q.y, (float)FAR)), pair(-0.501f)), pair(MAGIC));
            const float2 spots = unpair(at);
            b[h] = bin(spots.x), b[h + 1] = bin(spots.y);
            const u64 f = fma2(add2(np, add2(at, pair(-MAGIC))), minus, lack);
            const u64 r = mul2(f, pair(0.0216608493924982909f));  // ln(2) / 32
            u64 y = fma2(r, pair(1.f / 120), pair(-1.f / 24));
            y = fma2(r, y, pair(1.f / 6));
            y = fma2(r, y, pair(-0.5f));
            y = fma2(r, y, pair(1.f));
            const float2 z = unpair(mul2(mul2(r, y), pair(4294967296.f)));  // (1 - exp(-r)) 2^32
            w[h] = less(weight[b[h]], __float2uint_rn(z.x));
            w[h + 1] = less(weight[b[h + 1]], __float2uint_rn(z.y));
        }
    }
    __device__ __forceinline__ static u64 less(u64 w, uint32_t part) {  // w (1 - part / 2^32)
        return w - ((w >> 32) * part + __umulhi((uint32_t)w, part));
    }
    __device__ __forceinline__ u64 weight_of(const u64 *weight, float l) const {
        const float x[4] = {l, l, l, l};
        int b[4];
        u64 w[4];
        weigh(weight, x, b, w);
        return w[0];
    }
    // bins sum weights as what they have over the bin's lower end, in 30 bits of a weight's own
    __device__ __forceinline__ static int drop(int b) { return max(SCALE - 30 - max(b - 1, 0) / OCTAVE, 0); }
    __device__ __forceinline__ static int base(const u64 *weight, int b) { return (int)(weight[b + 1] >> drop(b)) - SLACK; }
};

// the part p in [0, 1) of a sum, rounded down, and up (p as 64 bits after the point: exact from 2^-40 on)
__device__ __forceinline__ u64 fixed(float p) { return __float2ull_rz(p * 18446744073709551616.f); }
__device__ __forceinline__ u64 share(float p, u64 sum) { return __umul64hi(fixed(p), sum); }
__device__ __forceinline__ u64 share_up(float p, u64 sum) {
    if (!(p > 0.f)) return 0;
    const u64 f = fixed(p);
    return __umul64hi(f, sum) + (f * sum != 0);
}

template <class T>
__device__ __forceinline__ T warp_scan(T v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const T w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += w;
    }
    return v;
}

// inclusive scans over the CTA of two values, and their totals
__device__ __forceinline__ void block_scan(Shared &sh, uint32_t &c, u64 &m, uint32_t &c_all, u64 &m_all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    c = warp_scan(c, lane);
    m = warp_scan(m, lane);
    __syncthreads();
    if (lane == 31) sh.count_part[warp] = c, sh.part[warp] = m;
    __syncthreads();
    uint32_t c0 = 0;
    u64 m0 = 0;
    c_all = 0, m_all = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w == warp) c0 = c_all, m0 = m_all;
        c_all += sh.count_part[w], m_all += sh.part[w];
    }
    c += c0, m += m0;
}
template <class T>
__device__ __forceinline__ T block_scan(Shared &sh, T v, T &all) {  // one value, 32 or 64 bits
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_scan(v, lane);
    __syncthreads();
    if (lane == 31) sh.part[warp] = v;
    __syncthreads();
    T before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w == warp) before = all;
        all += (T)sh.part[w];
    }
    return v + before;
}
__device__ __forceinline__ u64 block_sum(Shared &sh, u64 v) {
    u64 all;
    block_scan(sh, v, all);
    return all;
}

// ascending sort of `size` values (a power of two, at most H * THREADS), a thread's at threadIdx.x and (H = 2) THREADS further on;
// steps inside a warp by shuffles, the others through v
template <int H>
__device__ __forceinline__ void sort(u64 *v, u64 (&x)[H], int size) {
    const int i = threadIdx.x;
#pragma unroll 1
    for (int k = 2; k <= size; k *= 2)
#pragma unroll 1
        for (int j = k / 2; j > 0; j /= 2) {
            u64 y[H];
            if (H == 2 && j == THREADS) {
                y[0] = x[H - 1], y[H - 1] = x[0];
            } else if (j >= 32) {
                __syncthreads();
#pragma unroll
                for (int h = 0; h < H; ++h) v[i + h * THREADS] = x[h];
                __syncthreads();
#pragma unroll
                for (int h = 0; h < H; ++h) y[h] = v[(i ^ j) + h * THREADS];
            } else {
#pragma unroll
                for (int h = 0; h < H; ++h) y[h] = __shfl_xor_sync(0xffffffffu, x[h], j);
            }
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int at = i + h * THREADS;
                const bool low = ((at & j) == 0) == ((at & k) == 0);  // keeps the smaller
                x[h] = (x[h] < y[h]) == low ? x[h] : y[h];
            }
        }
}

__device__ __forceinline__ void st_remote(uint32_t addr, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_remote(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

template <bool FP32>
__global__ void __launch_bounds__(THREADS, 2) sample_kernel(const Args a, int parts_log, int chunk) {
    extern __shared__ __align__(128) uint8_t smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem);
    // the CTA's logits from line[shift] on, in fours; -infinity before and behind them
    float *line = reinterpret_cast<float *>(smem + (sizeof(Shared) + 127) / 128 * 128);
    int shift;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, parts = 1 << parts_log;
    const int rank = (int)cluster_rank();
    const int64_t row = blockIdx.x >> parts_log;
    const int c0 = rank * chunk, n = max(0, min(chunk, a.V - c0));
    int swaps = 0;

    // every CTA's four values to every CTA
    auto exchange = [&](u64 v0, u64 v1, u64 v2, u64 v3) -> u64(*)[4] {
        u64(*slot)[4] = sh.swap[swaps];
        swaps = swaps == 2 ? 0 : swaps + 1;
        __syncthreads();
        if ((int)threadIdx.x < 4 * parts) {
            const int j = threadIdx.x & 3;
            st_remote(map_rank(smem_u32(&slot[rank][j]), threadIdx.x >> 2), j == 0 ? v0 : j == 1 ? v1 : j == 2 ? v2 : v3);
        }
        __syncwarp();
        cluster_sync();
        return slot;
    };

    for (int i = threadIdx.x; i < BINS; i += THREADS) sh.count[i] = sh.lo[i] = sh.hi[i] = 0;
    for (int b = threadIdx.x; b <= FAR; b += THREADS) {
        const int n = max(b - 1, 0), by = n / OCTAVE;  // (bin 0, a hair above the largest: P - 1)
        const u64 w = (TABLE[n % OCTAVE] + ((1ull << by) >> 1)) >> by;
        sh.weight[b] = b == 0 ? 2 * TABLE[OCTAVE - 1] : b == FAR ? 0 : w;
    }
    if (threadIdx.x < 4) sh.listed[threadIdx.x] = 0;
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // waited for before the first exchange
    pdl_acquire();

    const float t = a.temperature ? a.temperature[row] : 1.f, top_p = a.top_p ? a.top_p[row] : 1.f;
    const float min_p = a.min_p ? a.min_p[row] : 0.f, u = a.u[row];
    const int top_k = a.top_k ? a.top_k[row] : 0;
    // one thread: fp64 is slow here, and the row's loads hide it
    if (threadIdx.x == THREADS - 1 && min_p > 0.f && min_p < 1.f && t > 0.f) sh.min_drop = (double)t * log((double)min_p);

    // ---- the row into shared memory, with its maximum ----
    float top = -INFINITY;
    bool bad = false;
    {
        auto see = [&](float l) {
            top = fmaxf(top, l);
            bad |= !(l < INFINITY);  // NaN, +infinity
        };
        constexpr int VEC = FP32 ? 4 : 8, SIZE = FP32 ? 4 : 2;
        const uint8_t *src = static_cast<const uint8_t *>(a.logits) + (row * a.stride + c0) * SIZE;
        const int head = min(n, (int)((16 - (reinterpret_cast<uintptr_t>(src) & 15)) & 15) / SIZE);  // up to 16-byte pieces
        shift = (VEC - head) & (VEC - 1);  // pieces are aligned here too
        float *data = line + shift;
        auto one = [&](int i) {
            const float l = FP32 ? reinterpret_cast<const float *>(src)[i] : bf16_to_f32(reinterpret_cast<const uint16_t *>(src)[i]);
            data[i] = l;
            see(l);
        };
        const int vecs = (n - head) / VEC;
        const uint4 *v = reinterpret_cast<const uint4 *>(src + head * SIZE);
        constexpr int U = 4;
        for (int i = threadIdx.x; i < vecs; i += U * THREADS) {
            uint4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i + u * THREADS < vecs) x[u] = __ldg(v + i + u * THREADS);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i + u * THREADS < vecs) {
                    float4 *to = reinterpret_cast<float4 *>(data + head + (i + u * THREADS) * VEC);
                    if constexpr (FP32) {
                        const float4 f = make_float4(__uint_as_float(x[u].x), __uint_as_float(x[u].y), __uint_as_float(x[u].z),
                                                     __uint_as_float(x[u].w));
                        see(f.x), see(f.y), see(f.z), see(f.w);
                        to[0] = f;
                    } else {
                        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            f[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
                            see(f[e]);
                        }
                        to[0] = make_float4(f[0], f[1], f[2], f[3]);
                        to[1] = make_float4(f[4], f[5], f[6], f[7]);
                    }
                }
        }
        if ((int)threadIdx.x < head) one(threadIdx.x);
        const int tail = head + vecs * VEC + (int)threadIdx.x;
        if (tail < n) one(tail);
        if ((int)threadIdx.x < shift) line[threadIdx.x] = -INFINITY;
        if (threadIdx.x < 4) data[n + threadIdx.x] = -INFINITY;
    }
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // the other CTAs have begun
    uint32_t key = bad ? UINT32_MAX : key_of(top);
    {  // the largest of each group of 4 * parts lanes: GROUPS of them in the cluster
        const int size = 4 * parts;
        for (int o = size / 2; o; o /= 2) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
        const int group = (rank * THREADS + (int)threadIdx.x) / size;
        for (int r = lane % size; r < parts; r += size)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_rank(smem_u32(&sh.tops[group]), r)), "r"(key) : "memory");
    }
    __syncwarp();
    cluster_sync();
    key = 0;
    for (int i = lane; i < GROUPS; i += 32) key = max(key, sh.tops[i]);
    key = __reduce_max_sync(0xffffffffu, key);
    bad = key >= KEY_INF;
    top = value_of(key);
    // (one thread) the token at a logit, whose weight is w of `sum`
    auto answer = [&](int token, float l, u64 w, u64 sum) {
        a.tokens[row] = token;
        if (!a.logprobs) return;
        float lp = 0.f;
        if (t > 0.f) {
            if (2 * w > sum) lp = log1pf(-((float)(sum - w) / (float)sum));  // near 0 by what the others weigh
            else lp = 2.f * ((0.5f * l - 0.5f * top) / t) - logf((float)sum * (1.f / (1ull << SCALE)));
        }
        a.logprobs[row] = lp;
    };
    if (bad || !(top > -INFINITY) || !(t >= 0.f && t < INFINITY) || isnan(top_p) || isnan(min_p) || !(u >= 0.f && u < 1.f)) {
        if (rank == 0 && threadIdx.x == 0) {
            a.tokens[row] = -1;
            if (a.logprobs) a.logprobs[row] = __uint_as_float(0x7FC00000u);
            atomicOr(a.status, PQE_STATUS_NO_TOKEN);
        }
        return;
    }

    // a warp's stretch of the row: fours [four0, four1), a lane each 32nd
    const int fours = (shift + n + 3) / 4, per_warp = (fours + THREADS - 1) / THREADS * 32;
    const int four0 = min(fours, warp * per_warp), four1 = min(fours, four0 + per_warp);
    auto four = [&](int g, float(&l)[4]) {
        const float4 v = reinterpret_cast<const float4 *>(line)[g];
        l[0] = v.x, l[1] = v.y, l[2] = v.z, l[3] = v.w;
    };
    auto each4 = [&](auto f) {  // f(four, logits)
        for (int g = four0 + lane; g < four1; g += 32) {
            float l[4];
            four(g, l);
            f(g, l);
        }
    };
    auto index = [&](int g, int j) { return c0 - shift + 4 * g + j; };
    if (t == 0.f) {  // the first of the largest
        int at = INT32_MAX;
        each4([&](int g, const float(&l)[4]) {
#pragma unroll
            for (int j = 3; j >= 0; --j)
                if (l[j] == top) at = min(at, index(g, j));
        });
        at = __reduce_min_sync(0xffffffffu, at);
        __syncthreads();
        if (lane == 0) sh.part[warp] = (u64)at;
        __syncthreads();
        for (int w = 0; w < WARPS; ++w) at = min(at, (int)sh.part[w]);
        u64(*x)[4] = exchange((u64)at, 0, 0, 0);
        bool mine = at != INT32_MAX;
        for (int r = 0; r < rank; ++r) mine &= (int)x[r][0] == INT32_MAX;
        if (mine && threadIdx.x == 0) answer(at, top, 1, 1);
        return;
    }

    Scale sc;
    {
        constexpr float K_HI = 92.33248261689366f, K_LO = (float)(92.33248261689366 - (double)K_HI);  // 64 log2(e)
        sc.half_max = 0.5f * top;
        sc.c_hi = fminf(K_HI / t, 1e38f);
        sc.c_lo = sc.c_hi < 1e38f ? (fmaf(-sc.c_hi, t, K_HI) + K_LO) / t : 0.f;
    }
    // the lowest value that min_p leaves: w >= min_p exactly where l >= max + t ln(min_p)
    float low = -INFINITY;  // (and not equal to it)
    if (min_p >= 1.f) low = top;
    else if (min_p > 0.f) low = __double2float_ru((double)top + sh.min_drop);
    auto in_min = [&](float l) { return l >= low && l > -INFINITY; };

    // what is kept: values above the border, and its equals up to index `last`
    uint32_t border = low > -INFINITY ? key_of(low) : key_of(-INFINITY) + 1;
    int last = INT32_MAX;
    const bool by_k = top_k > 0 && top_k < a.V, by_p = top_p < 1.f;
    if (by_k || by_p) {
        // the elements whose spots lie in [s0, s1], in any order, to the first CTA's list
        auto gather = [&](float s0, float s1, uint32_t &listed, uint32_t room) {
            auto in = [&](float l) {
                const float at = sc.spot(l);
                return in_min(l) && at >= s0 && at <= s1;
            };
            // a lane's own, as bits of its fours
            uint32_t mine = 0, has = 0;
            each4([&](int g, const float(&l)[4]) {
                uint32_t any = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) any += in(l[j]);
                mine += any;
                if (any) has |= 1u << ((g - four0) / 32);
            });
            // a warp takes its places, if it needs any
            const uint32_t upto = warp_scan(mine, lane);
            uint32_t at = 0;
            if (lane == 31 && upto)
                asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;"
                             : "=r"(at)
                             : "r"(map_rank(smem_u32(&listed), 0)), "r"(upto)
                             : "memory");
            at = __shfl_sync(0xffffffffu, at, 31) + upto - mine;
            const uint32_t to_list = map_rank(smem_u32(sh.list), 0);
            for (; has; has &= has - 1) {
                const int g = four0 + 32 * (__ffs(has) - 1) + lane;
                float l[4];
                four(g, l);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (in(l[j])) {
                        if (at < room) st_remote(to_list + 8 * at, (u64)~key_of(l[j]) << 32 | (uint32_t)index(g, j));
                        ++at;
                    }
            }
            __syncwarp();
            cluster_sync();
        };
        auto by_key = [](u64 v) { return value_of(~(uint32_t)(v >> 32)); };

        // (first CTA) the rest, from a list of m <= RANKED that holds all that top_k or top_p may leave: each compares itself with
        // each. `total` is the weight of the row
        auto finish = [&](int m, bool cut_k, u64 total) {
            const int i = threadIdx.x;
            const u64 v = i < m ? sh.list[i] : 0;
            const float l = by_key(v);
            const u64 w = i < m ? sc.weight_of(sh.weight, l) : 0;
            if (i < m) sh.spare[i] = w;
            __syncthreads();
            int before = 0;
            u64 above = 0;
            if (i < m)
#pragma unroll 4
                for (int j = 0; j < m; ++j)
                    if (sh.list[j] < v) ++before, above += sh.spare[j];
            bool stays = i < m && (!cut_k || before < top_k);
            if (by_p) {
                const u64 sum = block_sum(sh, stays ? w : 0);
                stays = stays && (before == 0 || above < share_up(top_p, cut_k ? sum : total));
            }
            __syncthreads();
            if (i < m) sh.spare[i] = stays ? w : 0;
            __syncthreads();
            u64 lower = 0;
            if (i < m)
#pragma unroll 4
                for (int j = 0; j < m; ++j)
                    if ((uint32_t)sh.list[j] < (uint32_t)v) lower += sh.spare[j];
            const u64 sum = block_sum(sh, stays ? w : 0), want = share(u, sum);
            if (stays && lower <= want && want < lower + w) answer((int)(uint32_t)v, l, w, sum);
        };
        // ---- a small top_k: at least that many logits are not below the top_k-th of the groups' largest, and hardly more ----
        if (by_k && top_k <= FEW_K) {
            if ((int)threadIdx.x < GROUPS) {
                const uint32_t mine = sh.tops[threadIdx.x];
                int before = 0;
#pragma unroll 8
                for (int i = 0; i < GROUPS; ++i) {
                    const uint32_t x = sh.tops[i];
                    before += x > mine || (x == mine && i < (int)threadIdx.x);
                }
                if (before == top_k - 1) sh.floor = mine > KEY_NEG_INF ? value_of(mine) : -INFINITY;
            }
            __syncthreads();
            // (spots rise as logits fall: all of the floor's spot come along)
            gather(Scale::spot_of(0), sc.spot(sh.floor), sh.listed[0], RANKED);
            const uint32_t m = ld_remote(map_rank(smem_u32(&sh.listed[0]), 0));
            if (m <= RANKED) {
                __syncwarp();
                asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
                if (rank != 0) return;
                finish((int)m, true, 0);
                __syncwarp();
                asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // all have read the count here
                return;
            }
        }
        // ---- the histogram. What weighs nothing is only counted. Without top_k so is, with its weight, what all of a row's V logits
        // together could not lift over 1 - top_p of the largest's weight alone: it holds no border ----
        const int limit = by_k || top_p <= 0.f ? FAR : min(FAR, (int)((float)OCTAVE * log2f((float)a.V / (1.f - top_p))) + 3);
        uint32_t far_count = 0;
        u64 far_mass = 0;
        if (by_p)
            each4([&](int, const float(&l)[4]) {
                int b[4];
                u64 w[4];
                sc.weigh(sh.weight, l, b, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (!in_min(l[j])) continue;
                    if (b[j] >= limit) {
                        ++far_count;
                        far_mass += w[j];
                        continue;
                    }
                    const uint32_t over = (uint32_t)((int)(w[j] >> Scale::drop(b[j])) - Scale::base(sh.weight, b[j]));  // 25 bits
                    atomicAdd(&sh.count[b[j]], 1u);
                    atomicAdd(&sh.lo[b[j]], over & 4095u);
                    atomicAdd(&sh.hi[b[j]], over >> 12);
                }
            });
        else
            each4([&](int, const float(&l)[4]) {
                int b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = Scale::bin(sc.spot(l[j]));
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (in_min(l[j])) {
                        if (b[j] >= FAR) ++far_count;
                        else atomicAdd(&sh.count[b[j]], 1u);
                    }
            });
        __syncwarp();
        cluster_sync();
        // ---- a slice of the bins from every CTA, merged in place ----
        const int per = BINS >> parts_log, own = rank * per, width = (per + THREADS - 1) / THREADS;  // neighbouring bins of a thread
        const int bin0 = own + min((int)threadIdx.x * width, per), bin1 = min(bin0 + width, own + per);
        uint32_t bins_count = 0;
        u64 bins_mass = 0;
        for (int b = bin0; b < bin1; ++b) {
            uint32_t c = 0;
            u64 s = 0;
#pragma unroll 4
            for (int r = 0; r < parts; ++r) {
                c += ld_remote(map_rank(smem_u32(&sh.count[b]), r));
                if (by_p)
                    s += ld_remote(map_rank(smem_u32(&sh.lo[b]), r)) + ((u64)ld_remote(map_rank(smem_u32(&sh.hi[b]), r)) << 12);
            }
            const u64 w = c && by_p ? (s + (u64)((int64_t)c * Scale::base(sh.weight, b))) << Scale::drop(b) : 0;
            sh.count[b] = c;
            sh.lo[b] = (uint32_t)w;
            sh.hi[b] = (uint32_t)(w >> 32);
            bins_count += c;
            bins_mass += w;
        }
        uint32_t slice_count = 0, far_all_count = 0, count_to = warp_scan(bins_count, lane);
        u64 slice_mass = 0, far_all_mass = 0, mass_to = by_p ? warp_scan(bins_mass, lane) : 0;
        far_count = __reduce_add_sync(0xffffffffu, far_count);
        if (by_p)
#pragma unroll
            for (int o = 16; o; o /= 2) far_mass += __shfl_xor_sync(0xffffffffu, far_mass, o);
        __syncthreads();
        if (lane == 31) sh.parts[warp] = {mass_to, far_mass, count_to, far_count};
        __syncthreads();
        {
            uint32_t c0_ = 0;
            u64 m0 = 0;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                if (w == warp) c0_ = slice_count, m0 = slice_mass;
                slice_count += sh.parts[w].count, slice_mass += sh.parts[w].mass;
                far_all_count += sh.parts[w].far_count, far_all_mass += sh.parts[w].far_mass;
            }
            count_to += c0_, mass_to += m0;
        }
        u64 total_count = 0, total_mass = 0, before_count = 0, before_mass = 0;
        {
            u64(*x)[4] = exchange(slice_count, slice_mass, far_all_count, far_all_mass);
            for (int r = 0; r < parts; ++r) {
                if (r < rank) before_count += x[r][0], before_mass += x[r][1];
                total_count += x[r][0] + x[r][2];
                total_mass += x[r][1] + x[r][3];
            }
        }
        // the first bin with `least` elements (or weight) up to its end; every CTA learns it
        auto find = [&](bool counts, u64 least) {
            auto enough = [&](u64 c, u64 m) { return (counts ? c : m) >= least; };
            if (threadIdx.x == 0) sh.found.bin = -1;
            __syncthreads();
            u64 c = before_count + count_to - bins_count, m = before_mass + mass_to - bins_mass;
            const bool had = before_count + count_to - bins_count > 0 && enough(c, m);
            if (!had && enough(c + bins_count, m + bins_mass))
                for (int b = bin0; b < bin1; ++b) {
                    const u64 c1 = c + sh.count[b], m1 = m + ((u64)sh.hi[b] << 32 | sh.lo[b]);
                    if (c1 > c && enough(c1, m1)) {
                        sh.found = {b, (uint32_t)c, (uint32_t)(c1 - c), m};
                        break;
                    }
                    c = c1, m = m1;
                }
            __syncthreads();
            const Found f = sh.found;
            u64(*x)[4] = exchange((u64)(uint32_t)f.bin << 32 | f.count, f.in, f.mass, 0);
            Found got{-1, 0, 0, 0};
            for (int r = 0; r < parts && got.bin < 0; ++r)
                got = {(int)(uint32_t)(x[r][0] >> 32), (uint32_t)x[r][0], (uint32_t)x[r][1], x[r][2]};
            return got;
        };
        bool cut_k = by_k && total_count > (u64)top_k;
        Found f{-1, 0, 0, 0};
        if (cut_k) {
            f = find(true, (u64)top_k);
            cut_k = f.bin >= 0;  // (else what is cut weighs nothing)
        }
        if (!cut_k && by_p) f = find(false, share_up(top_p, total_mass));
        if (f.bin >= 0 && (u64)f.count + f.in <= RANKED) {
            // ---- few candidates down to the border's bin: the first CTA does the rest ----
            gather(Scale::spot_of(0), Scale::spot_of(f.bin), sh.listed[1], RANKED);
            if (rank == 0) finish((int)(f.count + f.in), cut_k, total_mass);
            return;
        }
        // ---- the border's value alone ----
        u64 equals = ~0ull;       // of the border's own equals: this many
        u64 ties = 0;             // there are so many of them
        u64 kept_mass = total_mass;
        // (first CTA) a bin's list in order, with sums up to each: the border's key, how many of its equals are kept, how many there
        // are, and the weight of all that is kept
        auto ordered = [&](auto halves, const Found &g, bool counts, u64 least, u64(&got)[4]) {
            constexpr int H = decltype(halves)::value;
            const int m = (int)g.in;
            u64 v[H], sums[H], all, run = g.mass;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int i = threadIdx.x + h * THREADS;
                v[h] = i < m ? sh.list[i] : ~0ull;
            }
            int size = 2;
            while (size < m) size *= 2;
            sort<H>(sh.list, v, size);
            int short_of = 0;  // elements that are not enough: the next one is the border's
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int i = threadIdx.x + h * THREADS;
                const u64 own = i < m && by_p ? sc.weight_of(sh.weight, by_key(v[h])) : 0;
                sums[h] = run + block_scan(sh, own, all);
                run += all;
                short_of += __syncthreads_count(i < m && (counts ? g.count + i + 1 < least : sums[h] < least));
            }
            const int at = min(short_of, m - 1);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int i = threadIdx.x + h * THREADS;
                if (i == at) sh.found = {0, ~(uint32_t)(v[h] >> 32), 0, sums[h]};
            }
            __syncthreads();
            got[0] = sh.found.count;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int i = threadIdx.x + h * THREADS;
                const bool same = i < m && ~(uint32_t)(v[h] >> 32) == (uint32_t)got[0];
                got[1] += __syncthreads_count(same && i <= at);
                got[2] += __syncthreads_count(same);
            }
            got[3] = sh.found.mass;
        };
        // border, equals, ties from the bin where it falls: `least` elements from the row's first (or weight); returns the weight
        // of all that is kept
        auto refine = [&](const Found &g, bool counts, u64 least, uint32_t &listed) -> u64 {
            if (g.in <= LIST) {
                gather(Scale::spot_of(g.bin), Scale::spot_of(g.bin), listed, LIST);
                u64 got[4] = {};
                if (rank == 0) {
                    if (g.in <= THREADS) ordered(std::integral_constant<int, 1>(), g, counts, least, got);
                    else ordered(std::integral_constant<int, 2>(), g, counts, least, got);
                }
                u64(*x)[4] = exchange(got[0], got[1], got[2], got[3]);
                border = (uint32_t)x[0][0], equals = x[0][1], ties = x[0][2];
                return x[0][3];
            }
            auto inside = [&](float l) { return in_min(l) && Scale::bin(sc.spot(l)) == g.bin; };
            // count and sum of the bin's elements from key k on
            auto since = [&](uint32_t k, u64 &c, u64 &m) {
                uint32_t nc = 0, nc_all;
                u64 nm = 0, nm_all;
                each4([&](int, const float(&l)[4]) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (inside(l[j]) && key_of(l[j]) >= k) ++nc, nm += sc.weight_of(sh.weight, l[j]);
                });
                block_scan(sh, nc, nm, nc_all, nm_all);
                u64(*x)[4] = exchange(nc_all, nm_all, 0, 0);
                c = g.count, m = g.mass;
                for (int r = 0; r < parts; ++r) c += x[r][0], m += x[r][1];
            };
            uint32_t lo = UINT32_MAX, hi = 0;
            each4([&](int, const float(&l)[4]) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (inside(l[j])) lo = min(lo, key_of(l[j])), hi = max(hi, key_of(l[j]));
            });
            lo = __reduce_min_sync(0xffffffffu, lo), hi = __reduce_max_sync(0xffffffffu, hi);
            __syncthreads();
            if (lane == 0) sh.part[threadIdx.x >> 5] = (u64)lo << 32 | hi;
            __syncthreads();
            for (int w = 0; w < WARPS; ++w) lo = min(lo, (uint32_t)(sh.part[w] >> 32)), hi = max(hi, (uint32_t)sh.part[w]);
            {
                u64(*x)[4] = exchange(lo, hi, 0, 0);
                for (int r = 0; r < parts; ++r) lo = min(lo, (uint32_t)x[r][0]), hi = max(hi, (uint32_t)x[r][1]);
            }
            u64 c, m;
            while (lo < hi) {  // the largest key that gives enough
                const uint32_t mid = lo + (hi - lo + 1) / 2;
                since(mid, c, m);
                if ((counts ? c : m) >= least) lo = mid;
                else hi = mid - 1;
            }
            border = lo;
            u64 c1, m1;
            since(lo, c1, m1);
            since(lo + 1, c, m);  // (an infinity's key is above every other's)
            ties = c1 - c;
            const u64 w = ties ? (m1 - m) / ties : 0;
            equals = counts ? least - c : w && least > m ? (least - m + w - 1) / w : 1;
            equals = min(equals, ties);
            return m + equals * w;
        };
        if (cut_k) kept_mass = refine(f, true, (u64)top_k, sh.listed[2]);
        if (by_p) {
            const u64 want = share_up(top_p, kept_mass);
            const uint32_t k_border = border;
            const u64 k_equals = equals, k_ties = ties;
            const Found g = cut_k ? find(false, want) : f;
            if (g.bin >= 0 && !(cut_k && g.bin > f.bin)) {
                refine(g, false, want, sh.listed[3]);
                if (cut_k && border < k_border) border = k_border, equals = k_equals, ties = k_ties;
                else if (cut_k && border == k_border) equals = min(equals, k_equals);
            }
        }
        if (equals < ties) {  // the index of the last equal that is kept
            uint32_t mine = 0, all;
            const float value = value_of(border);
            each4([&](int, const float(&l)[4]) {
#pragma unroll
                for (int j = 0; j < 4; ++j) mine += l[j] == value;
            });
            mine = __reduce_add_sync(0xffffffffu, mine);
            const uint32_t upto = block_scan(sh, lane == 31 ? mine : 0u, all);  // (lane 31: up to the warp's end)
            u64 before = 0;
            {
                u64(*x)[4] = exchange(all, 0, 0, 0);
                for (int r = 0; r < rank; ++r) before += x[r][0];
            }
            if (threadIdx.x == 0) sh.part[0] = ~0ull;
            __syncthreads();
            u64 c = before + __shfl_sync(0xffffffffu, upto, 31) - mine;  // before the warp
            if (c < equals && equals <= c + mine)
                for (int g0 = four0; g0 < four1; g0 += 32) {
                    float l[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    if (g0 + lane < four1) four(g0 + lane, l);
                    uint32_t own = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) own += l[j] == value;
                    const uint32_t to_here = warp_scan(own, lane);
                    if (c + to_here - own < equals && equals <= c + to_here) {
                        uint32_t at = (uint32_t)(equals - (c + to_here - own));
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (l[j] == value && --at == 0) sh.part[0] = (u64)index(g0 + lane, j);
                    }
                    c += __shfl_sync(0xffffffffu, to_here, 31);
                }
            __syncthreads();
            u64(*x)[4] = exchange(sh.part[0], 0, 0, 0);
            for (int r = 0; r < parts; ++r)
                if (x[r][0] != ~0ull) last = (int)x[r][0];
        }
    }

    // ---- the kept weights' sums in index order, and where u falls ----
    const float value = value_of(border);
    auto kept = [&](float l, int i) { return l > value || (l == value && i <= last); };
    auto weights = [&](int g, const float(&l)[4], u64 sum) {  // sum + those of a four
        int b[4];
        u64 w[4];
        sc.weigh(sh.weight, l, b, w);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (kept(l[j], index(g, j))) sum += w[j];
        return sum;
    };
    u64 mine = 0, all;
    if (last == INT32_MAX)
        each4([&](int, const float(&l)[4]) {
            if (fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])) < value) return;
            int b[4];
            u64 w[4];
            sc.weigh(sh.weight, l, b, w);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (l[j] >= value) mine += w[j];
        });
    else each4([&](int g, const float(&l)[4]) { mine = weights(g, l, mine); });
    const u64 upto = block_scan(sh, mine, all);
    u64 before = 0, sum = 0;
    {
        u64(*x)[4] = exchange(all, 0, 0, 0);
        for (int r = 0; r < parts; ++r) {
            if (r < rank) before += x[r][0];
            sum += x[r][0];
        }
    }
    const u64 want = share(u, sum), warp_end = before + __shfl_sync(0xffffffffu, upto, 31);
    u64 at = before + __shfl_sync(0xffffffffu, upto - mine, 0);
    if (at > want || warp_end <= want) return;
    // one warp of all: it walks its stretch
    for (int g0 = four0; g0 < four1; g0 += 32) {
        float l[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (g0 + lane < four1) four(g0 + lane, l);
        const u64 own = weights(g0 + lane, l, 0), to_here = at + warp_scan(own, lane);
        const uint32_t past = __ballot_sync(0xffffffffu, to_here > want);
        if (past) {
            if (lane == __ffs(past) - 1) {
                u64 c = to_here - own;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const u64 w = kept(l[j], index(g0 + lane, j)) ? sc.weight_of(sh.weight, l[j]) : 0;
                    if (c <= want && c + w > want) answer(index(g0 + lane, j), l[j], w, sum);
                    c += w;
                }
            }
            return;
        }
        at = __shfl_sync(0xffffffffu, to_here, 31);
    }
}

template <bool FP32>
static int launch(const Args &a, int B, cudaStream_t s) {
    static std::atomic<int> attr_set[PQE_MAX_DEVICES];
    int dev = 0, sms = 0;
    const int rc = device_info(dev, sms);
    if (rc != PQE_OK) return rc;
    if (!attr_set[dev].load(std::memory_order_relaxed)) {
        PQE_CUDA_TRY(cudaFuncSetAttribute(sample_kernel<FP32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          (int)(HEAD + CHUNK_MAX * sizeof(float))));
        attr_set[dev].store(1, std::memory_order_relaxed);
    }
    // as few CTAs a row as leave room for two on an SM; more where SMs would stay idle
    int log = 0;
    while (log < 3 && (a.V + (1 << log) - 1) >> log > CHUNK_TWO) ++log;
    while (log < 3 && ((int64_t)B << (log + 1)) <= sms && a.V >> (log + 1) >= 2048) ++log;
    const int chunk = (a.V + (1 << log) - 1) >> log;
    if (((int64_t)B << log) > INT32_MAX) return PQE_ERR_INVALID_ARG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)B << log);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = HEAD + (size_t)chunk * sizeof(float);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 1u << log;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    PQE_CUDA_TRY(cudaLaunchKernelEx(&cfg, sample_kernel<FP32>, a, log, chunk));
    count_launch();
    return PQE_OK;
}

}  // namespace sampling
}  // namespace pqe

using namespace pqe;

extern "C" {

int sample_tokens(const void *logits, int fp32, int64_t stride, int B, int V, const float *temperature,
                  const int32_t *top_k, const float *top_p, const float *min_p, const float *u, int32_t *tokens,
                  float *logprobs, int32_t *status, void *stream) {
    PQE_CHECK_ARG(B >= 0 && V >= 1 && V <= sampling::MAX_PARTS * sampling::CHUNK_MAX);
    if (B == 0) return PQE_OK;
    PQE_CHECK_ARG(logits && u && tokens && status && stride >= V && aligned(logits, fp32 ? 4 : 2));
    PQE_CHECK_ARG(aligned(temperature, 4) && aligned(top_k, 4) && aligned(top_p, 4) && aligned(min_p, 4) && aligned(u, 4) &&
                  aligned(tokens, 4) && aligned(logprobs, 4) && aligned(status, 4));
    const sampling::Args a{logits, stride, V, temperature, top_p, min_p, u, top_k, tokens, status, logprobs};
    return fp32 ? sampling::launch<true>(a, B, as_stream(stream)) : sampling::launch<false>(a, B, as_stream(stream));
}

}  // extern "C"
