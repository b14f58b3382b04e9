// sample.cu -- sample_tokens: the next token of each row of logits.
//
// What is kept of a row is a beginning of its order (logits descending, lower index first), and the token is where the sum of
// the kept weights, in index order, passes u times their total. A row lies in the shared memory of a cluster of 1 to 8 CTAs, so
// logits are read once; sums are whole numbers (weights times 2^43), the same in any order.
//
//   all kept (no top_k, no top_p)  a sum for each thread's stretch of the row, a scan, and the thread whose stretch u falls
//                                  into walks it.
//   a border to be found           a histogram of the logits, 32 bins for each factor of two of the weights: counts, and for
//                                  top_p sums. The bins are merged in slices, a CTA each; the CTA whose slice the border falls
//                                  into finds the bin. Where what lies above the border's bin and in it fits a list (2048),
//                                  the first CTA sorts and finishes it. Otherwise the bin alone goes to a list (1024), which
//                                  gives the border's value and how many of its equals are kept, and the row is walked as above.
//   more than that in one bin      (thousands of equal logits, or nearly) bisection on the values' bits.
//
// Weights: with P = 32 log2(e) (max - l) / t, its whole part n and rest f, w = 2^(-n / 32) 2^(-f / 32): the first factor from a
// table of 32 and a shift, the second from five terms of its series. P is held in two floats: 2^-29 of a weight, against which
// a sum of thousands of them is more exact still. u of 24 bits falls so near a border of two tokens that it matters about once
// in a million rows of 10^5 nearly equal tokens.
#include <math.h>

#include <atomic>

#include "pqe_common.cuh"
#include "tc_ptx.cuh"

namespace pqe {
namespace sampling {
using namespace ptx;
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
constexpr int BINS = 2048, OCTAVE = 32;      // bins in all, and for a factor of two
constexpr int LAST_MASS = 44 * OCTAVE;       // bins from here on weigh less than 2^-44 each: nothing
constexpr int LIST = 2048, INNER = 1024;     // candidates that one CTA sorts: all of a row's, or a bin's
constexpr int MAX_PARTS = 8;
constexpr int SCALE = 43;                    // the largest logit's weight: 2^43; 2^18.6 of them fit 63 bits
constexpr int CHUNK_MAX = 49152;             // logits of a CTA; sums of a bin's 13-bit parts stay below 2^32
static_assert((int64_t)CHUNK_MAX << 13 < (int64_t)1 << 32, "");

// 2^30 2^(-i / 32)
__constant__ int32_t TABLE[OCTAVE + 1] = {
    1073741824, 1050733751, 1028218693, 1006186087, 984625594, 963527098, 942880699, 922676710, 902905651, 883558244, 864625413,
    846098274, 827968132, 810226483, 792865000, 775875538, 759250125, 742980960, 727060411, 711481005, 696235434, 681316545,
    666717336, 652430958, 638450708, 624770026, 611382493, 598281827, 585461881, 572916640, 560640218, 548626854, 536870912};
constexpr int SLACK = 8192;                  // a mantissa is at most this much under its bin's end (roundings of P)

// Whole numbers that order as the values do (-0 as +0); -infinity gives KEY_NEG_INF, NaN below it or above +infinity's.
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
    u64 part[WARPS];                  // of block scans
    uint32_t count_part[WARPS];
    u64 swap[4][MAX_PARTS][4];        // of the cluster's exchanges, four in turn
    int32_t table[OCTAVE + 1];        // TABLE
    uint32_t listed[3];               // entries of the list, of the inner one, of that once more
    double min_drop;                  // t ln(min_p)
    Found found;
    u64 inner[INNER];
    union {
        struct {
            uint32_t count[BINS];     // merged in place: counts, and sums of weights as (low, high) words
            uint32_t lo[BINS], hi[BINS];
        };
        u64 list[LIST];
    };
};

// What a row's weights go by.
struct Scale {
    float half_max, c_hi, c_lo;  // max / 2, and 64 log2(e) / t in two parts (values enter halved: their difference does not overflow)
    __device__ __forceinline__ float place(float l) const { return (half_max - 0.5f * l) * c_hi; }  // P, of 24 bits: rises as l falls
    __device__ __forceinline__ static int bin(float p) { return p < (float)(BINS - 1) ? (int)p : BINS - 1; }
    // w / 2^(n / 32 rounded down) times 2^30 of a logit at p < LAST_MASS in bin n
    __device__ __forceinline__ uint32_t mantissa(const int32_t *table, float l, float p, int n) const {
        const float a = 0.5f * l, s = half_max - a;  // and what rounding took: s + e = half_max - a
        const float b = s - half_max, e = (half_max - (s - b)) - (a + b);
        const float f = (p - (float)n) + (fmaf(s, c_hi, -p) + fmaf(s, c_lo, e * c_hi));
        const float r = f * 0.0216608493924982909f;  // ln(2) / 32
        const float q = r * fmaf(r, fmaf(r, fmaf(r, fmaf(r, 1.f / 120, -1.f / 24), 1.f / 6), -0.5f), 1.f);  // 1 - exp(-r)
        const int t = table[n % OCTAVE];
        return (uint32_t)(t - (int)(((int64_t)t * __float2int_rn(q * 2147483648.f)) >> 31));
    }
    __device__ __forceinline__ static u64 shifted(u64 mantissas, int n) {  // sums of mantissas of a bin, as weights
        const int by = n / OCTAVE;
        return ((mantissas << (SCALE - 30)) + ((1ull << by) >> 1)) >> by;
    }
    __device__ __forceinline__ u64 weight(const int32_t *table, float l) const {
        const float p = place(l);
        const int n = bin(p);
        const u64 w = shifted(mantissa(table, l, p, n), n < LAST_MASS ? n : 0);
        return n < LAST_MASS ? w : 0;
    }
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

// ascending sort of n values (a power of two) by the whole CTA
__device__ __forceinline__ void sort(u64 *v, int n) {
    for (int k = 2; k <= n; k *= 2)
        for (int j = k / 2; j > 0; j /= 2) {
            __syncthreads();
            for (int i = threadIdx.x; i < n / 2; i += THREADS) {
                const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
                const u64 a = v[lo], b = v[hi];
                if ((a > b) == ((lo & k) == 0)) v[lo] = b, v[hi] = a;
            }
        }
    __syncthreads();
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
    float *data = reinterpret_cast<float *>(smem + (sizeof(Shared) + 127) / 128 * 128);
    const int lane = threadIdx.x & 31, parts = 1 << parts_log;
    const int rank = (int)cluster_rank();
    const int64_t row = blockIdx.x >> parts_log;
    const int c0 = rank * chunk, n = max(0, min(chunk, a.V - c0));
    int swaps = 0;

    // every CTA's four values to every CTA
    auto exchange = [&](u64 v0, u64 v1, u64 v2, u64 v3) -> u64(*)[4] {
        u64(*slot)[4] = sh.swap[swaps++ & 3];
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
    if (threadIdx.x <= OCTAVE) sh.table[threadIdx.x] = TABLE[threadIdx.x];
    if (threadIdx.x < 3) sh.listed[threadIdx.x] = 0;
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
        data += (VEC - head) & (VEC - 1);  // pieces are aligned here too
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
    }
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // the other CTAs have begun
    bad = __any_sync(0xffffffffu, bad);
    uint32_t key = __reduce_max_sync(0xffffffffu, key_of(top));
    if (lane == 0) sh.part[threadIdx.x >> 5] = (u64)bad << 32 | key;
    __syncthreads();
    for (int w = 0; w < WARPS; ++w) {
        bad |= (sh.part[w] >> 32) != 0;
        key = max(key, (uint32_t)sh.part[w]);
    }
    {
        u64(*x)[4] = exchange(key, bad, 0, 0);
        for (int r = 0; r < parts; ++r) key = max(key, (uint32_t)x[r][0]), bad |= x[r][1] != 0;
    }
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

    // a thread's stretch of the row, four logits at a time (behind its end: -infinity); an odd length keeps the threads of a warp in different banks
    const int len = ((chunk + THREADS - 1) / THREADS) | 1, from = min(n, (int)threadIdx.x * len), to = min(n, from + len);
    auto each4 = [&](auto f) {
        for (int i = from; i < to; i += 4) {
            float l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) l[j] = i + j < to ? data[i + j] : -INFINITY;
            f(i, l);
        }
    };
    if (t == 0.f) {  // the first of the largest
        int at = INT32_MAX;
        for (int i = from; i < to && at == INT32_MAX; ++i)
            if (data[i] == top) at = c0 + i;
        at = __reduce_min_sync(0xffffffffu, at);
        __syncthreads();
        if (lane == 0) sh.part[threadIdx.x >> 5] = (u64)at;
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
        // ---- the histogram. Below `prune` all of a row's V logits together are less than 1 - top_p of the largest's weight alone:
        // they hold no border, and go into two sums instead ----
        const float prune = by_k || top_p <= 0.f ? INFINITY : ceilf((float)OCTAVE * log2f((float)a.V / (1.f - top_p)) + 1.f);
        uint32_t far_count = 0;
        u64 far_mass = 0;
        if (by_p)
            each4([&](int, const float(&l)[4]) {
                int b[4];
                uint32_t w[4];
                bool near[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = sc.place(l[j]);
                    b[j] = Scale::bin(p);
                    near[j] = p < prune;
                    w[j] = b[j] < LAST_MASS ? sc.mantissa(sh.table, l[j], p, b[j]) : 0;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (!in_min(l[j])) continue;
                    if (!near[j]) {
                        ++far_count;
                        far_mass += Scale::shifted(w[j], min(b[j], LAST_MASS - 1));
                        continue;
                    }
                    atomicAdd(&sh.count[b[j]], 1u);
                    if (b[j] >= LAST_MASS) continue;
                    // what is above the bin's lower end, less a little for roundings: 25 bits
                    const uint32_t over = w[j] - (uint32_t)(sh.table[b[j] % OCTAVE + 1] - SLACK);
                    atomicAdd(&sh.lo[b[j]], over & 4095u);
                    atomicAdd(&sh.hi[b[j]], over >> 12);
                }
            });
        else
            each4([&](int, const float(&l)[4]) {
                int b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = Scale::bin(sc.place(l[j]));
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (in_min(l[j])) atomicAdd(&sh.count[b[j]], 1u);
            });
        __syncwarp();
        cluster_sync();
        // ---- a slice of the bins from every CTA, merged in place ----
        const int per = BINS >> parts_log, own = rank * per, width = max(1, per / THREADS);  // neighbouring bins of a thread
        uint32_t bins_count = 0;
        u64 bins_mass = 0;
        if ((int)threadIdx.x * width < per)
            for (int b = own + threadIdx.x * width, e = b + width; b < e; ++b) {
                uint32_t c = 0;
                u64 s = 0;
#pragma unroll 4
                for (int r = 0; r < parts; ++r) {
                    c += ld_remote(map_rank(smem_u32(&sh.count[b]), r));
                    if (by_p)
                        s += ld_remote(map_rank(smem_u32(&sh.lo[b]), r)) + ((u64)ld_remote(map_rank(smem_u32(&sh.hi[b]), r)) << 12);
                }
                const u64 w = by_p && b < LAST_MASS ? Scale::shifted(s + c * (u64)(sh.table[b % OCTAVE + 1] - SLACK), b) : 0;
                sh.count[b] = c;
                sh.lo[b] = (uint32_t)w;
                sh.hi[b] = (uint32_t)(w >> 32);
                bins_count += c;
                bins_mass += w;
            }
        uint32_t slice_count, far_all_count = 0, count_to = bins_count;
        u64 slice_mass, far_all_mass = 0, mass_to = bins_mass;
        block_scan(sh, count_to, mass_to, slice_count, slice_mass);
        if (by_p) block_scan(sh, far_count, far_mass, far_all_count, far_all_mass);
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
            if ((int)threadIdx.x * width < per && !had && enough(c + bins_count, m + bins_mass))
                for (int b = own + threadIdx.x * width;; ++b) {
                    const u64 c1 = c + sh.count[b], m1 = m + ((u64)sh.hi[b] << 32 | sh.lo[b]);
                    if (c1 > c && enough(c1, m1)) {
                        sh.found = {b, (uint32_t)c, (uint32_t)(c1 - c), m};
                        break;
                    }
                    c = c1, m = m1;
                    if (b + 1 == own + (int)threadIdx.x * width + width) break;
                }
            __syncthreads();
            const Found f = sh.found;
            u64(*x)[4] = exchange((u64)(uint32_t)f.bin << 32 | f.count, f.in, f.mass, 0);
            Found got{-1, 0, 0, 0};
            for (int r = 0; r < parts && got.bin < 0; ++r)
                got = {(int)(uint32_t)(x[r][0] >> 32), (uint32_t)x[r][0], (uint32_t)x[r][1], x[r][2]};
            return got;
        };
        // the elements in bins [b0, b1], in any order, to a list of the first CTA
        auto gather = [&](int b0, int b1, u64 *list, uint32_t &listed, uint32_t room) {
            auto in = [&](float l) {
                if (!in_min(l)) return false;
                const int b = Scale::bin(sc.place(l));
                return b >= b0 && b <= b1;
            };
            // a thread's own, as bits of the fours of its stretch
            uint32_t mine = 0, fours = 0;
            each4([&](int i, const float(&l)[4]) {
                uint32_t any = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) any += in(l[j]);
                mine += any;
                if (any) fours |= 1u << ((i - from) >> 2);
            });
            uint32_t all;
            const uint32_t upto = block_scan(sh, mine, all);
            __syncthreads();
            if (threadIdx.x == 0) {
                uint32_t at;
                asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;"
                             : "=r"(at)
                             : "r"(map_rank(smem_u32(&listed), 0)), "r"(all)
                             : "memory");
                sh.part[0] = at;
            }
            __syncthreads();
            uint32_t at = (uint32_t)sh.part[0] + upto - mine;
            const uint32_t to_list = map_rank(smem_u32(list), 0);
            for (; fours; fours &= fours - 1) {
                const int i0 = from + 4 * (__ffs(fours) - 1);
                for (int i = i0; i < min(i0 + 4, to); ++i)
                    if (in(data[i])) {
                        if (at < room) st_remote(to_list + 8 * at, (u64)~key_of(data[i]) << 32 | (uint32_t)(c0 + i));
                        ++at;
                    }
            }
            __syncwarp();
            cluster_sync();
        };
        // (first CTA) a list in order, padded to a power of two
        auto sort_list = [&](u64 *list, int m) {
            int size = 2;
            while (size < m) size *= 2;
            for (int i = m + threadIdx.x; i < size; i += THREADS) list[i] = ~0ull;
            sort(list, size);
        };
        constexpr int EACH = LIST / THREADS;
        // (first CTA) sums of the first m of the list, whose values `value` gives, for the EACH elements of a thread from `sums`:
        // inclusive sums
        auto list_sums = [&](const u64 *list, int m, auto value, u64(&sums)[EACH]) {
            u64 run = 0;
#pragma unroll
            for (int j = 0; j < EACH; ++j) {
                const int i = threadIdx.x * EACH + j;
                if (i < m) run += sc.weight(sh.table, value(list[i]));
                sums[j] = run;
            }
            u64 total;
            const u64 upto = block_scan(sh, run, total);
#pragma unroll
            for (int j = 0; j < EACH; ++j) sums[j] += upto - run;
            return total;
        };
        auto first_where = [&](int none, const bool(&is)[EACH]) {  // the lowest index of the list where `is`, or none
            int at = INT32_MAX;
#pragma unroll
            for (int j = EACH - 1; j >= 0; --j)
                if (is[j]) at = threadIdx.x * EACH + j;
            at = __reduce_min_sync(0xffffffffu, at);
            __syncthreads();
            if (lane == 0) sh.part[threadIdx.x >> 5] = (u64)at;
            __syncthreads();
            for (int w = 0; w < WARPS; ++w) at = min(at, (int)sh.part[w]);
            __syncthreads();
            return at == INT32_MAX ? none : at;
        };
        auto by_key = [](u64 v) { return value_of(~(uint32_t)(v >> 32)); };

        const bool cut_k = by_k && total_count > (u64)top_k;
        Found f{-1, 0, 0, 0};
        if (cut_k) f = find(true, (u64)top_k);
        else if (by_p) f = find(false, share_up(top_p, total_mass));
        if (f.bin >= 0 && (u64)f.count + f.in <= LIST) {
            // ---- a list of everything down to the border's bin: the first CTA does the rest ----
            gather(0, f.bin, sh.list, sh.listed[0], LIST);
            if (rank != 0) return;
            const int m = (int)(f.count + f.in);
            sort_list(sh.list, m);
            int keep = cut_k ? min(m, top_k) : m;
            u64 sums[EACH];
            bool is[EACH];
            if (by_p) {
                const u64 sum = list_sums(sh.list, keep, by_key, sums);
                const u64 want = share_up(top_p, cut_k ? sum : total_mass);
#pragma unroll
                for (int j = 0; j < EACH; ++j) is[j] = (int)threadIdx.x * EACH + j < keep && sums[j] >= want;
                keep = first_where(keep - 1, is) + 1;
            }
            // the kept ones by index
            int size = 2;
            while (size < keep) size *= 2;
            for (int i = threadIdx.x; i < size; i += THREADS) sh.list[i] = i < keep ? sh.list[i] << 32 | sh.list[i] >> 32 : ~0ull;
            sort(sh.list, size);
            auto by_index = [](u64 v) { return value_of(~(uint32_t)v); };
            const u64 sum = list_sums(sh.list, keep, by_index, sums);
            const u64 want = share(u, sum);
#pragma unroll
            for (int j = 0; j < EACH; ++j) is[j] = (int)threadIdx.x * EACH + j < keep && sums[j] > want;
            const int at = first_where(keep - 1, is);
            if (threadIdx.x == 0) {
                const float l = by_index(sh.list[at]);
                answer((int)(sh.list[at] >> 32), l, sc.weight(sh.table, l), sum);
            }
            return;
        }
        // ---- the border's value alone ----
        u64 equals = ~0ull;       // of the border's own equals: this many
        u64 ties = 0;             // there are so many of them
        u64 kept_mass = total_mass;
        // border, equals, ties from the bin where it falls: `least` elements from the row's first (or weight); returns the weight
        // of all that is kept
        auto refine = [&](const Found &g, bool counts, u64 least, uint32_t &listed) -> u64 {
            if (g.in <= INNER) {
                gather(g.bin, g.bin, sh.inner, listed, INNER);
                u64 got[4] = {};
                if (rank == 0) {
                    const int m = (int)g.in;
                    sort_list(sh.inner, m);
                    u64 sums[EACH];
                    bool is[EACH];
                    if (by_p) list_sums(sh.inner, m, by_key, sums);
                    else
                        for (int j = 0; j < EACH; ++j) sums[j] = 0;
                    int at = (int)(least - g.count) - 1;
                    if (!counts) {
#pragma unroll
                        for (int j = 0; j < EACH; ++j)
                            is[j] = (int)threadIdx.x * EACH + j < m && g.mass + sums[j] >= least;
                        at = first_where(m - 1, is);
                    }
                    const uint32_t k = ~(uint32_t)(sh.inner[at] >> 32);
                    u64 same = 0;
#pragma unroll
                    for (int j = 0; j < EACH; ++j) {
                        const int i = threadIdx.x * EACH + j;
                        is[j] = i < m && ~(uint32_t)(sh.inner[i] >> 32) == k;
                        same += is[j];
                        if (i == at) sh.found.mass = sums[j];
                    }
                    got[0] = k;
                    got[1] = (u64)(at - first_where(at, is) + 1);
                    got[2] = block_sum(sh, same);
                    got[3] = g.mass + sh.found.mass;
                }
                u64(*x)[4] = exchange(got[0], got[1], got[2], got[3]);
                border = (uint32_t)x[0][0], equals = x[0][1], ties = x[0][2];
                return x[0][3];
            }
            auto inside = [&](float l) { return in_min(l) && Scale::bin(sc.place(l)) == g.bin; };
            // count and sum of the bin's elements from key k on
            auto since = [&](uint32_t k, u64 &c, u64 &m) {
                uint32_t nc = 0, nc_all;
                u64 nm = 0, nm_all;
                each4([&](int, const float(&l)[4]) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (inside(l[j]) && key_of(l[j]) >= k) ++nc, nm += sc.weight(sh.table, l[j]);
                });
                block_scan(sh, nc, nm, nc_all, nm_all);
                u64(*x)[4] = exchange(nc_all, nm_all, 0, 0);
                c = g.count, m = g.mass;
                for (int r = 0; r < parts; ++r) c += x[r][0], m += x[r][1];
            };
            uint32_t lo = UINT32_MAX, hi = 0;
            for (int i = from; i < to; ++i)
                if (inside(data[i])) lo = min(lo, key_of(data[i])), hi = max(hi, key_of(data[i]));
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
        if (cut_k) kept_mass = refine(f, true, (u64)top_k, sh.listed[1]);
        if (by_p) {
            const u64 want = share_up(top_p, kept_mass);
            const uint32_t k_border = border;
            const u64 k_equals = equals, k_ties = ties;
            const Found g = cut_k ? find(false, want) : f;
            if (g.bin >= 0 && !(cut_k && g.bin > f.bin)) {
                refine(g, false, want, sh.listed[2]);
                if (cut_k && border < k_border) border = k_border, equals = k_equals, ties = k_ties;
                else if (cut_k && border == k_border) equals = min(equals, k_equals);
            }
        }
        if (equals < ties) {  // the index of the last equal that is kept
            u64 mine = 0, all;
            for (int i = from; i < to; ++i) mine += key_of(data[i]) == border;
            const u64 upto = block_scan(sh, mine, all);
            u64 before = 0;
            {
                u64(*x)[4] = exchange(all, 0, 0, 0);
                for (int r = 0; r < rank; ++r) before += x[r][0];
            }
            u64 c = before + upto - mine;
            __syncthreads();
            if (threadIdx.x == 0) sh.part[0] = ~0ull;
            __syncthreads();
            if (c < equals && equals <= c + mine)
                for (int i = from;; ++i)
                    if (key_of(data[i]) == border && ++c == equals) {
                        sh.part[0] = (u64)(c0 + i);
                        break;
                    }
            __syncthreads();
            u64(*x)[4] = exchange(sh.part[0], 0, 0, 0);
            for (int r = 0; r < parts; ++r)
                if (x[r][0] != ~0ull) last = (int)x[r][0];
        }
    }

    // ---- the kept weights' sums in index order, and where u falls ----
    auto kept = [&](float l, int i) {
        const uint32_t k = key_of(l);
        return k > border || (k == border && c0 + i <= last);
    };
    u64 mine = 0, all;
    each4([&](int i, const float(&l)[4]) {
        u64 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = sc.weight(sh.table, l[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (kept(l[j], i + j)) mine += w[j];
    });
    const u64 upto = block_scan(sh, mine, all);
    u64 before = 0, sum = 0;
    {
        u64(*x)[4] = exchange(all, 0, 0, 0);
        for (int r = 0; r < parts; ++r) {
            if (r < rank) before += x[r][0];
            sum += x[r][0];
        }
    }
    const u64 want = share(u, sum), c = before + upto;
    const uint32_t here = __ballot_sync(0xffffffffu, c - mine <= want && c > want);  // one thread of all
    if (!here) return;
    // its warp walks the stretch
    const int who = __ffs(here) - 1;
    u64 at = __shfl_sync(0xffffffffu, c - mine, who);
    const int first = __shfl_sync(0xffffffffu, from, who), end = __shfl_sync(0xffffffffu, to, who);
    for (int i0 = first; i0 < end; i0 += 32) {
        const int i = i0 + lane;
        const u64 w = i < end && kept(data[i], i) ? sc.weight(sh.table, data[i]) : 0;
        const u64 to_here = at + warp_scan(w, lane);
        const uint32_t past = __ballot_sync(0xffffffffu, to_here > want);
        if (past) {
            if (lane == __ffs(past) - 1) answer(c0 + i, data[i], w, sum);
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
    constexpr size_t HEAD = (sizeof(Shared) + 127) / 128 * 128 + 64;  // + room to align the pieces
    if (!attr_set[dev].load(std::memory_order_relaxed)) {
        PQE_CUDA_TRY(cudaFuncSetAttribute(sample_kernel<FP32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          (int)(HEAD + CHUNK_MAX * sizeof(float))));
        attr_set[dev].store(1, std::memory_order_relaxed);
    }
    // as few CTAs a row as leave room for two on an SM; more where SMs would stay idle
    constexpr int CHUNK_TWO = 20224;
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
