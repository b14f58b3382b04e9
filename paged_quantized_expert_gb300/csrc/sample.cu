// sample.cu -- sample_tokens: the next token of each row of logits.
//
// What is kept of a row is a beginning of its order (logits descending, lower
// index first): all above a border value, and of the border's own equals the
// first few. The border is found by bisection on the logits' bits, with counts for
// top_k and sums of weights for top_p; then the kept weights are summed in index
// order until u is passed. The simplest form: a CTA a row, every step a pass over
// the row, weights in fp64.
#include <math.h>

#include "pqe_common.cuh"

namespace pqe {
namespace sampling {

struct Args {
    const void *logits;
    int64_t stride;
    int V, fp32;
    const float *temperature, *top_p, *min_p, *u;
    const int32_t *top_k;
    int32_t *tokens, *status;
    float *logprobs;
};

// Whole numbers that order as the values do (-0 as +0); -infinity gives 0x007FFFFF, NaN 0 or above +infinity's.
__device__ __forceinline__ uint32_t key_of(float l) {
    const uint32_t b = __float_as_uint(l + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t KEY_NEG_INF = 0x007FFFFFu, KEY_INF = 0xFF800000u;

constexpr int THREADS = 512;
constexpr double ONE = 8796093022208.0;  // 2^43: the weight of the largest logit

__global__ void __launch_bounds__(THREADS) sample_kernel(const Args a) {
    __shared__ unsigned long long part[THREADS / 32];
    const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_acquire();
    auto logit = [&](int i) {
        return a.fp32 ? static_cast<const float *>(a.logits)[row * a.stride + i]
                      : bf16_to_f32(static_cast<const uint16_t *>(a.logits)[row * a.stride + i]);
    };
    // sum over the CTA of what each thread holds
    auto total = [&](unsigned long long v) {
        for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        __syncthreads();
        if (lane == 0) part[warp] = v;
        __syncthreads();
        v = 0;
        for (int i = 0; i < THREADS / 32; ++i) v += part[i];
        return v;
    };
    auto sum = [&](auto f) {
        unsigned long long v = 0;
        for (int i = threadIdx.x; i < a.V; i += THREADS) v += f(key_of(logit(i)), i);
        return total(v);
    };
    // the largest key with f(keys from it on) true; f falls as the key rises
    auto border = [&](auto f) {
        uint32_t lo = 0;
        for (int bit = 31; bit >= 0; --bit)
            if (f(lo | 1u << bit)) lo |= 1u << bit;
        return lo;
    };
    const float t = a.temperature ? a.temperature[row] : 1.f, p = a.top_p ? a.top_p[row] : 1.f;
    const float mp = a.min_p ? a.min_p[row] : 0.f, u = a.u[row];
    const int k = a.top_k ? a.top_k[row] : 0;
    const uint32_t top = border([&](uint32_t x) { return sum([&](uint32_t y, int) { return y >= x; }) > 0; });
    const bool nan = sum([](uint32_t y, int) { return y < KEY_NEG_INF; }) > 0;
    if (nan || top >= KEY_INF || top <= KEY_NEG_INF || !(t >= 0.f) || isinf(t) || isnan(p) || isnan(mp) || !(u >= 0.f && u < 1.f)) {
        if (threadIdx.x == 0) {
            a.tokens[row] = -1;
            if (a.logprobs) a.logprobs[row] = __uint_as_float(0x7FC00000u);
            atomicOr(a.status, PQE_STATUS_NO_TOKEN);
        }
        return;
    }
    const double m = value_of(top);
    auto weight = [&](uint32_t y) { return (unsigned long long)(ONE * exp(((double)value_of(y) - m) / (double)t) + 0.5); };
    // the border: at least this key, and of its equals those up to an index
    uint32_t least = KEY_NEG_INF + 1;
    if (mp > 0.f) {
        const double z = m + (double)t * log((double)mp);
        const uint32_t y = key_of(__double2float_ru(z));
        least = max(least, mp >= 1.f ? top : y);
    }
    auto above = [&](uint32_t x) { return sum([&](uint32_t y, int) { return y >= x; }); };
    unsigned long long equals = 0xFFFFFFFFull;  // of the border's own equals: this many
    if (t == 0.f) least = top, equals = 1;
    else if (k > 0 && above(least) > (unsigned)k) {
        least = border([&](uint32_t x) { return above(x) >= (unsigned)k; });
        equals = k - above(least + 1);
    }
    if (t > 0.f && p < 1.f) {
        auto mass = [&](uint32_t x) { return sum([&](uint32_t y, int) { return y >= x ? weight(y) : 0ull; }); };
        const unsigned long long w = weight(least), over = mass(least + 1);
        const unsigned long long eq = min(equals, above(least) - above(least + 1));
        const double want = (double)p * ((double)over + (double)eq * (double)w);
        if (over > 0 && ((double)over >= want || w == 0)) {
            // the border is above: the largest key whose sum reaches what is wanted
            const uint32_t x = border([&](uint32_t z) { return (double)mass(z) >= want && z <= top; });
            least = max(min(x, top), least + 1);
            equals = 0xFFFFFFFFull;
        }
        const unsigned long long more = mass(least + 1), wl = weight(least);
        const double need = wl ? ceil((want - (double)more) / (double)wl) : 1.0;
        equals = min(equals, need <= 1.0 ? 1ull : (unsigned long long)need);
    }
    // the index of the last equal that is kept
    int last = a.V;
    if (equals != 0xFFFFFFFFull) {
        int lo = 0, hi = a.V - 1;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (sum([&](uint32_t y, int i) { return y == least && i <= mid; }) >= equals) hi = mid;
            else lo = mid + 1;
        }
        last = lo;
    }
    auto kept = [&](uint32_t y, int i) { return y > least || (y == least && i <= last) ? (t == 0.f ? 1ull : weight(y)) : 0ull; };
    const unsigned long long all = sum(kept);
    const double target = (double)u * (double)all;
    int lo = 0, hi = a.V - 1;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if ((double)sum([&](uint32_t y, int i) { return i <= mid ? kept(y, i) : 0ull; }) > target) hi = mid;
        else lo = mid + 1;
    }
    if (threadIdx.x == 0) {
        a.tokens[row] = lo;
        if (a.logprobs)
            a.logprobs[row] = t == 0.f ? 0.f : (float)(((double)logit(lo) - m) / (double)t - log((double)all / ONE));
    }
}

}  // namespace sampling
}  // namespace pqe

using namespace pqe;

extern "C" {

int sample_tokens(const void *logits, int fp32, int64_t stride, int B, int V, const float *temperature,
                  const int32_t *top_k, const float *top_p, const float *min_p, const float *u, int32_t *tokens,
                  float *logprobs, int32_t *status, void *stream) {
    PQE_CHECK_ARG(B >= 0 && V >= 1 && V <= 393216);
    if (B == 0) return PQE_OK;
    PQE_CHECK_ARG(logits && u && tokens && status && stride >= V && aligned(logits, fp32 ? 4 : 2));
    PQE_CHECK_ARG(aligned(temperature, 4) && aligned(top_k, 4) && aligned(top_p, 4) && aligned(min_p, 4) && aligned(u, 4) &&
                  aligned(tokens, 4) && aligned(logprobs, 4) && aligned(status, 4));
    const sampling::Args a{logits, stride, V, fp32, temperature, top_p, min_p, u, top_k, tokens, status, logprobs};
    return launch_pdl(sampling::sample_kernel, dim3((unsigned)B), dim3(sampling::THREADS), 0, as_stream(stream), a);
}

}  // extern "C"
