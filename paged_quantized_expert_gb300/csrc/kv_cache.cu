// kv_cache.cu -- writing K and V rows into the 4-bit paged cache, and reading
// them back.
//
// Per block of 32 values along d: amax, X = 2^(floor(log2 amax) - 2), codes
// RNE_e2m1(v / X). X is a power of two, so v / X is exact in fp32 and the only
// rounding is the code's own. Both kernels move bytes and do next to no
// arithmetic: bound by memory once there are enough tokens, by latency below.
#include "kv_layout.cuh"

namespace pqe {
namespace kv {

struct Codes {
    uint32_t word;   // eight codes, the first in the low nibble
    uint32_t scale;  // E8M0 byte of the 32 values
};

// Eight of the 32 values of a block, the other 24 in the three neighbouring
// lanes (four lanes, aligned): their codes and the block's scale. All 32 lanes
// call it.
__device__ __forceinline__ Codes quantize8(const uint4 &raw) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    // |v| of bf16 compares as its bits do; a NaN or an infinity ends at or above 0x7F80
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = w[i] & 0x7FFF7FFFu;
        top = max(top, max(a & 0xFFFFu, a >> 16));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    Codes c{0, 255};
    if (top < 0x7F80u) {
        // floor(log2 amax) + 127 is the exponent field; subnormal values end at scale byte 0
        const int e = (int)(top >> 7) - 2;
        c.scale = (uint32_t)max(e, 0);
        const float inv = __uint_as_float((254u - c.scale) << 23);  // 2^(127 - scale): 2^-127 is never asked for
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float lo = bf16_to_f32((uint16_t)(w[i] & 0xFFFFu)), hi = bf16_to_f32((uint16_t)(w[i] >> 16));
            c.word |= (uint32_t)f32x2_to_e2m1x2(lo * inv, hi * inv) << (8 * i);
        }
    }
    return c;
}

// One thread per eight values of a token's row: 2 * n_kv * D / 8 threads a
// token, K before V.
template <int D>
__global__ void __launch_bounds__(256) kv_write_kernel(const Cache c, const uint16_t *__restrict__ k,
                                                       const uint16_t *__restrict__ v, int64_t k_stride,
                                                       int64_t v_stride, const int64_t *__restrict__ slots, int n,
                                                       int32_t *status) {
    pdl_acquire();
    const int per = 2 * c.n_kv * (D / 8);
    const int64_t total = (int64_t)n * per;  // a multiple of four: the lanes of a block of 32 act together
    for (int64_t i0 = (int64_t)blockIdx.x * 256; i0 < total; i0 += (int64_t)gridDim.x * 256) {
        const int64_t i = i0 + threadIdx.x;
        const bool in = i < total;
        const int tok = in ? (int)(i / per) : 0, r = in ? (int)(i % per) : 0;
        const bool is_v = r >= per / 2;
        const int rr = is_v ? r - per / 2 : r, h = rr / (D / 8), e = (rr % (D / 8)) * 8;
        int64_t slot = in ? slots[tok] : -1;
        if (slot >> c.page_shift >= c.n_pages) {
            if (r == 0) atomicOr(status, PQE_STATUS_BAD_PAGE);
            slot = -1;
        }
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (slot >= 0)
            raw = *reinterpret_cast<const uint4 *>((is_v ? v + tok * v_stride : k + tok * k_stride) + h * D + e);
        const Codes q = quantize8(raw);
        if (slot < 0) continue;
        const int at = (int)(slot & ((1 << c.page_shift) - 1)), t = at & 15;
        uint8_t *b = block_of<D>(c, slot >> c.page_shift, at, h);
        if (!is_v) {
            *reinterpret_cast<uint32_t *>(b + k_code<D>(t, e)) = q.word;
            if (e % 32 == 0) b[k_scale<D>(t, e / 32)] = (uint8_t)q.scale;
        } else {
            *reinterpret_cast<uint16_t *>(b + v_code<D>(t, e)) = (uint16_t)q.word;
            *reinterpret_cast<uint16_t *>(b + v_code<D>(t, e + 4)) = (uint16_t)(q.word >> 16);
            if (e % 32 == 0) b[v_scale<D>(t, e / 32)] = (uint8_t)q.scale;
        }
    }
}

// eight codes (the first in the low nibble) times 2^(scale - 127), as bf16
__device__ __forceinline__ uint4 values8(uint32_t word, uint32_t scale) {
    const float s = scale_value(scale);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = e2m1x2_to_f32x2((uint8_t)(word >> (8 * i)));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(f.y * s), "f"(f.x * s));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int D>
__global__ void __launch_bounds__(256) kv_read_kernel(const Cache c, const int64_t *__restrict__ slots, int n,
                                                      uint16_t *k, uint16_t *v, int32_t *status) {
    pdl_acquire();
    const int per = 2 * c.n_kv * (D / 8);
    const int64_t total = (int64_t)n * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int tok = (int)(i / per), r = (int)(i % per);
        const bool is_v = r >= per / 2;
        uint16_t *out = is_v ? v : k;
        const int rr = is_v ? r - per / 2 : r, h = rr / (D / 8), e = (rr % (D / 8)) * 8;
        int64_t slot = slots[tok];
        if (slot >> c.page_shift >= c.n_pages) {
            if (r == 0) atomicOr(status, PQE_STATUS_BAD_PAGE);
            slot = -1;
        }
        if (!out) continue;
        uint4 val = make_uint4(0, 0, 0, 0);
        if (slot >= 0) {
            const int at = (int)(slot & ((1 << c.page_shift) - 1)), t = at & 15;
            const uint8_t *b = block_of<D>(c, slot >> c.page_shift, at, h);
            if (!is_v)
                val = values8(*reinterpret_cast<const uint32_t *>(b + k_code<D>(t, e)), b[k_scale<D>(t, e / 32)]);
            else
                val = values8((uint32_t)*reinterpret_cast<const uint16_t *>(b + v_code<D>(t, e)) |
                                  (uint32_t)*reinterpret_cast<const uint16_t *>(b + v_code<D>(t, e + 4)) << 16,
                              b[v_scale<D>(t, e / 32)]);
        }
        *reinterpret_cast<uint4 *>(out + ((size_t)tok * c.n_kv + h) * D + e) = val;
    }
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
    int dev = 0, sms = 0;
    const int rc = device_info(dev, sms);
    if (rc != PQE_OK) return rc;
    const int64_t ctas = ((int64_t)n * 2 * row / 8 + 255) / 256, most = (int64_t)sms * 16;
    const dim3 grid((unsigned)(ctas < most ? ctas : most));
    const uint16_t *kp = static_cast<const uint16_t *>(k), *vp = static_cast<const uint16_t *>(v);
    return launch_pdl(cache->d == 128 ? kv::kv_write_kernel<128> : kv::kv_write_kernel<64>, grid, dim3(256), 0,
                      as_stream(stream), c, kp, vp, k_stride, v_stride, slots, n, status);
}

int kv_cache_read(const pqe_kv_cache *cache, const int64_t *slots, int n, void *k, void *v, int32_t *status,
                  void *stream) {
    PQE_CHECK_ARG(kv::cache_ok(cache) && n >= 0);
    if (n == 0) return PQE_OK;
    PQE_CHECK_ARG((k || v) && slots && status && aligned(k, 16) && aligned(v, 16) && aligned(slots, 8));
    const kv::Cache c = kv::cache_of(cache);
    int dev = 0, sms = 0;
    const int rc = device_info(dev, sms);
    if (rc != PQE_OK) return rc;
    const int64_t ctas = ((int64_t)n * 2 * cache->n_kv * cache->d / 8 + 255) / 256, most = (int64_t)sms * 16;
    const dim3 grid((unsigned)(ctas < most ? ctas : most));
    return launch_pdl(cache->d == 128 ? kv::kv_read_kernel<128> : kv::kv_read_kernel<64>, grid, dim3(256), 0,
                      as_stream(stream), c, slots, n, static_cast<uint16_t *>(k), static_cast<uint16_t *>(v), status);
}

}  // extern "C"
