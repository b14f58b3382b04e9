// kv_layout.cuh -- byte layout of the 4-bit paged KV cache (internal; the
// layout itself is stated in pqe.h, "KV cache").
#pragma once

#include "pqe_common.cuh"

namespace pqe {
namespace kv {

constexpr int BLOCK = 16;  // tokens of a block

__host__ __device__ constexpr int block_bytes(int d) { return 17 * d; }

__host__ inline bool cache_shape_ok(int page_size, int n_kv, int d) {
    return (d == 64 || d == 128) && page_size >= BLOCK && page_size <= 1024 && (page_size & (page_size - 1)) == 0 &&
           n_kv >= 1 && n_kv <= 256;
}

__host__ inline bool cache_ok(const pqe_kv_cache *c) {
    return c && c->pages && c->n_pages >= 1 && cache_shape_ok(c->page_size, c->n_kv, c->d) && aligned(c->pages, 16) &&
           c->page_stride % 16 == 0 && c->page_stride >= pqe_kv_page_bytes(c->page_size, c->n_kv, c->d);
}

// What the kernels need of a cache. 64-bit byte offsets throughout: a cache may
// hold far more than 2^32 bytes.
struct Cache {
    uint8_t *pages;
    size_t page_stride;
    int32_t n_pages, page_shift, n_kv;
};

__host__ inline Cache cache_of(const pqe_kv_cache *c) {
    int sh = 0;
    while ((1 << sh) < c->page_size) ++sh;
    return Cache{static_cast<uint8_t *>(c->pages), c->page_stride, c->n_pages, sh, c->n_kv};
}

// head h's block that holds place `at` of page `page`
template <int D>
__device__ __forceinline__ uint8_t *block_of(const Cache &c, int64_t page, int at, int h) {
    return c.pages + (size_t)page * c.page_stride +
           ((size_t)h * (size_t)(1 << (c.page_shift - 4)) + (size_t)(at >> 4)) * block_bytes(D);
}

// byte offsets inside a block, for token tok (0..15); e even
template <int D>
__device__ __forceinline__ int k_code(int tok, int e) {
    return tok * (D / 2) + ((e & 31) >> 3) * (D / 8) + (e >> 5) * 4 + ((e & 7) >> 1);
}
template <int D>
__device__ __forceinline__ int v_code(int tok, int e) {
    const int G = e >> 5;
    return 8 * D + (G >> 1) * 512 + (((e & 31) >> 2) * 4 + ((tok & 7) >> 1)) * 16 + ((tok & 1) + 2 * (tok >> 3)) * 4 +
           (G & 1) * 2 + ((e & 3) >> 1);
}
template <int D>
__device__ __forceinline__ int k_scale(int tok, int G) {
    return 16 * D + tok * (D / 32) + G;
}
template <int D>
__device__ __forceinline__ int v_scale(int tok, int G) {
    return 16 * D + D / 2 + ((tok & 7) >> 1) * (D / 8) + G * 4 + (tok & 1) + 2 * (tok >> 3);
}

// four bytes of two E2M1 codes each to four f16 pairs (a byte's low nibble in the low half)
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 "
        "%1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}

}  // namespace kv
}  // namespace pqe
