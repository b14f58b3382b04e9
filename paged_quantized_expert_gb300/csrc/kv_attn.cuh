// kv_attn.cuh -- what the attention kernels over the 4-bit paged cache share (internal).
#pragma once

#include "kv_layout.cuh"

namespace pqe {
namespace kv {

constexpr int TILE = 64;  // tokens that the split kernel takes of the cache at a time
// Tokens that a block table may describe: the kernels count them in 32 bits, in steps of up to 2^13 tokens that may begin
// before the last one and end behind it.
constexpr int64_t MAX_TOKENS = (1ll << 31) - (1 << 16);

struct AttnArgs {
    Cache c;
    const uint16_t *q;
    int64_t q_stride;
    const int32_t *q_offsets, *kv_lens, *block_table;
    int max_pages, B, total_q, n_q, causal, window;
    float scale;  // times log2(e): scores are kept as exponents of two
    uint16_t *out;
    float *lse;
    int32_t *status;
    uint32_t wait_limit;
    int rows_min, rows_max;  // sequences with that many query rows (m * group) are this kernel's; the others are skipped
};

__device__ __forceinline__ bool is_ours(const AttnArgs &a, int m) {
    const int64_t rows = (int64_t)m * (a.n_q / a.c.n_kv);
    return rows >= a.rows_min && rows <= a.rows_max;
}

// sequence b's first query row, query tokens and cached tokens, held to what
// the arguments describe
__device__ __forceinline__ void sequence_of(const AttnArgs &a, int b, int &first, int &m, int &len) {
    first = min(max(a.q_offsets[b], 0), a.total_q);
    m = max(min(a.q_offsets[b + 1], a.total_q) - first, 0);
    len = min(max(a.kv_lens[b], 0), a.max_pages << a.c.page_shift);
}

// tokens [lo, hi) that query i of m sees (pos is below zero where there are more queries than tokens, and the window may be as
// wide as an int: their difference is not taken there. Comparing them instead took the prompt kernel five spilled words more:
// 204.5 us against 199 for two chunks of 2048)
__device__ __forceinline__ void visible(const AttnArgs &a, int i, int m, int len, int &lo, int &hi) {
    const int pos = len - m + i;
    hi = a.causal ? min(pos + 1, len) : len;
    lo = a.window > 0 ? max(max(pos, 0) - a.window + 1, 0) : 0;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The power of two that brings a row's largest |q| (amax, bf16 bits without
// sign, finite) to [2^8, 2^9), as fp32, and its inverse. f16 then holds every
// bf16 value of the row down to 2^-22 of the largest exactly.
__device__ __forceinline__ void q_factor(uint32_t amax, float &f, float &inv) {
    const int k = min(135 - (int)(amax >> 7), 126);
    f = amax == 0 ? 1.f : __uint_as_float((uint32_t)(127 + k) << 23);
    inv = amax == 0 ? 1.f : __uint_as_float((uint32_t)(127 - k) << 23);
}

// 2^(r - 142) for an E8M0 byte r in [0, 254]: a V tile's common factor 2^(r - 127) without
// the 2^15 that its products carry
__device__ __forceinline__ float v_factor(uint32_t r) {
    return __uint_as_float(r > 15 ? (r - 15) << 23 : 1u << (r + 7));
}

int attn_split(const pqe_kv_cache *cache, const AttnArgs &a, int max_q, int sms, void *ws, cudaStream_t s);
int attn_prompt(const pqe_kv_cache *cache, const AttnArgs &a, int splits, void *ws, cudaStream_t s);
size_t attn_prompt_ws(int B, int total_q, int n_q, int n_kv, int d, int sms);
int prompt_splits(int B, int total_q, int n_q, int n_kv, int64_t tokens, int sms);
size_t attn_split_ws(int B, int max_q, int group, int d);

}  // namespace kv
}  // namespace pqe
