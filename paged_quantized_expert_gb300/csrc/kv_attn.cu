// kv_attn.cu -- kv_paged_attention: argument checks and the choice of kernel.
#include <math.h>

#include <atomic>

#include "kv_attn.cuh"

namespace pqe {
namespace kv {

static std::atomic<int> g_kernel{0};  // pqe_test_set_attention_kernel

// Which kernels a call takes: the split kernel, the prompt kernel, or both, where max_q speaks of prompts but the mean does
// not, as when a step carries single tokens beside a prompt's chunk. A sequence with more than `few_rows` query rows of a
// KV head (m * group) is the prompt kernel's.
struct Choice {
    bool few, many;
    int few_rows, few_q;  // the split kernel's bounds on rows and on m
};

// The split kernel's time goes with the 16-row sets of all (sequence, head), whose tiles it spreads over all SMs; the prompt
// kernel's with the CTAs of 256 rows that an SM gets, each a whole sequence long. Measured at equal lengths: a set's tile
// of 64 tokens takes 1/430 us of the chip (heads of 64: 1/630), a CTA's step of 128 tokens 1.9 us, so that the split
// kernel is faster below sets * 16 = 5700 (8400) rows for each CTA of an SM. (1 sequence of 8192 tokens, 4 heads of 128,
// 256 rows: 30 us and 130 us; 8 of 2000, 4 heads, 128 rows: 33 and 36, 192 rows: 43 and 43; 64 of 4000, 4 heads, 48 rows:
// 130 and 127, 64 rows: 167 and 127; 32 of 4000, 8 heads of 64, 48 rows: 87 and 94, 64 rows: 112 and 94.)
static Choice choose(int B, int total_q, int max_q, int n_q, int n_kv, int d, int sms) {
    const int64_t group = n_q / n_kv, rows = (int64_t)max_q * group, most = d == 128 ? 5700 : 8400;
    const int64_t pairs = (int64_t)B * n_kv, per_sm = (pairs * ((rows + 255) / 256) + sms - 1) / sms;
    const int kind = g_kernel.load(std::memory_order_relaxed);
    if (kind == 2) return {false, true, 0, 0};
    const bool many = kind == 0 && rows > 16 && pairs * rows > most * per_sm;
    const bool mixed = many && (int64_t)total_q * 4 < (int64_t)B * max_q;
    if (!many) return {true, false, INT32_MAX, max_q};
    return {mixed, true, 64, (int)(64 / group > 0 ? 64 / group : 1)};
}

}  // namespace kv
}  // namespace pqe

using namespace pqe;

extern "C" {

int pqe_test_set_attention_kernel(int kind) {
    PQE_CHECK_ARG(kind >= 0 && kind <= 2);
    kv::g_kernel.store(kind, std::memory_order_relaxed);
    return PQE_OK;
}

size_t kv_paged_attention_workspace_size(int B, int total_q, int max_q, int n_q, int n_kv, int d) {
    if (B < 0 || total_q < 0 || max_q < 0 || n_kv < 1 || n_q < n_kv || n_q > 1024 || n_q % n_kv || (d != 64 && d != 128))
        return 0;
    int dev = 0, sms = 0;
    if (device_info(dev, sms) != PQE_OK) sms = 152;
    const kv::Choice use = kv::choose(B, total_q, max_q, n_q, n_kv, d, sms);
    return use.few ? kv::attn_split_ws(B, use.few_q, n_q / n_kv, d) : 256;
}

int kv_paged_attention(const pqe_kv_cache *cache, const void *q, int64_t q_stride, const int32_t *q_offsets,
                       const int32_t *kv_lens, const int32_t *block_table, int max_pages, int B, int total_q,
                       int max_q, int n_q, float scale, int causal, int window, void *out, float *lse, void *ws,
                       size_t ws_bytes, int32_t *status, void *stream) {
    PQE_CHECK_ARG(kv::cache_ok(cache) && B >= 0 && total_q >= 0 && max_q >= 0 && window >= 0 && max_pages >= 1);
    PQE_CHECK_ARG(n_q >= cache->n_kv && n_q <= 1024 && n_q % cache->n_kv == 0 && isfinite(scale));
    PQE_CHECK_ARG((int64_t)total_q * n_q <= INT32_MAX);
    PQE_CHECK_ARG((causal || window == 0) && (int64_t)max_pages * cache->page_size <= INT32_MAX);
    if (B == 0 || total_q == 0) return PQE_OK;
    PQE_CHECK_ARG(q && q_offsets && kv_lens && block_table && out && ws && status && max_q >= 1);
    PQE_CHECK_ARG(aligned(q, 16) && aligned(out, 16) && aligned(ws, 256) && aligned(lse, 4));
    PQE_CHECK_ARG(q_stride >= (int64_t)n_q * cache->d && q_stride % 8 == 0);
    PQE_CHECK_ARG(ws_bytes >= kv_paged_attention_workspace_size(B, total_q, max_q, n_q, cache->n_kv, cache->d));
    int dev = 0, sms = 0;
    const int rc = device_info(dev, sms);
    if (rc != PQE_OK) return rc;
    const kv::Choice use = kv::choose(B, total_q, max_q, n_q, cache->n_kv, cache->d, sms);
    kv::AttnArgs a{kv::cache_of(cache), static_cast<const uint16_t *>(q), q_stride, q_offsets, kv_lens, block_table, max_pages,
                   B, total_q, n_q, causal, window, scale * 1.44269504088896341f, static_cast<uint16_t *>(out), lse, status,
                   wait_limit(), 1, INT32_MAX};
    if (use.many) {
        if (use.few) a.rows_min = use.few_rows + 1;
        const int rc2 = kv::attn_prompt(cache, a, as_stream(stream));
        if (rc2 != PQE_OK || !use.few) return rc2;
        a.rows_min = 1;
        a.rows_max = use.few_rows;
    }
    return kv::attn_split(cache, a, use.few_q, sms, ws, as_stream(stream));
}

}  // extern "C"
