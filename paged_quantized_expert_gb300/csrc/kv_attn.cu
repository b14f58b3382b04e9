// kv_attn.cu -- kv_paged_attention: argument checks and the choice of kernel.
#include <math.h>

#include <atomic>

#include "kv_attn.cuh"

namespace pqe {
namespace kv {

static std::atomic<int> g_kernel{0};  // pqe_test_set_attention_kernel
static std::atomic<int> g_polls{-1};  // pqe_test_set_attention_polls

// Which kernels a call takes: the split kernel, the prompt kernel, or both, where max_q speaks of prompts but the mean does
// not, as when a step carries single tokens beside a prompt's chunk. A sequence with more than `few_rows` query rows of a
// KV head (m * group) is the prompt kernel's.
struct Choice {
    bool few, many;
    int few_rows, few_q;  // the split kernel's bounds on rows and on m
    int splits;           // the prompt kernel's parts of a tile pair
};
constexpr int MIXED_ROWS = 64;
static int mixed_q(int64_t group) { return (int)(MIXED_ROWS / group > 0 ? MIXED_ROWS / group : 1); }

// Estimates in us, for sequences as long as the block table describes, from the measurements below. The split kernel: 10,
// and 1/400 for each 16 rows and 64 tokens of a (sequence, head), which it spreads over all SMs (heads of 64: 1/550). The
// prompt kernel: 11, 9 more where its tile pairs are cut into parts, and 1.9 for each of an SM's steps of 128 tokens (1.5
// where a sequence has one tile of 128 rows); a prompt's own tokens see half of each other.
// (m queries over L tokens of B sequences; split kernel, prompt kernel: 1 x 8192, 4 heads of 128, 128 rows: 22, 27; 256
// rows: 30, 32; 512: 48, 36. 8 x 2000, 4 of 128, 64 rows: 22, 26; 128: 33, 27. 64 x 4000, 4 of 128, 32 rows: 92, 138; 64:
// 167, 140. 32 x 4000, 8 of 64, 32 rows: 60, 96; 64: 111, 97. 1 x 1000, 4 of 128, 256 rows: 15, 26; 2048: 39, 25.)
static Choice choose(int B, int total_q, int max_q, int n_q, int n_kv, int d, int64_t tokens, int sms) {
    const int64_t group = n_q / n_kv, rows = (int64_t)max_q * group, pairs = (int64_t)B * n_kv;
    const int kind = g_kernel.load(std::memory_order_relaxed);
    const int splits = prompt_splits(B, total_q, n_q, n_kv, tokens, sms);
    if (kind == 2) return {false, true, 0, 0, splits};
    if (kind == 1 || rows <= 16) return {true, false, INT32_MAX, max_q, 1};
    const double t_split = 10 + (double)pairs * ((rows + 15) / 16) * ((double)tokens / 64) / (d == 128 ? 400 : 550);
    const int64_t per_sm = (pairs * ((rows + 255) / 256) * splits + sms - 1) / sms;
    const double seen = 1 - 0.5 * (max_q < tokens ? (double)max_q / tokens : 1);
    const double t_prompt = 11 + (splits > 1 ? 9 : 0) + (double)per_sm * tokens / 128 / splits * seen * (rows > 128 ? 1.9 : 1.5);
    if (t_split <= t_prompt) return {true, false, INT32_MAX, max_q, 1};
    return {(int64_t)total_q * 4 < (int64_t)B * max_q, true, MIXED_ROWS, mixed_q(group), splits};
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

int pqe_test_set_attention_polls(int polls) {
    PQE_CHECK_ARG(polls >= -1);
    kv::g_polls.store(polls, std::memory_order_relaxed);
    return PQE_OK;
}

size_t kv_paged_attention_workspace_size(int B, int total_q, int max_q, int n_q, int n_kv, int d) {
    if (B < 0 || total_q < 0 || max_q < 0 || n_kv < 1 || n_q < n_kv || n_q > 1024 || n_q % n_kv || (d != 64 && d != 128))
        return 0;
    int dev = 0, sms = 0;
    if (device_info(dev, sms) != PQE_OK) sms = 152;
    // whatever the call chooses; where it takes both kernels, one runs after the other
    const int64_t group = n_q / n_kv;
    size_t n = kv::attn_split_ws(B, max_q, (int)group, d);
    if (max_q * group > 16 || kv::g_kernel.load(std::memory_order_relaxed) == 2) {
        const size_t mixed = kv::attn_split_ws(B, kv::mixed_q(group), (int)group, d);
        const size_t many = kv::attn_prompt_ws(B, total_q, n_q, n_kv, d, sms);
        n = n > mixed ? n : mixed;
        n = n > many ? n : many;
    }
    return n;
}

int kv_paged_attention(const pqe_kv_cache *cache, const void *q, int64_t q_stride, const int32_t *q_offsets,
                       const int32_t *kv_lens, const int32_t *block_table, int max_pages, int B, int total_q,
                       int max_q, int n_q, float scale, int causal, int window, void *out, float *lse, void *ws,
                       size_t ws_bytes, int32_t *status, void *stream) {
    PQE_CHECK_ARG(kv::cache_ok(cache) && B >= 0 && total_q >= 0 && max_q >= 0 && window >= 0 && max_pages >= 1);
    PQE_CHECK_ARG(n_q >= cache->n_kv && n_q <= 1024 && n_q % cache->n_kv == 0 && isfinite(scale));
    PQE_CHECK_ARG((int64_t)total_q * n_q <= INT32_MAX);
    PQE_CHECK_ARG((causal || window == 0) && (int64_t)max_pages * cache->page_size <= kv::MAX_TOKENS);
    if (B == 0 || total_q == 0) return PQE_OK;
    PQE_CHECK_ARG(q && q_offsets && kv_lens && block_table && out && ws && status && max_q >= 1);
    PQE_CHECK_ARG(aligned(q, 16) && aligned(out, 16) && aligned(ws, 256) && aligned(lse, 4));
    PQE_CHECK_ARG(q_stride >= (int64_t)n_q * cache->d && q_stride % 8 == 0);
    PQE_CHECK_ARG(ws_bytes >= kv_paged_attention_workspace_size(B, total_q, max_q, n_q, cache->n_kv, cache->d));
    int dev = 0, sms = 0;
    const int rc = device_info(dev, sms);
    if (rc != PQE_OK) return rc;
    const kv::Choice use =
        kv::choose(B, total_q, max_q, n_q, cache->n_kv, cache->d, (int64_t)max_pages * cache->page_size, sms);
    const int polls = kv::g_polls.load(std::memory_order_relaxed);
    kv::AttnArgs a{kv::cache_of(cache), static_cast<const uint16_t *>(q), q_stride, q_offsets, kv_lens, block_table, max_pages,
                   B, total_q, n_q, causal, window, scale * 1.44269504088896341f, static_cast<uint16_t *>(out), lse, status,
                   polls < 0 ? wait_limit() : (uint32_t)polls, 1, INT32_MAX};
    if (use.many) {
        if (use.few) a.rows_min = use.few_rows + 1;
        const int rc2 = kv::attn_prompt(cache, a, use.splits, ws, as_stream(stream));
        if (rc2 != PQE_OK || !use.few) return rc2;
        a.rows_min = 1;
        a.rows_max = use.few_rows;
    }
    return kv::attn_split(cache, a, use.few_q, sms, ws, as_stream(stream));
}

}  // extern "C"
