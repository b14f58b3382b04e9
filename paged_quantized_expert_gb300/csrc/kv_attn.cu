// kv_attn.cu -- kv_paged_attention: argument checks and the choice of kernel.
#include <math.h>

#include "kv_attn.cuh"

namespace pqe {
namespace kv {

// The split kernel takes 16 rows of a KV head at a time and reads the cache again for the next 16; the prompt kernel
// takes 256 whatever their number. Sides measured below.
static bool many_rows(int max_q, int group) { return (int64_t)max_q * group > 64; }

}  // namespace kv
}  // namespace pqe

using namespace pqe;

extern "C" {

size_t kv_paged_attention_workspace_size(int B, int total_q, int max_q, int n_q, int n_kv, int d) {
    if (B < 0 || total_q < 0 || max_q < 0 || n_kv < 1 || n_q < n_kv || n_q > 1024 || n_q % n_kv || (d != 64 && d != 128))
        return 0;
    return kv::attn_split_ws(B, max_q, n_q / n_kv, d);
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
    const kv::AttnArgs a{kv::cache_of(cache), static_cast<const uint16_t *>(q), q_stride, q_offsets, kv_lens,
                         block_table, max_pages, B, total_q, n_q, causal, window, scale * 1.44269504088896341f,
                         static_cast<uint16_t *>(out), lse, status, wait_limit()};
    if (kv::many_rows(max_q, n_q / cache->n_kv)) return kv::attn_prompt(cache, a, as_stream(stream));
    return kv::attn_split(cache, a, max_q, sms, ws, as_stream(stream));
}

}  // extern "C"
