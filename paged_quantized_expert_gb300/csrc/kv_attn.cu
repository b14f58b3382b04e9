// kv_attn.cu -- grouped-query attention over the 4-bit paged KV cache.
//
// out = sum_j softmax_j(scale q.k_j) v_j over the tokens a query sees, in one
// pass with the running maximum and sum of the softmax. One warp per (query
// token, query head): the lanes share out the head's d values.
#include "kv_layout.cuh"

#include <math.h>

namespace pqe {
namespace kv {

struct AttnArgs {
    Cache c;
    const uint16_t *q;
    int64_t q_stride;
    const int32_t *q_offsets, *kv_lens, *block_table;
    int max_pages, B, total_q, n_q, causal, window;
    float scale;
    uint16_t *out;
    float *lse;
    int32_t *status;
};

// sequence b's first query row, query tokens and cached tokens, held to what the arguments describe
__device__ __forceinline__ void sequence_of(const AttnArgs &a, int b, int &first, int &m, int &len) {
    first = min(max(a.q_offsets[b], 0), a.total_q);
    m = max(min(a.q_offsets[b + 1], a.total_q) - first, 0);
    len = min(max(a.kv_lens[b], 0), a.max_pages << a.c.page_shift);
}

template <int D>
__global__ void __launch_bounds__(256) attn_rows_kernel(const AttnArgs a) {
    constexpr int E = D / 32;  // values of a lane
    pdl_acquire();
    const int lane = threadIdx.x & 31;
    const int64_t rows = (int64_t)a.total_q * a.n_q;
    for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < rows; w += (int64_t)gridDim.x * 8) {
        const int tok = (int)(w / a.n_q), h = (int)(w % a.n_q);
        int b = 0, first = 0, m = 0, len = 0;
        for (; b < a.B; ++b) {
            sequence_of(a, b, first, m, len);
            if (tok >= first && tok < first + m) break;
        }
        if (b == a.B) continue;  // a row of no sequence
        if (a.kv_lens[b] > len && lane == 0) atomicOr(a.status, PQE_STATUS_BAD_PAGE);
        const int pos = len - m + (tok - first);
        const int hi = a.causal ? min(pos + 1, len) : len, lo = a.window > 0 ? max(pos - a.window + 1, 0) : 0;
        const int hk = h / (a.n_q / a.c.n_kv), e0 = lane * E;
        float q[E], acc[E];
        for (int e = 0; e < E; ++e) {
            q[e] = bf16_to_f32(a.q[tok * a.q_stride + (int64_t)h * D + e0 + e]);
            acc[e] = 0.f;
        }
        float top = -INFINITY, sum = 0.f;
        for (int j = lo; j < hi; ++j) {
            const int page = a.block_table[(size_t)b * a.max_pages + (j >> a.c.page_shift)];
            if (page < 0 || page >= a.c.n_pages) {
                if (lane == 0) atomicOr(a.status, PQE_STATUS_BAD_PAGE);
                continue;
            }
            const int at = j & ((1 << a.c.page_shift) - 1), t = at & 15;
            const uint8_t *blk = block_of<D>(a.c, page, at, hk);
            const float ks = scale_value(blk[k_scale<D>(t, e0 / 32)]), vs = scale_value(blk[v_scale<D>(t, e0 / 32)]);
            float s = 0.f, v[E];
            for (int e = 0; e < E; e += 2) {
                const float2 kf = e2m1x2_to_f32x2(blk[k_code<D>(t, e0 + e)]);
                const float2 vf = e2m1x2_to_f32x2(blk[v_code<D>(t, e0 + e)]);
                s = fmaf(q[e], kf.x * ks, fmaf(q[e + 1], kf.y * ks, s));
                v[e] = vf.x * vs;
                v[e + 1] = vf.y * vs;
            }
            s = warp_sum(s) * a.scale;
            const float now = fmaxf(top, s), keep = expf(top - now), p = expf(s - now);
            sum = fmaf(sum, keep, p);
            for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], keep, p * v[e]);
            top = now;
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        for (int e = 0; e < E; ++e) a.out[w * D + e0 + e] = f32_to_bf16_rn(acc[e] * inv);
        if (a.lse && lane == 0) a.lse[w] = sum == 0.f ? -INFINITY : top + logf(sum);
    }
}

}  // namespace kv
}  // namespace pqe

using namespace pqe;

extern "C" {

size_t kv_paged_attention_workspace_size(int B, int total_q, int max_q, int n_q, int n_kv, int d) {
    if (B < 0 || total_q < 0 || max_q < 0 || n_kv < 1 || n_q < n_kv || n_q > 1024 || n_q % n_kv || (d != 64 && d != 128))
        return 0;
    return 256;
}

int kv_paged_attention(const pqe_kv_cache *cache, const void *q, int64_t q_stride, const int32_t *q_offsets,
                       const int32_t *kv_lens, const int32_t *block_table, int max_pages, int B, int total_q,
                       int max_q, int n_q, float scale, int causal, int window, void *out, float *lse, void *ws,
                       size_t ws_bytes, int32_t *status, void *stream) {
    PQE_CHECK_ARG(kv::cache_ok(cache) && B >= 0 && total_q >= 0 && max_q >= 0 && window >= 0 && max_pages >= 1);
    PQE_CHECK_ARG(n_q >= cache->n_kv && n_q <= 1024 && n_q % cache->n_kv == 0 && isfinite(scale));
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
                         block_table, max_pages, B, total_q, n_q, causal, window, scale, static_cast<uint16_t *>(out),
                         lse, status};
    const int64_t ctas = ((int64_t)total_q * n_q + 7) / 8, most = (int64_t)sms * 8;
    return launch_pdl(cache->d == 128 ? kv::attn_rows_kernel<128> : kv::attn_rows_kernel<64>,
                      dim3((unsigned)(ctas < most ? ctas : most)), dim3(256), 0, as_stream(stream), a);
}

}  // extern "C"
