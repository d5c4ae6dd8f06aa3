// Attention of drafted tokens over a paged cache (lora_tree_attention).
//
// For drafted token i of a request with prefix P = kv_len - n:
//   o = sum_c p_c v_c / sum_c p_c,  p_c = exp(scale q . k_c - m),  m the running maximum,
// over the visible c: every c < P, and drafted j (c = P + j) that the token's
// mask row names (or j <= i without a mask).
#include "decode.cuh"

namespace lora {
namespace {

using namespace decode;

struct AttnParams {
    const void *q;
    const void *k, *v;
    int n_q, n_kv, d, page_shift, n_pages;
    const int *starts, *lens, *table;
    int S, T, max_pages;
    const long long *mask;
    int words;
    float scale;
    void *out;
    int *status;
};

// One warp per (token, query head); each lane holds 8 elements of the head.
template <typename E>
__global__ void __launch_bounds__(128) attention_rows_kernel(const AttnParams p) {
    const int lane = threadIdx.x & 31, at = lane * 8;
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (blockIdx.x == 0) check_starts(p.starts, p.S, p.T, p.status);
    if (w >= (long long)p.T * p.n_q) return;
    const int t = (int)(w / p.n_q), h = (int)(w % p.n_q);
    const int s = segment_of(p.starts, p.S, t);
    const int begin = p.starts[s], n = p.starts[s + 1] - begin, i = t - begin;
    int len = p.lens[s], bad = 0;
    if (i < 0 || i >= n) bad |= LORA_DEV_BAD_SEGMENTS;
    if (len < n || len > ((long long)p.max_pages << p.page_shift)) {
        bad |= LORA_DEV_BAD_LENGTH;
        len = len < n ? n : p.max_pages << p.page_shift;
    }
    const int prefix = max(0, len - n);
    float q[8] = {}, o[8] = {}, m = -INFINITY, l = 0.f;
    if (at < p.d) load8(static_cast<const E *>(p.q) + w * p.d + at, q);
    const int page_mask = (1 << p.page_shift) - 1, kv_head = h / (p.n_q / p.n_kv);
    for (int c = 0; c < len && !(bad & LORA_DEV_BAD_SEGMENTS); ++c) {
        const int j = c - prefix;
        if (j >= 0) {
            if (!p.mask) {
                if (j > i) break;
            } else if (j >= 64 * p.words || !((p.mask[(long long)t * p.words + (j >> 6)] >> (j & 63)) & 1)) {
                continue;
            }
        }
        int page = p.table[(long long)s * p.max_pages + (c >> p.page_shift)];
        if (page < 0 || page >= p.n_pages) {
            bad |= LORA_DEV_BAD_PAGE;
            page = 0;
        }
        const long long off = ((((long long)page * p.n_kv + kv_head) << p.page_shift) + (c & page_mask)) * p.d + at;
        float kk[8] = {}, vv[8] = {}, dot = 0.f;
        if (at < p.d) {
            load8(static_cast<const E *>(p.k) + off, kk);
            load8(static_cast<const E *>(p.v) + off, vv);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) dot += q[e] * kk[e];
        dot = warp_sum(dot) * p.scale;
        const float m2 = fmaxf(m, dot), a = __expf(m - m2), b = __expf(dot - m2);
        m = m2;
        l = l * a + b;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = o[e] * a + b * vv[e];
    }
    if (bad && lane == 0) flag_status(p.status, bad);
    const float r = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= r;
    if (at < p.d) store8(static_cast<E *>(p.out) + w * p.d + at, o);
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" size_t lora_tree_attention_workspace_size(const lora_kv_pages *kv, int n_q_heads, int S, int T) {
    if (decode::check_kv(kv, n_q_heads) || n_q_heads < 1 || S < 0 || T < 0) return 0;
    return 256;
}

extern "C" int lora_tree_attention(const lora_kv_pages *kv, const void *q, int n_q_heads, const int *seg_starts, int S,
                                   int T, const int *kv_lens, const int *page_table, int max_pages,
                                   const long long *tree_mask, int mask_words, float scale, void *out, void *workspace,
                                   size_t ws_bytes, lora_stream stream) {
    int rc = decode::check_kv(kv, n_q_heads);
    if (rc) return rc;
    if (n_q_heads < 1) return LORA_ERR_SHAPE;
    if (S < 0 || T < 0 || (S == 0 && T > 0) || max_pages < 0 || (tree_mask && mask_words < 1)) return LORA_ERR_ARG;
    if ((long long)max_pages * kv->page_size > 0x7fffffffLL) return LORA_ERR_SHAPE;
    if (T == 0) return LORA_OK;
    if (!q || !out || !seg_starts || !kv_lens || !page_table || !workspace || max_pages < 1) return LORA_ERR_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || ((uintptr_t)tree_mask & 7u) ||
        (((uintptr_t)seg_starts | (uintptr_t)kv_lens | (uintptr_t)page_table) & 3u))
        return LORA_ERR_ARG;
    if (ws_bytes < lora_tree_attention_workspace_size(kv, n_q_heads, S, T)) return LORA_ERR_ARG;
    AttnParams p;
    p.q = q;
    p.k = kv->k;
    p.v = kv->v;
    p.n_q = n_q_heads;
    p.n_kv = kv->n_kv_heads;
    p.d = kv->head_dim;
    p.page_shift = decode::log2_of(kv->page_size);
    p.n_pages = kv->n_pages;
    p.starts = seg_starts;
    p.lens = kv_lens;
    p.table = page_table;
    p.S = S;
    p.T = T;
    p.max_pages = max_pages;
    p.mask = tree_mask;
    p.words = mask_words;
    p.scale = scale;
    p.out = out;
    p.status = kv->status;
    const long long warps = (long long)T * n_q_heads;
    if (warps > 4LL * 0x7fffffff) return LORA_ERR_SHAPE;
    const unsigned grid = (unsigned)((warps + 3) / 4);
    if (kv->dtype == LORA_BF16) attention_rows_kernel<__nv_bfloat16><<<grid, 128, 0, (cudaStream_t)stream>>>(p);
    else attention_rows_kernel<float><<<grid, 128, 0, (cudaStream_t)stream>>>(p);
    count_launch();
    return cuda_status(cudaGetLastError());
}
