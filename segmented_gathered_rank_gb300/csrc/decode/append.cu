// Norm, rotation and append of new tokens (lora_kv_append).
//
// Per query and key head h (d elements, fp32 arithmetic, one rounding on store):
//   h <- h / sqrt(mean(h^2) + eps) * norm,  then (a, b) <- (a c - b s, a s + b c)
// over the pairs of the first rot elements; values are copied.  The bytes are
// each head read once and written once: memory is the bound for large T, the
// chain of dependent loads (position -> table row; slot -> address) for small.
//
// Layout: `lanes` threads (the power of two >= d/8) hold one head, 8 elements
// each, so the sum of squares is a few shuffles and the partner of a
// half-split pair is a shuffle away (or, when rot/2 is no multiple of 8, in a
// row of shared memory).
#include "decode.cuh"

namespace lora {
namespace {

using namespace decode;

constexpr int kThreads = 256;

struct AppendParams {
    const void *q, *k, *v;
    long long ld_q, ld_k, ld_v;
    int n_q, n_kv, d, page_shift;
    const int *positions;
    const long long *slots;
    const float *cos_sin;
    int n_pos, rot;
    const void *q_norm, *k_norm;
    float eps;
    void *q_out, *k_pages, *v_pages;
    long long n_slots;
    int *status;
};

// One block: `heads_per_block` consecutive heads (queries, keys, values in that
// order) of token blockIdx.x; LANES threads a head.
template <typename E, int LANES, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
    __shared__ float row[kThreads * 8];
    const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    const int head = blockIdx.y * (kThreads / LANES) + group;
    const int heads = p.n_q + 2 * p.n_kv;
    const long long t = blockIdx.x;
    const int at = lane * 8;
    const bool live = head < heads && at < p.d;
    const bool is_q = head < p.n_q, is_k = !is_q && head < p.n_q + p.n_kv;

    float x[8] = {};
    if (live) {
        const E *src = is_q   ? static_cast<const E *>(p.q) + t * p.ld_q + (long long)head * p.d
                       : is_k ? static_cast<const E *>(p.k) + t * p.ld_k + (long long)(head - p.n_q) * p.d
                              : static_cast<const E *>(p.v) + t * p.ld_v + (long long)(head - p.n_q - p.n_kv) * p.d;
        load8(src + at, x);
    }
    const E *norm = static_cast<const E *>(is_q ? p.q_norm : is_k ? p.k_norm : nullptr);
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += x[e] * x[e];
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (norm && live) {
        float w[8];
        load8(norm + at, w);
        const float r = rsqrtf(sum / (float)p.d + p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * r * w[e];
    }
    const int half = p.rot >> 1;
    if (half) {
        int pos = p.positions[t];
        if (pos < 0 || pos >= p.n_pos) {
            if (threadIdx.x == 0) flag_status(p.status, LORA_DEV_BAD_POSITION);
            pos = pos < 0 ? 0 : p.n_pos - 1;
        }
        const float *c = p.cos_sin + (long long)pos * p.rot, *s = c + half;
        const bool turn = live && (is_q || is_k);
        if (INTERLEAVED) {
#pragma unroll
            for (int e = 0; e < 8; e += 2)
                if (turn && at + e < p.rot) {
                    const int i = (at + e) >> 1;
                    const float a = x[e], b = x[e + 1];
                    x[e] = a * c[i] - b * s[i];
                    x[e + 1] = a * s[i] + b * c[i];
                }
        } else {
            float *mine = row + group * (LANES * 8);
#pragma unroll
            for (int e = 0; e < 8; ++e) mine[at + e] = x[e];
            __syncwarp();
            if (turn) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = at + e;
                    if (i < half) x[e] = x[e] * c[i] - mine[i + half] * s[i];
                    else if (i < p.rot) x[e] = mine[i - half] * s[i - half] + x[e] * c[i - half];
                }
            }
        }
    }
    if (!live) return;
    if (is_q) {
        store8(static_cast<E *>(p.q_out) + (t * p.n_q + head) * p.d + at, x);
        return;
    }
    const long long slot = p.slots[t];
    if (slot < 0) return;
    if (slot >= p.n_slots) {
        flag_status(p.status, LORA_DEV_BAD_SLOT);
        return;
    }
    const int kv_head = head - p.n_q - (is_k ? 0 : p.n_kv);
    const long long page = slot >> p.page_shift, off = slot & ((1 << p.page_shift) - 1);
    E *dst = static_cast<E *>(is_k ? p.k_pages : p.v_pages);
    store8(dst + (((page * p.n_kv + kv_head) << p.page_shift) + off) * p.d + at, x);
}

template <typename E, int LANES>
void launch(const AppendParams &p, int T, bool interleaved, cudaStream_t st) {
    const int per = kThreads / LANES, heads = p.n_q + 2 * p.n_kv;
    const dim3 grid(T, (heads + per - 1) / per);
    if (interleaved) append_kernel<E, LANES, true><<<grid, kThreads, 0, st>>>(p);
    else append_kernel<E, LANES, false><<<grid, kThreads, 0, st>>>(p);
}

template <typename E>
void launch(const AppendParams &p, int T, bool interleaved, cudaStream_t st) {
    if (p.d <= 64) launch<E, 8>(p, T, interleaved, st);
    else if (p.d <= 128) launch<E, 16>(p, T, interleaved, st);
    else launch<E, 32>(p, T, interleaved, st);
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" int lora_kv_append(const lora_kv_pages *kv, const void *q, int ld_q, const void *k, int ld_k, const void *v,
                              int ld_v, int T, int n_q_heads, const int *positions, const long long *slots,
                              const float *cos_sin, int n_pos, int rot_dim, int interleaved, const void *q_norm,
                              const void *k_norm, float eps, void *q_out, lora_stream stream) {
    int rc = decode::check_kv(kv, n_q_heads);
    if (rc) return rc;
    if (T < 0 || rot_dim < 0 || !(eps >= 0.f)) return LORA_ERR_ARG;
    const int d = kv->head_dim, vec = kv->dtype == LORA_BF16 ? 8 : 4;   // elements of 16 bytes
    if (rot_dim > d || rot_dim % 2) return LORA_ERR_SHAPE;
    if ((long long)n_q_heads + 2LL * kv->n_kv_heads > 65535) return LORA_ERR_SHAPE;
    if (ld_k < kv->n_kv_heads * d || ld_v < kv->n_kv_heads * d || ld_k % vec || ld_v % vec) return LORA_ERR_SHAPE;
    if (n_q_heads && (ld_q < n_q_heads * d || ld_q % vec)) return LORA_ERR_SHAPE;
    if (T == 0) return LORA_OK;
    if (!k || !v || !slots || !aligned16(k) || !aligned16(v) || ((uintptr_t)slots & 7u)) return LORA_ERR_ARG;
    if (n_q_heads && (!q || !q_out || !aligned16(q) || !aligned16(q_out))) return LORA_ERR_ARG;
    if (q_out && q_out == q && ld_q != n_q_heads * d && T > 1) return LORA_ERR_ARG;
    if (rot_dim && (!cos_sin || !positions || n_pos < 1 || ((uintptr_t)cos_sin & 3u) || ((uintptr_t)positions & 3u)))
        return LORA_ERR_ARG;
    if (!aligned16(q_norm) || !aligned16(k_norm)) return LORA_ERR_ARG;
    AppendParams p;
    p.q = q;
    p.k = k;
    p.v = v;
    p.ld_q = ld_q;
    p.ld_k = ld_k;
    p.ld_v = ld_v;
    p.n_q = n_q_heads;
    p.n_kv = kv->n_kv_heads;
    p.d = d;
    p.page_shift = decode::log2_of(kv->page_size);
    p.positions = positions;
    p.slots = slots;
    p.cos_sin = cos_sin;
    p.n_pos = n_pos;
    p.rot = rot_dim;
    p.q_norm = q_norm;
    p.k_norm = k_norm;
    p.eps = eps;
    p.q_out = q_out;
    p.k_pages = kv->k;
    p.v_pages = kv->v;
    p.n_slots = (long long)kv->n_pages * kv->page_size;
    p.status = kv->status;
    if (kv->dtype == LORA_BF16) launch<__nv_bfloat16>(p, T, interleaved != 0, (cudaStream_t)stream);
    else launch<float>(p, T, interleaved != 0, (cudaStream_t)stream);
    count_launch();
    return cuda_status(cudaGetLastError());
}
