// Norm, rotation and append of new tokens (lora_kv_append).
//
// Per query and key head h (d elements, fp32 arithmetic, one rounding on store):
//   h <- h / sqrt(mean(h^2) + eps) * norm,  then (a, b) <- (a c - b s, a s + b c)
// over the pairs of the first rot elements; values are copied.  The bytes are
// each head read once and written once: memory is the bound for large T, the
// chain of dependent loads (position -> table row; slot -> address) for small.
//
// Layout: LANES threads (the power of two >= d/8) hold one head, 8 elements each,
// so the sum of squares is a few shuffles and the partner of a half-split pair is a
// shuffle away (or, when rot/2 is no multiple of 8, in a row of shared memory).  A
// block takes the heads of one token, kHeads a thread at a time with their loads in
// flight together; its lanes keep their elements' cosines and sines for all heads.
#include "decode.cuh"

namespace lora {
namespace {

using namespace decode;

constexpr int kThreads = 256;
constexpr int kHeads = 3, kManyBlocks = 4096;

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

// The lanes of this thread's head within its warp.
template <int LANES>
__device__ __forceinline__ unsigned group_mask() {
    return LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1) << ((threadIdx.x & 31) / LANES * LANES);
}

// Eight elements as loaded, and as floats.
template <typename E>
struct Held {
    uint4 v[sizeof(E) / 2];
    __device__ __forceinline__ void load(const E *p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(E) / 2; ++i) v[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    __device__ __forceinline__ void get(float (&f)[8]) const { load8(reinterpret_cast<const E *>(v), f); }
};

// PAIRS: how elements pair up.  kNear: neighbours; kFar: i and i + rot/2 with rot/2 a
// multiple of 8; both with an aligned table (kNear: rot a multiple of 8).  kAnyNear, kAnyFar:
// without those conditions.  HEADS: heads a thread.
enum { kNear, kFar, kAnyNear, kAnyFar };

template <typename E, int LANES, int PAIRS, int HEADS>
__global__ void __launch_bounds__(kThreads, 5) append_kernel(const AppendParams p) {
    constexpr int kGroups = kThreads / LANES;
    constexpr bool kFarPairs = PAIRS == kFar || PAIRS == kAnyFar;
    __shared__ float rows[PAIRS == kAnyFar ? kThreads * 8 : 1];
    const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES, at = lane * 8;
    const int heads = p.n_q + 2 * p.n_kv, half = p.rot >> 1;
    const int head_first = blockIdx.y * kGroups * HEADS + group;
    const long long t = blockIdx.x;
    const bool inside = at < p.d;

    Held<E> held[HEADS];
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
        const int head = head_first + u * kGroups;
        const E *src = head < p.n_q ? static_cast<const E *>(p.q) + t * p.ld_q + head * p.d
                       : head < p.n_q + p.n_kv ? static_cast<const E *>(p.k) + t * p.ld_k + (head - p.n_q) * p.d
                                               : static_cast<const E *>(p.v) + t * p.ld_v + (head - p.n_q - p.n_kv) * p.d;
        if (head < heads && inside) held[u].load(src + at);
    }
    const long long slot = p.slots[t];
    float c[kFarPairs ? 8 : 4], s[kFarPairs ? 8 : 4];
    if (half) {
        int pos = p.positions[t];
        if (pos < 0 || pos >= p.n_pos) {
            if (threadIdx.x == 0) flag_status(p.status, LORA_DEV_BAD_POSITION);
            pos = pos < 0 ? 0 : p.n_pos - 1;
        }
        const float *row = p.cos_sin + (long long)pos * p.rot;
        if (PAIRS == kFar) {
            if (at < p.rot) {
                const int i = at < half ? at : at - half;
                load8(row + i, c);
                load8(row + half + i, s);
            }
        } else if (PAIRS == kNear) {
            if (at < p.rot) {
                *reinterpret_cast<float4 *>(c) = *reinterpret_cast<const float4 *>(row + (at >> 1));
                *reinterpret_cast<float4 *>(s) = *reinterpret_cast<const float4 *>(row + half + (at >> 1));
            }
        } else {
#pragma unroll
            for (int e = 0; e < (kFarPairs ? 8 : 4); ++e) {
                const int x = kFarPairs ? at + e : at + 2 * e, i = !kFarPairs ? x >> 1 : x < half ? x : x - half;
                if (x < p.rot) {
                    c[e] = row[i];
                    s[e] = row[half + i];
                }
            }
        }
    }
    const long long page = slot >> p.page_shift, off = slot & ((1 << p.page_shift) - 1);
    const bool stored = slot >= 0 && slot < p.n_slots;
    if (slot >= p.n_slots && threadIdx.x == 0) flag_status(p.status, LORA_DEV_BAD_SLOT);

#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
        const int head = head_first + u * kGroups;
        if (head >= heads) return;
        const bool is_q = head < p.n_q, is_v = head >= p.n_q + p.n_kv;
        float h[8] = {};
        if (inside) held[u].get(h);
        const E *norm = static_cast<const E *>(is_q ? p.q_norm : p.k_norm);
        if (!is_v && norm) {
            float sum = 0.f, w[8] = {};
            if (inside) load8(norm + at, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += h[e] * h[e];
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(group_mask<LANES>(), sum, o);
            const float r = rsqrtf(sum / (float)p.d + p.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = h[e] * r * w[e];
        }
        if (!is_v && half) {
            if (!kFarPairs) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (at + 2 * e < p.rot) {
                        const float a = h[2 * e], b = h[2 * e + 1];
                        h[2 * e] = a * c[e] - b * s[e];
                        h[2 * e + 1] = a * s[e] + b * c[e];
                    }
            } else {
                float other[8];
                if (PAIRS == kFar) {
                    const int partner = (at < half ? lane + half / 8 : lane - half / 8) & (LANES - 1);
#pragma unroll
                    for (int e = 0; e < 8; ++e) other[e] = __shfl_sync(group_mask<LANES>(), h[e], partner, LANES);
                } else {
                    float *mine = rows + group * (LANES * 8);
#pragma unroll
                    for (int e = 0; e < 8; ++e) mine[at + e] = h[e];
                    __syncwarp(group_mask<LANES>());
#pragma unroll
                    for (int e = 0; e < 8; ++e) other[e] = at + e < p.rot ? mine[at + e < half ? at + e + half : at + e - half] : 0.f;
                    __syncwarp(group_mask<LANES>());
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (at + e < p.rot) h[e] = at + e < half ? h[e] * c[e] - other[e] * s[e] : other[e] * s[e] + h[e] * c[e];
            }
        }
        if (!inside) continue;
        if (is_q) {
            store8(static_cast<E *>(p.q_out) + (t * p.n_q + head) * p.d + at, h);
        } else if (stored) {
            E *dst = static_cast<E *>(is_v ? p.v_pages : p.k_pages);
            const int kv_head = head - p.n_q - (is_v ? p.n_kv : 0);
            store8(dst + (((page * p.n_kv + kv_head) << p.page_shift) + off) * p.d + at, h);
        }
    }
}

template <typename E, int LANES, int PAIRS>
void launch(const AppendParams &p, int T, cudaStream_t st) {
    constexpr int kGroups = kThreads / LANES;
    const int heads = p.n_q + 2 * p.n_kv;
    const dim3 one(T, (heads + kGroups - 1) / kGroups), more(T, (heads + kGroups * kHeads - 1) / (kGroups * kHeads));
    if ((long long)one.x * one.y > kManyBlocks) append_kernel<E, LANES, PAIRS, kHeads><<<more, kThreads, 0, st>>>(p);
    else append_kernel<E, LANES, PAIRS, 1><<<one, kThreads, 0, st>>>(p);
}

template <typename E, int LANES>
void launch(const AppendParams &p, int T, bool interleaved, cudaStream_t st) {
    const bool table = aligned16(p.cos_sin);
    if (interleaved) {
        if (table && p.rot % 8 == 0) launch<E, LANES, kNear>(p, T, st);
        else launch<E, LANES, kAnyNear>(p, T, st);
    } else {
        if (table && p.rot % 16 == 0) launch<E, LANES, kFar>(p, T, st);
        else launch<E, LANES, kAnyFar>(p, T, st);
    }
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
