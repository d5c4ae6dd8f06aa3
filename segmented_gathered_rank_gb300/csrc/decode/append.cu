// Norm, rotation and append of new tokens (lora_kv_append).
//
// Per query and key head h (d elements, fp32 arithmetic, one rounding on store):
//   h <- h / sqrt(mean(h^2) + eps) * norm,  then (a, b) <- (a c - b s, a s + b c)
// over the pairs of the first rot elements; values are copied.  The bytes are
// each head read once and written once: memory is the bound for large T, the
// chain of dependent loads (position -> table row; slot -> address) for small.
// Measured, bf16, heads of 128: 1 token 2.0 us, 256 tokens of 48 heads with norms
// 3.1 us, 8192 tokens 39.8 us (5.2 TB/s).
//
// Layout: LANES threads (the power of two >= d/8) hold one head, 8 elements each in two
// quads that are each other's partners in the rotation, so a pair meets in a thread (or,
// when rot is no multiple of 8, in a row of shared memory).  A block takes heads of one
// token, several a thread for long batches; its lanes keep their pairs' cosines and
// sines for all of them.
#include "decode.cuh"

namespace lora {
namespace {

using namespace decode;

constexpr int kThreads = 256;
// Heads a thread when neighbours pair up, one block does not hold all heads of a token
// and one head a thread would make more than kManyBlocks blocks: the loads of three heads
// are in flight at once, and position, slot and table row are read once for them.  bf16,
// one head a thread against three: 48 heads of 128, 256 tokens (768 blocks) 2.7 and 2.9
// us, 512 tokens (1536) 3.9 and 3.6, 4096 tokens 26.3 and 22.5, 8192 tokens 50.6 and 40.0
// (2, 4, 6 heads were slower than 3); 20 heads of 128, 512 tokens (1024 blocks) 3.2 and 2.8;
// at 4096 tokens 80 heads of 128 40.4 and 34.5, 48 heads of 64 17.4 and 15.7, 24 heads of
// 256 26.3 and 22.4, 18 heads of 128 16.5 and 14.5.  Where a block holds all heads, threads
// would idle: 4096 tokens of 9 heads of 128 7.1 and 8.9, of 16 heads 11.7 and 12.9.  fp32
// has twice the bytes on their way as it is, and gains only in the largest calls: 48 heads
// of 128, 1024 tokens 11.3 and 13.6 us, 4096 tokens (12288 blocks) 36.2 and 37.8, 8192
// tokens 74.6 and 68.3; 20 heads, 8192 tokens (16384 blocks) 40.6 and 36.4.  Halves that
// pair up are read in 8-byte pieces, and there one head a thread is as fast or faster
// throughout (bf16, 48 heads of 128, 4096 tokens 27.3 against 30.2 us, 512 tokens 3.9
// against 4.9), so they always take it.
constexpr int kHeads = 3;
template <typename E>
constexpr int kManyBlocks = sizeof(E) == 2 ? 1000 : 16000;

struct AppendParams {
    const void *q, *k, *v;
    long long ld_q, ld_k, ld_v;
    int n_q, n_kv, d, page_shift;
    const int *positions;
    const long long *slots;
    const float *cos_sin;
    int n_pos, rot;
    const void *q_norm, *k_norm;
    float eps, inv_d;
    void *q_out, *k_pages, *v_pages;
    long long n_slots;
    int *status;
};

// The lanes of this thread's head within its warp.
template <int LANES>
__device__ __forceinline__ unsigned group_mask() {
    return LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1) << ((threadIdx.x & 31) / LANES * LANES);
}

// Four elements, as loaded and as floats.
template <typename E>
struct Quad;
template <>
struct Quad<__nv_bfloat16> {
    uint2 v;
    __device__ __forceinline__ void get(float *f) const {
        const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v.x));
        const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v.y));
        f[0] = a.x;
        f[1] = a.y;
        f[2] = b.x;
        f[3] = b.y;
    }
    __device__ __forceinline__ void set(const float *f) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
        v = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
};
template <>
struct Quad<float> {
    float4 v;
    __device__ __forceinline__ void get(float *f) const {
        f[0] = v.x;
        f[1] = v.y;
        f[2] = v.z;
        f[3] = v.w;
    }
    __device__ __forceinline__ void set(const float *f) { v = make_float4(f[0], f[1], f[2], f[3]); }
};

// Two quads of a head: places o0 and o1, or side by side (not APART).
template <typename E>
struct Quads {
    Quad<E> a, b;
};
template <typename E, bool APART>
__device__ __forceinline__ void load_quads(Quads<E> &h, const E *head, int o0, int o1) {
    if constexpr (!APART && sizeof(E) == 2) {
        const uint4 v = *reinterpret_cast<const uint4 *>(head + o0);
        h.a.v = make_uint2(v.x, v.y);
        h.b.v = make_uint2(v.z, v.w);
    } else {
        h.a = *reinterpret_cast<const Quad<E> *>(head + o0);
        h.b = *reinterpret_cast<const Quad<E> *>(head + o1);
    }
}
template <typename E, bool APART>
__device__ __forceinline__ void store_quads(const Quads<E> &h, E *head, int o0, int o1) {
    if constexpr (!APART && sizeof(E) == 2) {
        *reinterpret_cast<uint4 *>(head + o0) = make_uint4(h.a.v.x, h.a.v.y, h.b.v.x, h.b.v.y);
    } else {
        *reinterpret_cast<Quad<E> *>(head + o0) = h.a;
        *reinterpret_cast<Quad<E> *>(head + o1) = h.b;
    }
}

// PAIRS: how elements pair up.  kNear: neighbours (a thread's quads are neighbours too);
// kFar: i and i + rot/2 (its quads are rot/2 apart); both with rot a multiple of 8 and an
// aligned table.  kAnyNear, kAnyFar: without those conditions, quads side by side.
// HEADS: heads a thread.
enum { kNear, kFar, kAnyNear, kAnyFar };

template <typename E, int LANES, int PAIRS, int HEADS>
__global__ void __launch_bounds__(kThreads, 5) append_kernel(const AppendParams p) {
    constexpr int kGroups = kThreads / LANES;
    constexpr int kTable = PAIRS == kAnyFar ? 8 : 4;
    __shared__ float rows[PAIRS == kAnyFar ? kThreads * 8 : 1];
    const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    const int heads = p.n_q + 2 * p.n_kv, half = p.rot >> 1;
    const int head_first = blockIdx.y * kGroups * HEADS + group;
    const long long t = blockIdx.x;
    const int at = lane * 8;
    const bool inside = at < p.d, turns = at < p.rot;
    // places of the thread's two quads in a head
    const int o0 = PAIRS == kFar && turns ? lane * 4 : at, o1 = PAIRS == kFar && turns ? half + lane * 4 : at + 4;

    constexpr bool kApart = PAIRS == kFar;
    Quads<E> held[HEADS];
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
        const int head = head_first + u * kGroups;
        const E *src = head < p.n_q ? static_cast<const E *>(p.q) + t * p.ld_q + head * p.d
                       : head < p.n_q + p.n_kv ? static_cast<const E *>(p.k) + t * p.ld_k + (head - p.n_q) * p.d
                                               : static_cast<const E *>(p.v) + t * p.ld_v + (head - p.n_q - p.n_kv) * p.d;
        if (head < heads && inside) load_quads<E, kApart>(held[u], src, o0, o1);
    }
    const long long slot = p.slots[t];
    float c[kTable], s[kTable];
    if (half) {
        int pos = p.positions[t];
        if (pos < 0 || pos >= p.n_pos) {
            if (threadIdx.x == 0) flag_status(p.status, LORA_DEV_BAD_POSITION);
            pos = pos < 0 ? 0 : p.n_pos - 1;
        }
        const float *row = p.cos_sin + (long long)pos * p.rot;
        if (PAIRS == kNear || PAIRS == kFar) {
            if (turns) {
                *reinterpret_cast<float4 *>(c) = *reinterpret_cast<const float4 *>(row + lane * 4);
                *reinterpret_cast<float4 *>(s) = *reinterpret_cast<const float4 *>(row + half + lane * 4);
            }
        } else {
#pragma unroll
            for (int e = 0; e < kTable; ++e) {
                const int x = PAIRS == kAnyFar ? at + e : at + 2 * e, i = PAIRS == kAnyNear ? x >> 1 : x < half ? x : x - half;
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
        if (inside) {
            held[u].a.get(h);
            held[u].b.get(h + 4);
        }
        const E *norm = static_cast<const E *>(is_q ? p.q_norm : p.k_norm);
        if (!is_v && norm) {
            float sum = 0.f, w[8] = {};
            if (inside) {
                Quads<E> n;
                load_quads<E, kApart>(n, norm, o0, o1);
                n.a.get(w);
                n.b.get(w + 4);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += h[e] * h[e];
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(group_mask<LANES>(), sum, o);
            const float r = rsqrtf(fmaf(sum, p.inv_d, p.eps));
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = h[e] * r * w[e];
        }
        if (!is_v && half) {
            if (PAIRS == kFar) {
                if (turns) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float a = h[e], b = h[4 + e];
                        h[e] = a * c[e] - b * s[e];
                        h[4 + e] = a * s[e] + b * c[e];
                    }
                }
            } else if (PAIRS == kAnyFar) {
                float *mine = rows + group * (LANES * 8);
#pragma unroll
                for (int e = 0; e < 8; ++e) mine[at + e] = h[e];
                __syncwarp(group_mask<LANES>());
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (at + e < half) h[e] = h[e] * c[e] - mine[at + e + half] * s[e];
                    else if (at + e < p.rot) h[e] = mine[at + e - half] * s[e] + h[e] * c[e];
                __syncwarp(group_mask<LANES>());
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (at + 2 * e < p.rot) {
                        const float a = h[2 * e], b = h[2 * e + 1];
                        h[2 * e] = a * c[e] - b * s[e];
                        h[2 * e + 1] = a * s[e] + b * c[e];
                    }
            }
        }
        if (!inside) continue;
        E *dst;
        if (is_q) {
            dst = static_cast<E *>(p.q_out) + (t * p.n_q + head) * p.d;
        } else {
            if (!stored) continue;
            const int kv_head = head - p.n_q - (is_v ? p.n_kv : 0);
            dst = static_cast<E *>(is_v ? p.v_pages : p.k_pages) + (((page * p.n_kv + kv_head) << p.page_shift) + off) * p.d;
        }
        held[u].a.set(h);
        held[u].b.set(h + 4);
        store_quads<E, kApart>(held[u], dst, o0, o1);
    }
}

template <typename E, int LANES, int PAIRS>
void launch(const AppendParams &p, int T, cudaStream_t st) {
    constexpr int kGroups = kThreads / LANES;
    const int heads = p.n_q + 2 * p.n_kv;
    const dim3 one(T, (heads + kGroups - 1) / kGroups), more(T, (heads + kGroups * kHeads - 1) / (kGroups * kHeads));
    if constexpr (PAIRS == kNear) {
        if (one.y > 1 && (long long)one.x * one.y > kManyBlocks<E>) {
            append_kernel<E, LANES, PAIRS, kHeads><<<more, kThreads, 0, st>>>(p);
            return;
        }
    }
    append_kernel<E, LANES, PAIRS, 1><<<one, kThreads, 0, st>>>(p);
}

template <typename E, int LANES>
void launch(const AppendParams &p, int T, bool interleaved, cudaStream_t st) {
    const bool table = aligned16(p.cos_sin);
    if (interleaved) {
        if (table && p.rot % 8 == 0) launch<E, LANES, kNear>(p, T, st);
        else launch<E, LANES, kAnyNear>(p, T, st);
    } else {
        if (table && p.rot % 8 == 0) launch<E, LANES, kFar>(p, T, st);
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
    p.inv_d = 1.f / (float)d;
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
