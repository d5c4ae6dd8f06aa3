// Norm, rotation and append of new tokens (lora_kv_append, lora_kv_append_axes).
//
// Per query and key head h (d elements, fp32 arithmetic, one rounding on store):
//   h <- h / sqrt(mean(h^2) + eps) * norm,  then (a, b) <- (a c - b s, a s + b c)
// over the pairs of the first rot elements; values are copied.  The bytes are
// each head read once and written once: memory is the bound for large T, the
// chain of dependent loads (position -> table row; slot -> address) for small.
// Measured, bf16, heads of 128: 1 token 2.0 us, 256 tokens of 48 heads with norms
// 3.1 us, 8192 tokens 39.8 us (5.2 TB/s).  With axes 1 token 2.6 us: a position and a
// table entry a pair where a quad's pairs differ in axis, one of each where they do not.
// Many tokens with axes go to append_stream.cu.
//
// Layout: LANES threads (the power of two >= d/8) hold one head, 8 elements each in two
// quads that are each other's partners in the rotation, so a pair meets in a thread (or,
// when rot is no multiple of 8, in a row of shared memory).  A block takes heads of one
// token, several a thread for long batches; its lanes keep their pairs' cosines and
// sines for all of them.
#include <string.h>

#include "append.cuh"

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

// The table's row for an axis of token t, its position clamped into the table (flagged).
__device__ __forceinline__ const float *axis_row(const AppendParams &p, long long t, int axis) {
    int pos = __ldg(p.positions + t * p.n_axes + axis);
    if (pos < 0 || pos >= p.n_pos) {
        flag_status(p.status, LORA_DEV_BAD_POSITION);
        pos = pos < 0 ? 0 : p.n_pos - 1;
    }
    return p.cos_sin + (long long)pos * p.rot;
}
// Cosines and sines of the pairs 4 * quad .. + 3.  Sections of a head have whole quads of one axis: two vector loads.
__device__ __forceinline__ void load_axes(const AppendParams &p, long long t, int quad, int half, float *c, float *s) {
    const uint32_t axes = p.axes[quad], first = axes & 3;
    if (axes == first * 0x55u) {
        const float *row = axis_row(p, t, first) + quad * 4;
        *reinterpret_cast<float4 *>(c) = *reinterpret_cast<const float4 *>(row);
        *reinterpret_cast<float4 *>(s) = *reinterpret_cast<const float4 *>(row + half);
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float *row = axis_row(p, t, (axes >> (2 * e)) & 3) + quad * 4 + e;
        c[e] = row[0];
        s[e] = row[half];
    }
}

// AXES: a token has n_axes positions, and each pair turns by that of its axis.
template <typename E, int LANES, int PAIRS, int HEADS, bool AXES>
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
    if (AXES && half) {
        if (PAIRS == kNear || PAIRS == kFar) {
            if (turns) load_axes(p, t, lane, half, c, s);
        } else {
#pragma unroll
            for (int e = 0; e < kTable; ++e) {
                const int x = PAIRS == kAnyFar ? at + e : at + 2 * e, i = PAIRS == kAnyNear ? x >> 1 : x < half ? x : x - half;
                if (x < p.rot) {
                    const float *row = axis_row(p, t, (p.axes[i >> 2] >> (2 * (i & 3))) & 3);
                    c[e] = row[i];
                    s[e] = row[half + i];
                }
            }
        }
    } else if (half) {
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

template <typename E, int LANES, int PAIRS, bool AXES>
void launch(const AppendParams &p, int T, cudaStream_t st) {
    constexpr int kGroups = kThreads / LANES;
    const int heads = p.n_q + 2 * p.n_kv;
    const dim3 one(T, (heads + kGroups - 1) / kGroups), more(T, (heads + kGroups * kHeads - 1) / (kGroups * kHeads));
    if constexpr (PAIRS == kNear) {
        if (one.y > 1 && (long long)one.x * one.y > kManyBlocks<E>) {
            append_kernel<E, LANES, PAIRS, kHeads, AXES><<<more, kThreads, 0, st>>>(p);
            return;
        }
    }
    append_kernel<E, LANES, PAIRS, 1, AXES><<<one, kThreads, 0, st>>>(p);
}

template <typename E, int LANES, bool AXES>
void launch(const AppendParams &p, int T, bool interleaved, cudaStream_t st) {
    const bool table = aligned16(p.cos_sin);
    if (interleaved) {
        if (table && p.rot % 8 == 0) launch<E, LANES, kNear, AXES>(p, T, st);
        else launch<E, LANES, kAnyNear, AXES>(p, T, st);
    } else {
        if (table && p.rot % 8 == 0) launch<E, LANES, kFar, AXES>(p, T, st);
        else launch<E, LANES, kAnyFar, AXES>(p, T, st);
    }
}

template <typename E, bool AXES>
void launch(const AppendParams &p, int T, bool interleaved, cudaStream_t st) {
    if (p.d <= 64) launch<E, 8, AXES>(p, T, interleaved, st);
    else if (p.d <= 128) launch<E, 16, AXES>(p, T, interleaved, st);
    else launch<E, 32, AXES>(p, T, interleaved, st);
}

// pair_axis: NULL for one position a token.
int append(const lora_kv_pages *kv, const void *q, int ld_q, const void *k, int ld_k, const void *v, int ld_v, int T,
           int n_q_heads, const int *positions, int n_axes, const unsigned char *pair_axis, const long long *slots,
           const float *cos_sin, int n_pos, int rot_dim, int interleaved, const void *q_norm, const void *k_norm, float eps,
           void *q_out, cudaStream_t st) {
    int rc = decode::check_kv(kv, n_q_heads);
    if (rc) return rc;
    if (T < 0 || rot_dim < 0 || !(eps >= 0.f)) return LORA_ERR_ARG;
    const int d = kv->head_dim, vec = kv->dtype == LORA_BF16 ? 8 : 4;   // elements of 16 bytes
    if (rot_dim > d || rot_dim % 2) return LORA_ERR_SHAPE;
    if ((long long)n_q_heads + 2LL * kv->n_kv_heads > 65535) return LORA_ERR_SHAPE;
    if (ld_k < kv->n_kv_heads * d || ld_v < kv->n_kv_heads * d || ld_k % vec || ld_v % vec) return LORA_ERR_SHAPE;
    if (n_q_heads && (ld_q < n_q_heads * d || ld_q % vec)) return LORA_ERR_SHAPE;
    AppendParams p;
    p.n_axes = n_axes;
    p.used_axes = 0;
    if (pair_axis) {
        memset(p.axes, 0, sizeof(p.axes));
        for (int i = 0; i < rot_dim / 2; ++i) {
            if (pair_axis[i] >= n_axes) return LORA_ERR_ARG;
            p.axes[i >> 2] |= (unsigned char)(pair_axis[i] << (2 * (i & 3)));
            p.used_axes |= 1u << pair_axis[i];
        }
    }
    if (T == 0) return LORA_OK;
    if (!k || !v || !slots || !aligned16(k) || !aligned16(v) || ((uintptr_t)slots & 7u)) return LORA_ERR_ARG;
    if (n_q_heads && (!q || !q_out || !aligned16(q) || !aligned16(q_out))) return LORA_ERR_ARG;
    if (q_out && q_out == q && ld_q != n_q_heads * d && T > 1) return LORA_ERR_ARG;
    if (rot_dim && (!cos_sin || !positions || n_pos < 1 || ((uintptr_t)cos_sin & 3u) || ((uintptr_t)positions & 3u)))
        return LORA_ERR_ARG;
    if (!aligned16(q_norm) || !aligned16(k_norm)) return LORA_ERR_ARG;
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
    const bool near = interleaved != 0;
    if (pair_axis && streams(p, T, kv->dtype == LORA_BF16 ? 2 : 4)) return launch_append_stream(p, T, kv->dtype == LORA_BF16, near, st);
    if (pair_axis) {
        if (kv->dtype == LORA_BF16) launch<__nv_bfloat16, true>(p, T, near, st);
        else launch<float, true>(p, T, near, st);
    } else {
        if (kv->dtype == LORA_BF16) launch<__nv_bfloat16, false>(p, T, near, st);
        else launch<float, false>(p, T, near, st);
    }
    count_launch();
    return cuda_status(cudaGetLastError());
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" int lora_kv_append(const lora_kv_pages *kv, const void *q, int ld_q, const void *k, int ld_k, const void *v,
                              int ld_v, int T, int n_q_heads, const int *positions, const long long *slots,
                              const float *cos_sin, int n_pos, int rot_dim, int interleaved, const void *q_norm,
                              const void *k_norm, float eps, void *q_out, lora_stream stream) {
    return append(kv, q, ld_q, k, ld_k, v, ld_v, T, n_q_heads, positions, 1, nullptr, slots, cos_sin, n_pos, rot_dim, interleaved,
                  q_norm, k_norm, eps, q_out, (cudaStream_t)stream);
}

extern "C" int lora_kv_append_axes(const lora_kv_pages *kv, const lora_append_axes *a, lora_stream stream) {
    if (!a || a->n_axes < 1 || a->n_axes > LORA_MAX_AXES) return LORA_ERR_ARG;
    return append(kv, a->q, a->ld_q, a->k, a->ld_k, a->v, a->ld_v, a->T, a->n_q_heads, a->positions, a->n_axes, a->pair_axis, a->slots,
                  a->cos_sin, a->n_pos, a->rot_dim, a->interleaved, a->q_norm, a->k_norm, a->eps, a->q_out, (cudaStream_t)stream);
}
