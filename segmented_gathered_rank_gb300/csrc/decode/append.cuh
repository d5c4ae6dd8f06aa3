// Shared by the kernels that append new tokens.
#pragma once

#include "decode.cuh"

namespace lora {
namespace decode {

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
    int n_axes;                              // positions a token
    unsigned char axes[kMaxHeadDim / 8];     // axis of each pair, two bits each, four pairs a byte
    unsigned used_axes;                      // a bit for each that a pair names
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

// append_stream.cu: tokens with axes, pairs near or far.  launch_append_stream checks nothing: only where streams() holds.
bool streams(const AppendParams &p, int T, int esize);
int launch_append_stream(const AppendParams &p, int T, bool bf16, bool near, cudaStream_t st);

}  // namespace decode
}  // namespace lora
