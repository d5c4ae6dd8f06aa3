// Shared by the kernels for products with 4-bit weights.
#pragma once

#include "decode.cuh"

namespace lora {
namespace decode {

struct W4Params {
    const void *x;
    const uint8_t *codes;
    const __nv_bfloat16 *scales;
    const uint8_t *zeros;        // NULL: 8 everywhere
    void *y;
    int T, h_in, h_out, groups;  // groups: h_in / group
};

// Eight codes of one word as four bf16 pairs (k, k + 4), k = 0..3, less the zero:
// 0x4300 | code is 128 + code in bf16, and 128 + code - (128 + zero) is exact.  The
// order of k inside a word is free as long as x follows it (pair_x below).
__device__ __forceinline__ void code_pairs(uint32_t w, __nv_bfloat162 offset, uint32_t (&out)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t v = ((w >> (4 * k)) & 0x000f000fu) | 0x43004300u;
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), offset);
        out[k] = *reinterpret_cast<const uint32_t *>(&d);
    }
}
// The same as pairs of neighbours (2 k, 2 k + 1), for x as it lies in memory: two
// instructions a word more.
__device__ __forceinline__ void code_neighbours(uint32_t w, __nv_bfloat162 offset, uint32_t (&out)[4]) {
    const uint32_t odd = w >> 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t v = (__byte_perm(w, odd, 0x4400 + 0x1111 * k) & 0x000f000fu) | 0x43004300u;
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), offset);
        out[k] = *reinterpret_cast<const uint32_t *>(&d);
    }
}
// 128 + zero, twice.
__device__ __forceinline__ __nv_bfloat162 code_offset(uint32_t zero) {
    const uint32_t v = (0x4300u | zero) * 0x10001u;
    return *reinterpret_cast<const __nv_bfloat162 *>(&v);
}
// Eight bf16 of x (four words) in the order of code_pairs.
__device__ __forceinline__ void pair_x(uint4 x, uint32_t (&out)[4]) {
    out[0] = __byte_perm(x.x, x.z, 0x5410);
    out[1] = __byte_perm(x.x, x.z, 0x7632);
    out[2] = __byte_perm(x.y, x.w, 0x5410);
    out[3] = __byte_perm(x.y, x.w, 0x7632);
}
// fp32 x as three bf16 parts in the order of code_pairs: the leading 8 bits, the next
// 8 and the rest, which is exact.  What is not finite has no rest (infinity less
// itself would be NaN), and a NaN stays one without its lower bits.
__device__ __forceinline__ void split_x(const float (&x)[8], uint32_t (&hi)[4], uint32_t (&mid)[4], uint32_t (&lo)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t first[2], second[2];
        float rest[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float f = x[k + 4 * i];
            const bool finite = fabsf(f) < INFINITY;
            first[i] = __float_as_uint(f) | (f != f ? 0x00400000u : 0u);
            const float r = finite ? f - __uint_as_float(first[i] & 0xffff0000u) : 0.f;
            second[i] = __float_as_uint(r);
            rest[i] = r - __uint_as_float(second[i] & 0xffff0000u);
        }
        hi[k] = __byte_perm(first[0], first[1], 0x7632);
        mid[k] = __byte_perm(second[0], second[1], 0x7632);
        const __nv_bfloat162 h = __floats2bfloat162_rn(rest[0], rest[1]);
        lo[k] = *reinterpret_cast<const uint32_t *>(&h);
    }
}

// w4_tc.cu: T of more than a few tokens.
int launch_w4_tc(int dtype, const W4Params &p, int group, cudaStream_t st);

}  // namespace decode
}  // namespace lora
