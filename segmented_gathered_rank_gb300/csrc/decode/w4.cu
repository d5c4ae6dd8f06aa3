// Matrix products with 4-bit weights (lora_w4_matvec):
//   y[t][n] = sum_g s[n][g] * sum_{k in g} x[t][k] * (c[n][k] - z[n][g])
//
// The codes are read once: half a byte a weight against 2 T flops, so memory is the
// bound up to T of about 70.  Codes less zeros are whole numbers of 5 bits, exact in
// bf16, so the inner sums run on the tensor cores without rounding the weights, and
// each group's sum is scaled in fp32.
//
// Up to 16 tokens: w4_rows_kernel below, warp MMAs on registers filled straight from
// memory.  More: w4_tc.cu, whose tcgen05 rate the flops then need.
#include "w4.cuh"

namespace lora {
namespace {

using namespace decode;

constexpr int kWarps = 8;
constexpr int kBlock = 128;        // weights of a row that a warp takes at a time
constexpr int kDepth = 4;          // such blocks on their way from memory

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A block of 16 rows of W: warp w takes blocks w, w + 8, ... of kBlock columns for
// all rows (rows lane/4 and lane/4 + 8 a thread), so a row's 64 bytes are one
// request, x is read once a warp, and the warps' sums meet in shared memory.
// Word j of a thread's four holds columns column(j) .. + 7 of the block: a word's
// four threads (lane % 4) are in one group, whatever its size.
template <int GROUP>
__device__ __forceinline__ int column(int j, int t4) {
    return GROUP == 128 ? t4 * 32 + j * 8 : GROUP == 64 ? (j >> 1) * 64 + t4 * 16 + (j & 1) * 8 : j * 32 + t4 * 8;
}

// What a thread loads of a block: its words of two rows, and scales and zeros: those
// of group lane % 4 (they are passed around the four threads), or of the one group.
struct BlockWords {
    uint32_t w[2][4];
    uint32_t zero[2];
    float scale[2];
};

template <int GROUP>
__device__ __forceinline__ void load_block(const W4Params &p, const uint8_t *(&rows)[2], const int (&n)[2], int block, int t4,
                                           BlockWords &b) {
    constexpr int kGroups = kBlock / GROUP;
    const int g = min(block * kGroups + (kGroups > 1 ? t4 % kGroups : 0), p.groups - 1);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const uint8_t *src = rows[r] + block * (kBlock / 2);
        const int left = p.h_in - block * kBlock;      // h_in ends inside the last block at a group's end
        if (GROUP == 128) {
            const uint4 u = __ldg(reinterpret_cast<const uint4 *>(src + column<128>(0, t4) / 2));
            b.w[r][0] = u.x;
            b.w[r][1] = u.y;
            b.w[r][2] = u.z;
            b.w[r][3] = u.w;
        } else if (GROUP == 64) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint2 u = h * 64 < left ? __ldg(reinterpret_cast<const uint2 *>(src + column<64>(2 * h, t4) / 2)) : make_uint2(0, 0);
                b.w[r][2 * h] = u.x;
                b.w[r][2 * h + 1] = u.y;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                b.w[r][j] = j * 32 < left ? __ldg(reinterpret_cast<const uint32_t *>(src + column<32>(j, t4) / 2)) : 0u;
        }
        const long long at = (long long)n[r] * p.groups + g;
        b.scale[r] = __bfloat162float(p.scales[at]);
        b.zero[r] = p.zeros ? __ldg(p.zeros + at) : 8u;
    }
}

template <typename E, int NT>
struct BlockX {
    uint4 v[NT][4][sizeof(E) / 2];
};

template <typename E, int GROUP, int NT>
__device__ __forceinline__ void load_x(const W4Params &p, int block, int g4, int t4, BlockX<E, NT> &b) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int t = nt * 8 + g4;
        const E *src = static_cast<const E *>(p.x) + (long long)t * p.h_in + block * kBlock;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = column<GROUP>(j, t4);
            const bool in = t < p.T && block * kBlock + col < p.h_in;
#pragma unroll
            for (int h = 0; h < (int)sizeof(E) / 2; ++h)
                b.v[nt][j][h] = in ? __ldg(reinterpret_cast<const uint4 *>(src + col) + h) : make_uint4(0, 0, 0, 0);
        }
    }
}

template <typename E, int GROUP, int NT>
__global__ void __launch_bounds__(kWarps * 32) w4_rows_kernel(const W4Params p) {
    constexpr int kGroups = kBlock / GROUP;
    __shared__ float sums[kWarps][NT * 8][17];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g4 = lane >> 2, t4 = lane & 3;
    const int n0 = blockIdx.x * 16, blocks = (p.h_in + kBlock - 1) / kBlock;
    const int n[2] = {min(n0 + g4, p.h_out - 1), min(n0 + g4 + 8, p.h_out - 1)};
    const uint8_t *rows[2] = {p.codes + (long long)n[0] * (p.h_in / 2), p.codes + (long long)n[1] * (p.h_in / 2)};
    float acc[NT][4] = {};
    BlockWords ring[kDepth];
    BlockX<E, NT> xs;
#pragma unroll
    for (int i = 0; i < kDepth; ++i)
        if (warp + i * kWarps < blocks) load_block<GROUP>(p, rows, n, warp + i * kWarps, t4, ring[i]);
    for (int base = warp; base < blocks; base += kDepth * kWarps) {
#pragma unroll
        for (int i = 0; i < kDepth; ++i) {
            const int block = base + i * kWarps;
            if (block >= blocks) break;
            load_x<E, GROUP, NT>(p, block, g4, t4, xs);
            const BlockWords cur = ring[i];
            if (block + kDepth * kWarps < blocks) load_block<GROUP>(p, rows, n, block + kDepth * kWarps, t4, ring[i]);
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                float c[NT][4] = {};
                float scale[2];
                __nv_bfloat162 offset[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    uint32_t z = cur.zero[r];
                    scale[r] = cur.scale[r];
                    if (kGroups > 1) {
                        z = __shfl_sync(0xffffffffu, z, (lane & ~3) | g);
                        scale[r] = __shfl_sync(0xffffffffu, scale[r], (lane & ~3) | g);
                    }
                    offset[r] = code_offset(z);
                }
#pragma unroll
                for (int j = g * (4 / kGroups); j < (g + 1) * (4 / kGroups); ++j) {
                    uint32_t a[2][4];
                    code_pairs(cur.w[0][j], offset[0], a[0]);
                    code_pairs(cur.w[1][j], offset[1], a[1]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if constexpr (sizeof(E) == 2) {
                            uint32_t b[4];
                            pair_x(xs.v[nt][j][0], b);
                            mma16816(c[nt], a[0][0], a[1][0], a[0][1], a[1][1], b[0], b[1]);
                            mma16816(c[nt], a[0][2], a[1][2], a[0][3], a[1][3], b[2], b[3]);
                        } else {
                            const float f[8] = {__uint_as_float(xs.v[nt][j][0].x), __uint_as_float(xs.v[nt][j][0].y),
                                                __uint_as_float(xs.v[nt][j][0].z), __uint_as_float(xs.v[nt][j][0].w),
                                                __uint_as_float(xs.v[nt][j][1].x), __uint_as_float(xs.v[nt][j][1].y),
                                                __uint_as_float(xs.v[nt][j][1].z), __uint_as_float(xs.v[nt][j][1].w)};
                            uint32_t b[3][4];
                            split_x(f, b[0], b[1], b[2]);
#pragma unroll
                            for (int part = 2; part >= 0; --part) {
                                mma16816(c[nt], a[0][0], a[1][0], a[0][1], a[1][1], b[part][0], b[part][1]);
                                mma16816(c[nt], a[0][2], a[1][2], a[0][3], a[1][3], b[part][2], b[part][3]);
                            }
                        }
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[nt][e] = fmaf(scale[e >> 1], c[nt][e], acc[nt][e]);
            }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[warp][nt * 8 + t4 * 2 + (e & 1)][g4 + (e >> 1) * 8] = acc[nt][e];
    __syncthreads();
    for (int x = threadIdx.x; x < NT * 8 * 16; x += kWarps * 32) {
        const int t = x >> 4, r = x & 15;
        if (t >= p.T || n0 + r >= p.h_out) continue;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += sums[w][t][r];
        E *dst = static_cast<E *>(p.y) + (long long)t * p.h_out + n0 + r;
        if constexpr (sizeof(E) == 2) *dst = __float2bfloat16_rn(s);
        else *dst = s;
    }
}

template <typename E, int GROUP>
void launch(const W4Params &p, cudaStream_t st) {
    const unsigned grid = (p.h_out + 15) / 16;
    if (p.T <= 8) w4_rows_kernel<E, GROUP, 1><<<grid, kWarps * 32, 0, st>>>(p);
    else w4_rows_kernel<E, GROUP, 2><<<grid, kWarps * 32, 0, st>>>(p);
}

template <typename E>
void launch(const W4Params &p, int group, cudaStream_t st) {
    if (group == 128) launch<E, 128>(p, st);
    else if (group == 64) launch<E, 64>(p, st);
    else launch<E, 32>(p, st);
}

constexpr int kRowsTokens = 16;

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" int lora_w4_matvec(int dtype, const void *x, int T, int h_in, const void *codes, const void *scales,
                              const void *zeros, int group, int h_out, void *y, lora_stream stream) {
    if ((dtype != LORA_F32 && dtype != LORA_BF16) || T < 0 || h_in <= 0 || h_out <= 0) return LORA_ERR_ARG;
    if ((group != 32 && group != 64 && group != 128) || h_in % group) return LORA_ERR_SHAPE;
    if (T == 0) return LORA_OK;
    if (!x || !codes || !scales || !y || !aligned16(x) || !aligned16(codes) || !aligned16(y) ||
        ((uintptr_t)scales & 1u))
        return LORA_ERR_ARG;
    decode::W4Params p;
    p.x = x;
    p.codes = static_cast<const uint8_t *>(codes);
    p.scales = static_cast<const __nv_bfloat16 *>(scales);
    p.zeros = static_cast<const uint8_t *>(zeros);
    p.y = y;
    p.T = T;
    p.h_in = h_in;
    p.h_out = h_out;
    p.groups = h_in / group;
    const size_t e = dtype == LORA_BF16 ? 2 : 4;
    for (int t = 0; t < T; t += kRowsTokens) {
        p.x = static_cast<const char *>(x) + (size_t)t * h_in * e;
        p.y = static_cast<char *>(y) + (size_t)t * h_out * e;
        p.T = T - t < kRowsTokens ? T - t : kRowsTokens;
        if (dtype == LORA_BF16) launch<__nv_bfloat16>(p, group, (cudaStream_t)stream);
        else launch<float>(p, group, (cudaStream_t)stream);
        count_launch();
    }
    return cuda_status(cudaGetLastError());
}
