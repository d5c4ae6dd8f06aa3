// Matrix products with 4-bit weights (lora_w4_matvec):
//   y[t][n] = sum_g s[n][g] * sum_{k in g} x[t][k] * (c[n][k] - z[n][g])
//
// The codes are read once: half a byte a weight against 2 T flops (6 T with fp32
// activations), so the bytes are the larger part of the floor up to T of about 70 (23 in
// fp32) at 1.9 PFLOP/s and 6.8 TB/s.  Codes less zeros are whole numbers of 5 bits, exact
// in bf16, so the inner sums run on the tensor cores without rounding the weights, and
// each group's sum is scaled in fp32.
//
// Up to 8 tokens: w4_rows_kernel below, warp MMAs on registers filled straight from
// memory, unless its blocks would stage too much of x each (takes_rows).  More: w4_tc.cu,
// whose tcgen05 rate the flops then need; 16 tokens would be two columns of MMAs here
// (4096 -> 16384, two calls of 8: 29.6 against 16.6 us).
//
// w4_rows_kernel reads 3.4 TB/s of a large matrix (1 x 16384 -> 16384 41.0 us; 1 x 4096 ->
// 16384 12.3 us), half of what memory gives.  No unit is full either: the shifts and masks
// that turn codes into bf16 pairs take 58 % of the integer pipe, and a warp stalls about
// as long for that pipe as for its loads and for fixed latencies.  Starting, staging x
// and adding up take 3.5 us, which is all of a small call (1 x 4096 -> 1024 3.7 us).
//
// fp32 x enters as three bf16 parts, whose sum is x to 2^-24: the products with whole
// numbers are exact and the sums are fp32, so nothing is lost against fp32 arithmetic.
#include "w4.cuh"

namespace lora {
namespace {

using namespace decode;

constexpr int kMaxWarps = 16;
constexpr int kBlock = 128;        // weights of a row that a warp takes at a time
constexpr int kDepth = 4;          // such blocks on their way from memory
constexpr int kXBytes = 192 * 1024;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A thread block has `tiles` tiles of 16 rows of W, so that about one block a SM
// covers all rows, and `slices` warps a tile: warp s of them takes the blocks of
// kBlock columns s, s + slices, ...  Codes go from memory straight into registers,
// kDepth blocks ahead; x lies in shared memory in the order of the MMA operands.
// Word j of a thread's four (rows lane/4 and lane/4 + 8) holds columns column(j) ..
// + 7 of the block: a word's four threads (lane % 4) are in one group, whatever its
// size.
template <int GROUP>
__device__ __forceinline__ int column(int j, int t4) {
    return GROUP == 128 ? t4 * 32 + j * 8 : GROUP == 64 ? (j >> 1) * 64 + t4 * 16 + (j & 1) * 8 : j * 32 + t4 * 8;
}

// What a thread loads of a block: its words of two rows, and scales and zeros: those
// of group lane % 4 (they are passed around the four threads), or of the one group.
struct BlockWords {
    uint32_t w[2][4];
    uint32_t zero[2], scale[2];
};
// Where a thread's two rows are for a round of blocks.
struct Place {
    const uint8_t *codes[2], *zeros[2];
    const __nv_bfloat16 *scales[2];
};

// Codes are read once a call: they leave L2 first.
__device__ __forceinline__ uint64_t once_policy() {
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;\n" : "=l"(policy));
    return policy;
}
__device__ __forceinline__ uint4 ld_once(const uint4 *p, uint64_t policy) {
    uint4 u;
    asm volatile("ld.global.nc.L2::cache_hint.v4.b32 {%0, %1, %2, %3}, [%4], %5;\n"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(p), "l"(policy));
    return u;
}
__device__ __forceinline__ uint2 ld_once(const uint2 *p, uint64_t policy) {
    uint2 u;
    asm volatile("ld.global.nc.L2::cache_hint.v2.b32 {%0, %1}, [%2], %3;\n" : "=r"(u.x), "=r"(u.y) : "l"(p), "l"(policy));
    return u;
}
__device__ __forceinline__ uint32_t ld_once(const uint32_t *p, uint64_t policy) {
    uint32_t u;
    asm volatile("ld.global.nc.L2::cache_hint.b32 %0, [%1], %2;\n" : "=r"(u) : "l"(p), "l"(policy));
    return u;
}

// The block `step` blocks after the place, `left` columns before the row's end; at a row's
// end the words past it are read from the row's start (x is zero there).
template <int GROUP>
__device__ __forceinline__ void load_block(const Place &at, bool has_zeros, int step, int left, int t4, uint64_t policy,
                                           BlockWords &b) {
    constexpr int kGroups = kBlock / GROUP;
    const int g = step * kGroups + (kGroups > 1 ? min(t4 % kGroups, (left - 1) / GROUP) : 0);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const uint8_t *src = at.codes[r] + step * (kBlock / 2);
        if (GROUP == 128) {
            const uint4 u = ld_once(reinterpret_cast<const uint4 *>(src + column<128>(0, t4) / 2), policy);
            b.w[r][0] = u.x;
            b.w[r][1] = u.y;
            b.w[r][2] = u.z;
            b.w[r][3] = u.w;
        } else if (GROUP == 64) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint2 u = ld_once(reinterpret_cast<const uint2 *>(src + (h * 64 < left ? column<64>(2 * h, t4) / 2 : 0)), policy);
                b.w[r][2 * h] = u.x;
                b.w[r][2 * h + 1] = u.y;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                b.w[r][j] = ld_once(reinterpret_cast<const uint32_t *>(src + (j * 32 < left ? column<32>(j, t4) / 2 : 0)), policy);
        }
        b.scale[r] = __ldg(reinterpret_cast<const unsigned short *>(at.scales[r] + g));
        b.zero[r] = has_zeros ? __ldg(at.zeros[r] + g) : 8u;
    }
}

// One thread's operand of 16 bytes: x of one token in one word's columns.  Place of
// (block, word j, part, lane) in shared memory, 16-byte units.
template <int PARTS>
__device__ __forceinline__ int x_place(int block, int j, int part, int lane) {
    return ((block * 4 + j) * PARTS + part) * 32 + lane;
}

// x of the columns of blocks [first, first + blocks) into shared memory.
template <typename E, int GROUP>
__device__ __forceinline__ void stage_x(const W4Params &p, int first, int blocks, uint4 *xs) {
    constexpr int kParts = sizeof(E) == 2 ? 1 : 3;
    for (int i = threadIdx.x; i < blocks * 16 * p.T; i += blockDim.x) {
        const int t = i / (blocks * 16), x = i - t * (blocks * 16), block = x >> 4, j = (x >> 2) & 3, t4 = x & 3;
        const int k = (first + block) * kBlock + column<GROUP>(j, t4), lane = t * 4 + t4;
        const E *src = static_cast<const E *>(p.x) + (long long)t * p.h_in + k;
        uint4 part[kParts];
#pragma unroll
        for (int q = 0; q < kParts; ++q) part[q] = make_uint4(0, 0, 0, 0);
        if (k < p.h_in) {
            if constexpr (sizeof(E) == 2) {
                uint32_t o[4];
                pair_x(__ldg(reinterpret_cast<const uint4 *>(src)), o);
                part[0] = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
                float f[8];
                load8(src, f);
                uint32_t o[3][4];
                split_x(f, o[0], o[1], o[2]);
#pragma unroll
                for (int q = 0; q < kParts; ++q) part[q] = make_uint4(o[q][0], o[q][1], o[q][2], o[q][3]);
            }
        }
#pragma unroll
        for (int q = 0; q < kParts; ++q) xs[x_place<kParts>(block, j, q, lane)] = part[q];
    }
}

// A warp takes kDepth blocks a round.  LONG: consecutive ones (256 bytes of a row: memory
// is read in longer pieces); else one of every `slices`, for rows too short for that.
// span: blocks of columns whose x fits in shared memory, whole rounds of them.
template <typename E, int GROUP, bool LONG>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) w4_rows_kernel(const W4Params p, int tiles, int slices, int span) {
    constexpr int kGroups = kBlock / GROUP, kParts = sizeof(E) == 2 ? 1 : 3, kBlockX = 4 * kParts * 512;
    extern __shared__ uint4 xs[];
    float *sums = reinterpret_cast<float *>(xs);        // [warp][token][17], at the end
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g4 = lane >> 2, t4 = lane & 3;
    const int slice = warp % slices, blocks = (p.h_in + kBlock - 1) / kBlock;
    const int step = LONG ? 1 : slices, round = kDepth * slices, start = LONG ? slice * kDepth : slice;
    const uint32_t x_addr = (uint32_t)__cvta_generic_to_shared(xs) + lane * 16;
    const bool has_zeros = p.zeros != nullptr;
    const uint64_t policy = once_policy();
    for (int n_first = blockIdx.x * tiles * 16; n_first < p.h_out; n_first += gridDim.x * tiles * 16) {
        Place next;                 // of the round that is being fetched
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const long long n = min(n_first + (warp / slices) * 16 + g4 + r * 8, p.h_out - 1);
            next.codes[r] = p.codes + n * (p.h_in / 2) + start * (kBlock / 2);
            next.scales[r] = p.scales + n * p.groups + start * kGroups;
            next.zeros[r] = p.zeros + n * p.groups + start * kGroups;
        }
        float acc[4] = {};
        uint4 b = make_uint4(0, 0, 0, 0);       // of tokens past T for good
        BlockWords ring[kDepth];
#pragma unroll
        for (int i = 0; i < kDepth; ++i)
            if (start + i * step < blocks)
                load_block<GROUP>(next, has_zeros, i * step, p.h_in - (start + i * step) * kBlock, t4, policy, ring[i]);
        int base = start;           // the round's first block
        for (int first = 0; first < blocks; first += span) {
            const int end = min(blocks, first + span);
            if (first > 0 || n_first > (int)blockIdx.x * tiles * 16) __syncthreads();
            stage_x<E, GROUP>(p, first, end - first, xs);
            __syncthreads();
            for (; base < end; base += round) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    next.codes[r] += round * (kBlock / 2);
                    next.scales[r] += round * kGroups;
                    next.zeros[r] += round * kGroups;
                }
                uint32_t xb = x_addr + (base - first) * kBlockX;
#pragma unroll
                for (int i = 0; i < kDepth; ++i, xb += step * kBlockX) {
                    if (base + i * step >= end) break;
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        float c[2][4] = {};        // two chains of sums
                        float scale[2];
                        __nv_bfloat162 offset[2];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            uint32_t z = ring[i].zero[r], sc = ring[i].scale[r];
                            if (kGroups > 1) {
                                z = __shfl_sync(0xffffffffu, z, (lane & ~3) | g);
                                sc = __shfl_sync(0xffffffffu, sc, (lane & ~3) | g);
                            }
                            scale[r] = __uint_as_float(sc << 16);
                            offset[r] = code_offset(z);
                        }
#pragma unroll
                        for (int j = g * (4 / kGroups); j < (g + 1) * (4 / kGroups); ++j) {
                            uint32_t a[2][4];
                            code_pairs(ring[i].w[0][j], offset[0], a[0]);
                            code_pairs(ring[i].w[1][j], offset[1], a[1]);
#pragma unroll
                            for (int part = kParts - 1; part >= 0; --part) {        // the smallest part first
                                if (g4 < p.T)
                                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                                                 : "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                                                 : "r"(xb + (j * kParts + part) * 512));
                                mma16816(c[0], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
                                mma16816(c[1], a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[e] = fmaf(scale[e >> 1], c[0][e] + c[1][e], acc[e]);
                    }
                    const int ahead = base + round + i * step;
                    if (ahead < blocks) load_block<GROUP>(next, has_zeros, i * step, p.h_in - ahead * kBlock, t4, policy, ring[i]);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[(warp * 8 + t4 * 2 + (e & 1)) * 17 + g4 + (e >> 1) * 8] = acc[e];
        __syncthreads();
        for (int x = threadIdx.x; x < p.T * tiles * 16; x += blockDim.x) {
            const int t = x / (tiles * 16), r = x - t * (tiles * 16), tile = r >> 4;
            if (n_first + r >= p.h_out) continue;
            float s = 0.f;
            for (int w = 0; w < slices; ++w) s += sums[((tile * slices + w) * 8 + t) * 17 + (r & 15)];
            E *dst = static_cast<E *>(p.y) + (long long)t * p.h_out + n_first + r;
            if constexpr (sizeof(E) == 2) *dst = __float2bfloat16_rn(s);
            else *dst = s;
        }
    }
}

// x of a block of columns in shared memory, and blocks that fit there at once.
template <typename E>
constexpr int kBlockBytes = 4 * (sizeof(E) == 2 ? 1 : 3) * 512;
template <typename E>
constexpr int kFit = kXBytes / kBlockBytes<E>;

// Tiles of 16 rows a thread block: as few as let one block a SM cover all rows, at most 8.
int tiles_of(const W4Params &p, int sms) {
    const int row_tiles = (p.h_out + 15) / 16, each = (row_tiles + sms - 1) / sms;
    return each < 8 ? each : 8;
}

template <typename E, int GROUP>
int launch(const W4Params &p, int sms, cudaStream_t st) {
    const int row_tiles = (p.h_out + 15) / 16, tiles = tiles_of(p, sms);
    const int blocks = (p.h_in + kBlock - 1) / kBlock;
    // all of x in shared memory at once, or spans of whole rounds of the ring
    const int most = blocks <= kFit<E> ? kMaxWarps : kFit<E> / kDepth, slices = kMaxWarps / tiles < most ? kMaxWarps / tiles : most;
    const int span = blocks <= kFit<E> ? blocks : kFit<E> / (slices * kDepth) * (slices * kDepth);
    const size_t sums = (size_t)tiles * slices * 8 * 17 * sizeof(float);
    const size_t smem = (size_t)span * kBlockBytes<E> > sums ? (size_t)span * kBlockBytes<E> : sums;
    const int need = (row_tiles + tiles - 1) / tiles, grid = need < sms ? need : sms;
    const auto kernel = blocks >= kDepth * slices ? w4_rows_kernel<E, GROUP, true> : w4_rows_kernel<E, GROUP, false>;
    if (smem_optin(reinterpret_cast<const void *>(kernel), smem)) return LORA_ERR_CUDA;
    kernel<<<grid, tiles * slices * 32, smem, st>>>(p, tiles, slices, span);
    count_launch();
    return cuda_status(cudaGetLastError());
}

template <typename E>
int launch(const W4Params &p, int group, int sms, cudaStream_t st) {
    return group == 128 ? launch<E, 128>(p, sms, st) : group == 64 ? launch<E, 64>(p, sms, st) : launch<E, 32>(p, sms, st);
}

constexpr int kRowsTokens = 8;       // one MMA's columns
constexpr int kMaxSize = 0x7fff0000;  // of h_in and h_out: loops step past the end by up to 8 tiles of 16 rows on every SM

// Whether w4_rows_kernel takes the tokens: up to 8 when x fits in shared memory at once.  When
// it comes in parts, a block stages and awaits each of them, for as many row tiles as it
// has (0.065 us a thousand elements in bf16, twice that in fp32), while the other kernel
// is 3 to 4 us slower to start, so then only up to kStaged elements a row tile.  Here and
// there, us, one part: 4096 -> 16384 4 tokens 13.3 and 16.5, 8 tokens 14.9 and 16.7, in fp32
// 20.5 and 24.3; 4096 -> 4096 8 tokens 7.2 and 8.5, in fp32 10.3 and 9.9; 4096 -> 1024 8 tokens
// 5.8 and 6.8, in fp32 8.6 and 7.3; 4096 -> 2048 in fp32 8.7 and 9.7.  Parts, up to the limit
// and past it: 16384 -> 4096 (two row tiles) 4 tokens 17.4 and 18.7, 6 tokens 19.5 and 18.6, in
// fp32 3 tokens 23.5 and 26.7, 8 tokens 34.9 and 27.1 (but 4 tokens 25.6 and 27.0); 4128 -> 4001
// in fp32 5 tokens 11.3 and 12.8; 8192 -> 4096 in fp32 5 tokens 15.1 and 15.7, 7 tokens 17.4 and
// 15.8; 13312 -> 1024 (one) 3 tokens 9.6 and 10.5, 5 tokens 11.3 and 10.5; 14336 -> 1024 in fp32
// 1 token 12.4 and 12.9, 8 tokens 32.1 and 14.0; 16384 -> 16384 (seven) 8 tokens 50.1 and 52.7.
constexpr long long kStaged = 40960;        // elements of x, an fp32 one as one and a half
template <typename E>
bool takes_rows(const W4Params &p, int sms) {
    if (p.T > kRowsTokens) return false;
    return (p.h_in + kBlock - 1) / kBlock <= kFit<E> ||
           (long long)p.T * p.h_in * (sizeof(E) == 2 ? 2 : 3) <= 2 * kStaged * tiles_of(p, sms);
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" int lora_w4_matvec(int dtype, const void *x, int T, int h_in, const void *codes, const void *scales,
                              const void *zeros, int group, int h_out, void *y, lora_stream stream) {
    if ((dtype != LORA_F32 && dtype != LORA_BF16) || T < 0 || h_in <= 0 || h_out <= 0) return LORA_ERR_ARG;
    if ((group != 32 && group != 64 && group != 128) || h_in % group) return LORA_ERR_SHAPE;
    if (h_in > kMaxSize || h_out > kMaxSize) return LORA_ERR_SHAPE;
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
    const int sms = num_sms();
    if (sms < 1) return LORA_ERR_CUDA;
    constexpr int kTcTokens = 64;
    for (int t = 0; t < T; t += kTcTokens) {
        p.x = static_cast<const char *>(x) + (size_t)t * h_in * e;
        p.y = static_cast<char *>(y) + (size_t)t * h_out * e;
        p.T = T - t < kTcTokens ? T - t : kTcTokens;
        const bool rows = dtype == LORA_BF16 ? takes_rows<__nv_bfloat16>(p, sms) : takes_rows<float>(p, sms);
        const int rc = !rows                  ? decode::launch_w4_tc(dtype, p, group, (cudaStream_t)stream)
                       : dtype == LORA_BF16 ? launch<__nv_bfloat16>(p, group, sms, (cudaStream_t)stream)
                                            : launch<float>(p, group, sms, (cudaStream_t)stream);
        if (rc) return rc;
    }
    return LORA_OK;
}
