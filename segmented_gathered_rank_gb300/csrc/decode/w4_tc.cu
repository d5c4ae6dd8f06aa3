// Products with 4-bit weights for more than a few tokens, on the tensor cores (tcgen05).
//
// At 64 tokens the flops (128 a weight) need more than the warp-MMA rate while the
// codes still come at half a byte a weight.  A thread block has 128 rows of W:
//   one warp     copies code tiles (128 rows x 256 columns) by tensor copies;
//   twelve warps turn codes less zeros into bf16 (exact) in tensor memory, the A
//                operand (through shared memory its 32 KB a tile, written and read
//                again, bound an earlier form: 47 against 36 us at 64 x 4096 -> 16384);
//   x            is the B operand in shared memory: bf16 by tensor copies, whose order the
//                codes follow (through registers, in the codes' order, four warps were
//                what bound the kernel: 20.6 against 17.5 us); fp32 as three bf16 parts,
//                multiplied one after another, that four warps make;
//   one thread   issues the MMAs, one accumulator in tensor memory a group of columns;
//   four warps   scale each group's accumulator and add it up in fp32, a thread a row.
// When the rows give too few blocks the columns are split over a cluster, whose
// blocks each add up a share of the tokens, in rank order.
//
// 64 x 4096 -> 16384: 17.5 us (4.5 of them to start and end), 2.2 TB/s, 490 TFLOP/s.  128
// rows a block make 128 blocks.  What bounds them is the integer pipe, 78 % busy there,
// mostly with the shifts, byte moves and masks of the codes; a fourth warpgroup for
// those, and a second one that scales, changed nothing (17.0 against 17.0 us with 32
// tokens, 18.5 against 17.5 with 64).
#include <cudaTypedefs.h>

#include <atomic>

#include "tc_common.cuh"
#include "w4.cuh"

namespace lora {
namespace {

using namespace decode;
using namespace tc;

constexpr int kRows = 128, kCols = 128;          // of W, a tile
constexpr int kThreads = 24 * 32, kTurns = 3;
constexpr int kScaleWarp0 = 4 * kTurns, kXWarp0 = kScaleWarp0 + 4, kCopyWarp = kXWarp0 + 4, kMmaWarp = kCopyWarp + 1;      // warpgroups of one kind
constexpr int kCodeBytes = kRows * kCols, kACols = kCols / 2;      // codes of two tiles; tensor memory columns of an A tile
constexpr uint32_t kTmemCols = 512;
constexpr int kAccumulators = 4, kStages = 4, kACol0 = 256;      // kStages: A tiles

template <typename E, int NTOK>
struct W4Shape {
    static constexpr int kParts = sizeof(E) == 2 ? 1 : 3;
    static constexpr int kBPart = NTOK * kCols * 2;
    static constexpr int kStage = kParts * kBPart;
    static constexpr int kX = kParts > 1 ? 3 : kStages;      // tiles of x
    static constexpr int kCodes = kParts == 1 ? 8 : 4;
    static constexpr size_t kSmem = 1024 + (size_t)kX * kStage + (size_t)kCodes * kCodeBytes;
};

struct W4Control {
    uint64_t codes_full[8], codes_free[8], a_full[kStages], done[kStages], x_full[kStages], x_free[kStages], d_full[kAccumulators], d_free[kAccumulators], drain;
    volatile int abort;
    uint32_t tmem;
};

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, W4Control &ctl) {
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    if (wait_phase(bar, parity, &ctl.abort)) return true;
    ctl.abort = 1;
    return false;
}
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, W4Control &ctl) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, ctl));
}
// A place in a ring of N and its parity.
template <int N>
struct Ring {
    int at = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++at == N) {
            at = 0;
            parity ^= 1;
        }
    }
};

// Byte offset of 16-byte chunk `chunk` (0..15) of row `row` in a tile of `rows` x 128 bf16 (128-byte swizzling).
__device__ __forceinline__ uint32_t tile_off(int rows, int row, int chunk) {
    return (uint32_t)((chunk >> 3) * (rows * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}
// D[tmem] (+)= A[tmem] . B[smem]^T, A as bf16 pairs in columns; b_lo: the lower half of
// B's descriptor (128-byte swizzling, K-major), whose upper half is constant.
template <uint32_t IDESC>
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t accumulate) {
    constexpr uint32_t kSwizzled = (1024u >> 4) | (1u << 14) | (2u << 29);
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        ".reg .b64 b;\n"
        "setp.ne.b32 p, %5, 0;\n"
        "mov.b64 b, {%2, %3};\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n"
        "}\n" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "n"(kSwizzled), "n"(IDESC), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr)
        : "memory");
}
// Two fp32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n.reg .b64 a, b, c, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\n"
        "fma.rn.f32x2 d, a, b, c;\nmov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

template <typename E, int GROUP, int NTOK>
__global__ void __launch_bounds__(kThreads, 1) w4_tc_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap x_map, const W4Params p,
                                                            int splits) {
    using Sh = W4Shape<E, NTOK>;
    constexpr int kGroups = kCols / GROUP;               // a tile
    constexpr bool kCopiesX = Sh::kParts == 1;           // x needs no splitting: tensor copies
    // One commit a tile says that its A and x stages are free, and, with one group a tile, that its sums are there.
    constexpr bool kOneX = Sh::kX == kStages, kOneD = kGroups == 1;
    extern __shared__ uint8_t raw[];
    __shared__ W4Control ctl;
    uint8_t *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint8_t *codes = smem + Sh::kX * Sh::kStage;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % splits, n0 = (blockIdx.x / splits) * kRows;
    const int tiles = (p.h_in + kCols - 1) / kCols;
    const int pairs = (tiles + 1) / 2;                   // of tiles, whose codes are copied together
    const int first = 2 * (pairs * rank / splits), end = min(tiles, 2 * (pairs * (rank + 1) / splits));

    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::kCodes; ++i) {
            mbar_init(&ctl.codes_full[i], 1);
            mbar_init(&ctl.codes_free[i], 8);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&ctl.a_full[i], 4);
            mbar_init(&ctl.done[i], 1);
        }
        for (int i = 0; i < Sh::kX; ++i) {
            mbar_init(&ctl.x_full[i], kCopiesX ? 1 : 4);
            mbar_init(&ctl.x_free[i], 1);
        }
        for (int i = 0; i < kAccumulators; ++i) {
            mbar_init(&ctl.d_full[i], 1);
            mbar_init(&ctl.d_free[i], 4);
        }
        mbar_init(&ctl.drain, 1);
        ctl.abort = 0;
        mbar_fence_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&ctl.tmem, kTmemCols);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();

    E *y = static_cast<E *>(p.y);
    auto store = [](E *dst, float v) {
        if constexpr (sizeof(E) == 2) *dst = __float2bfloat16_rn(v);
        else *dst = v;
    };
    // registers: six warpgroups start with 80 a thread; 3 x 80 + 136 + 64 + 40 is the same sum
    if (warp < kScaleWarp0) {
        // the codes of a row of the tile a thread; the warpgroups take turns (and have a stage each), so
        // that one's waits lie under the others' work
        const int row = threadIdx.x & 127;
        const long long n = min(n0 + row, p.h_out - 1);
        const uint8_t *zeros = p.zeros ? p.zeros + n * p.groups : nullptr;
        const uint32_t a_tmem = ctl.tmem + ((uint32_t)((warp & 3) * 32) << 16) + kACol0;
        uint32_t zero[kGroups], next[kGroups];
        auto fetch = [&](int tile, uint32_t (&z)[kGroups]) {
#pragma unroll
            for (int i = 0; i < kGroups; ++i) z[i] = zeros ? __ldg(zeros + min(tile * kGroups + i, p.groups - 1)) : 8u;
        };
        const int turn = warp >> 2;
        fetch(first + turn, zero);
        for (int rel = turn; first + rel < end; rel += kTurns) {
            fetch(first + rel + kTurns, next);
            const int slot = (rel >> 1) % Sh::kCodes;
            if (!wait_warp(&ctl.codes_full[slot], (rel >> 1) / Sh::kCodes & 1, ctl)) break;
            const uint8_t *src = codes + slot * kCodeBytes + row * 128;
            uint4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)      // tensor copies with 128-byte swizzling: 16-byte chunks XORed with the row
                w[i] = *reinterpret_cast<const uint4 *>(src + ((((rel & 1) * 4 + i) ^ (row & 7)) << 4));
            bool ok = true;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t a[32];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int q = h * 2 + i;               // 32 columns
                    const __nv_bfloat162 offset = code_offset(zero[q * kGroups / 4]);
                    const uint32_t words[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t o[4];
                        if constexpr (kCopiesX) code_neighbours(words[j], offset, o);
                        else code_pairs(words[j], offset, o);
#pragma unroll
                        for (int e = 0; e < 4; ++e) a[(i * 4 + j) * 4 + e] = o[e];
                    }
                }
                if (h == 0) {
                    if (!(ok = wait_warp(&ctl.done[rel % kStages], (rel / kStages & 1) ^ 1, ctl))) break;
                    fence_after_sync();        // the products that read the stage come before these stores
                }
                tmem_st32(a_tmem + rel % kStages * kACols + h * 32, a);
            }
            if (!ok) break;
            asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
            fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&ctl.a_full[rel % kStages]);
                // The slot is given back here and not after the loads above: what the codes became is in tensor
                // memory, so the loads are complete.  Right after them the next copy overtook some of them.
                mbar_arrive(&ctl.codes_free[slot]);
            }
#pragma unroll
            for (int i = 0; i < kGroups; ++i) zero[i] = next[i];
        }
    } else if (warp < kXWarp0) {
        // this thread's row: each group's sums, scaled
        asm volatile("setmaxnreg.inc.sync.aligned.u32 136;\n");
        float2 acc[NTOK / 2];
#pragma unroll
        for (int t = 0; t < NTOK / 2; ++t) acc[t] = make_float2(0.f, 0.f);
        const int row = (warp - kScaleWarp0) * 32 + lane;
        const __nv_bfloat16 *scales = p.scales + (long long)min(n0 + row, p.h_out - 1) * p.groups;
        const uint32_t quad = (uint32_t)((warp - kScaleWarp0) * 32) << 16;
        const int g0 = first * kGroups, g1 = end * kGroups;        // past p.groups: columns past h_in, zeros
        float scale[kAccumulators];
#pragma unroll
        for (int i = 0; i < kAccumulators; ++i) scale[i] = __bfloat162float(scales[min(g0 + i, p.groups - 1)]);
        uint32_t parity = 0;
        bool ok = true;
        for (int g = g0; ok && g < g1; g += kAccumulators, parity ^= 1) {
            float after[kAccumulators];
#pragma unroll
            for (int i = 0; i < kAccumulators; ++i)
                after[i] = __bfloat162float(scales[min(g + kAccumulators + i, p.groups - 1)]);
#pragma unroll
            for (int i = 0; i < kAccumulators; ++i) {
                if (g + i >= g1) break;
                if (!(ok = wait_warp(kOneD ? &ctl.done[i] : &ctl.d_full[i], parity, ctl))) break;
                fence_after_sync();
                constexpr int kPart = NTOK < 32 ? NTOK : 32;
#pragma unroll
                for (int b = 0; b < NTOK / kPart; ++b) {
                    float d[kPart];
                    if constexpr (kPart == 32) tmem_ld32(ctl.tmem + quad + i * NTOK + b * 32, d);
                    else tmem_ld16(ctl.tmem + quad + i * NTOK, d);
#pragma unroll
                    for (int t = 0; t < kPart / 2; ++t)
                        acc[b * 16 + t] = fma2(make_float2(scale[i], scale[i]), make_float2(d[2 * t], d[2 * t + 1]), acc[b * 16 + t]);
                }
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.d_free[i]);
            }
#pragma unroll
            for (int i = 0; i < kAccumulators; ++i) scale[i] = after[i];
        }
        const float lost = ctl.abort ? __uint_as_float(0x7fffffffu) : 0.f;       // a wait gave up: no numbers rather than wrong ones
        if (splits == 1) {
            if (n0 + row < p.h_out) {
                E *dst = y + n0 + row;
#pragma unroll
                for (int t = 0; t < NTOK; ++t, dst += p.h_out)
                    if (t < p.T) store(dst, (t & 1 ? acc[t / 2].y : acc[t / 2].x) + lost);
            }
        } else {
            // every block's sums of token t go to block t % splits: [from][t / splits][row]
            cluster_barrier();                 // all of the cluster's blocks are past their tiles
            const uint32_t local = smem_u32(smem) + (uint32_t)(rank * (NTOK / splits) * kRows + row) * 4;
#pragma unroll
            for (int t = 0; t < NTOK; ++t) {
                uint32_t remote;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n"
                             : "=r"(remote)
                             : "r"(local + (uint32_t)(t / splits) * kRows * 4), "r"((uint32_t)(t % splits)));
                asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(remote), "f"((t & 1 ? acc[t / 2].y : acc[t / 2].x) + lost)
                             : "memory");
            }
        }
    } else if (warp < kCopyWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
        const int tid = threadIdx.x - kXWarp0 * 32;
        // every block will want all of x at about the same time: each brings a share of it into L2
        const size_t bytes = (size_t)p.T * p.h_in * sizeof(E);
        for (size_t i = ((size_t)blockIdx.x * 128 + tid) * 128; i < bytes; i += (size_t)gridDim.x * 128 * 128)
            asm volatile("prefetch.global.L2 [%0];\n" ::"l"(static_cast<const char *>(p.x) + i));
        if constexpr (kCopiesX) {
            // two panels of 64 columns a tile; what lies outside of x reads as zeros
            if (warp == kXWarp0 && elect_lane()) {
                Ring<Sh::kX> r;
                for (int tile = first; tile < end; ++tile, r.next()) {
                    if (!wait_bar(&ctl.done[r.at], r.parity ^ 1, ctl)) {
                        for (int i = 0; i < Sh::kX && tile - (i + 1) >= first; ++i)      // as below, for the codes
                            wait_phase(&ctl.x_full[(r.at + Sh::kX - 1 - i) % Sh::kX], i < r.at ? r.parity : r.parity ^ 1, nullptr);
                        break;
                    }
                    mbar_arrive_expect_tx(&ctl.x_full[r.at], Sh::kStage);
#pragma unroll
                    for (int panel = 0; panel < 2; ++panel)
                        tma_load_2d(smem + r.at * Sh::kStage + panel * (NTOK * 128), &x_map, tile * kCols + panel * 64, 0, &ctl.x_full[r.at]);
                }
            }
            __syncwarp();
        } else {
            // the parts of x of the tile's columns, in the order of code_pairs; tokens past T are zeros.  Each
            // thread's next pieces are on their way while these are written.
            constexpr int kPieces = NTOK * 16 / 128, kHeld = kPieces / 2;
            const int t0 = tid >> 4, k0 = (tid & 15) * 8;          // piece i: token t0 + 8 i
            const E *src = static_cast<const E *>(p.x) + (long long)t0 * p.h_in + k0;
            const long long step = 8LL * p.h_in;
            const uint32_t place = tile_off(NTOK, t0, tid & 15);   // 8 tokens are one swizzle atom: piece i is i KB further
            const int pieces = (p.T - t0 + 7) / 8;                 // that exist
            uint4 v[kHeld][2];
            auto load = [&](int tile, int i0) {
                const E *at = src + tile * kCols;
                const int n = tile * kCols + k0 < p.h_in ? pieces - i0 : 0;
#pragma unroll
                for (int i = 0; i < kHeld; ++i) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        v[i][h] = i < n ? __ldg(reinterpret_cast<const uint4 *>(at + (i0 + i) * step) + h) : make_uint4(0, 0, 0, 0);
                }
            };
            Ring<Sh::kX> xr;
            load(first, 0);
            for (int tile = first; tile < end; ++tile, xr.next()) {
                if (!wait_warp(&ctl.x_free[xr.at], xr.parity ^ 1, ctl)) break;
                uint8_t *b = smem + xr.at * Sh::kStage;
#pragma unroll
                for (int i0 = 0; i0 < kPieces; i0 += kHeld) {
#pragma unroll
                    for (int i = 0; i < kHeld; ++i) {
                        const uint32_t at = place + (i0 + i) * 1024;
                        const float f[8] = {__uint_as_float(v[i][0].x), __uint_as_float(v[i][0].y), __uint_as_float(v[i][0].z),
                                            __uint_as_float(v[i][0].w), __uint_as_float(v[i][1].x), __uint_as_float(v[i][1].y),
                                            __uint_as_float(v[i][1].z), __uint_as_float(v[i][1].w)};
                        uint32_t o[3][4];
                        split_x(f, o[0], o[1], o[2]);
#pragma unroll
                        for (int q = 0; q < 3; ++q)
                            *reinterpret_cast<uint4 *>(b + q * Sh::kBPart + at) = make_uint4(o[q][0], o[q][1], o[q][2], o[q][3]);
                    }
                    if (i0 + kHeld < kPieces) load(tile, i0 + kHeld);
                    else if (tile + 1 < end) load(tile + 1, 0);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.x_full[xr.at]);
            }
        }
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 40;\n");
      if (warp == kCopyWarp) {
        if (elect_lane()) {
            // codes are read once a call: they leave L2 first
            uint64_t policy;
            asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;\n" : "=l"(policy));
            Ring<Sh::kCodes> c;
            for (int tile = first; tile < end; tile += 2, c.next()) {
                if (!wait_bar(&ctl.codes_free[c.at], c.parity ^ 1, ctl)) {
                    // the copies on their way land before the block leaves: the ring's last uses
                    for (int i = 0; i < Sh::kCodes && tile - 2 * (i + 1) >= first; ++i)
                        wait_phase(&ctl.codes_full[(c.at + Sh::kCodes - 1 - i) % Sh::kCodes], i < c.at ? c.parity : c.parity ^ 1, nullptr);
                    break;
                }
                mbar_arrive_expect_tx(&ctl.codes_full[c.at], kCodeBytes);
                asm volatile(
                    "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
                    "[%0], [%1, {%2, %3}], [%4], %5;\n" ::"r"(smem_u32(codes + c.at * kCodeBytes)),
                    "l"(&map), "r"(tile * (kCols / 2)), "r"(n0), "r"(smem_u32(&ctl.codes_full[c.at])), "l"(policy)
                    : "memory");
            }
        }
        __syncwarp();
      } else if (warp == kMmaWarp) {
        if (elect_lane()) {
            constexpr uint32_t idesc = idesc_bf16_f32(kRows, NTOK);
            const uint32_t b0 = (uint32_t)desc_kmajor_sw128(smem_u32(smem)), tmem = ctl.tmem;
            Ring<kStages> ar;
            Ring<Sh::kX> xr;
            Ring<kAccumulators> d;
            for (int tile = first; tile < end; ++tile, ar.next(), xr.next()) {
                // asked for together, as each answer takes longer than the products of a few columns
                const bool ready = mbar_try_wait(&ctl.x_full[xr.at], xr.parity) & mbar_try_wait(&ctl.a_full[ar.at], ar.parity) &
                                   mbar_try_wait(&ctl.d_free[d.at], d.parity ^ 1);
                if (!ready && !(wait_bar(&ctl.x_full[xr.at], xr.parity, ctl) && wait_bar(&ctl.a_full[ar.at], ar.parity, ctl) &&
                                wait_bar(&ctl.d_free[d.at], d.parity ^ 1, ctl)))
                    break;
                fence_after_sync();
                const uint32_t a = tmem + kACol0 + ar.at * kACols, b = b0 + xr.at * (Sh::kStage / 16);
                bool ok = true;
#pragma unroll
                for (int g = 0; g < kGroups; ++g, d.next()) {
                    if (g > 0) {
                        if (!(ok = wait_bar(&ctl.d_free[d.at], d.parity ^ 1, ctl))) break;
                        fence_after_sync();
                    }
#pragma unroll
                    for (int q = Sh::kParts - 1; q >= 0; --q)      // the smallest part first
#pragma unroll
                        for (int ks = g * (8 / kGroups); ks < (g + 1) * (8 / kGroups); ++ks)
                            mma_ts<idesc>(tmem + d.at * NTOK, a + ks * 8,
                                          b + (q * Sh::kBPart + (ks >> 2) * (NTOK * 128) + (ks & 3) * 32) / 16,
                                          q < Sh::kParts - 1 || ks > g * (8 / kGroups));
                    if (!kOneD) mma_commit(&ctl.d_full[d.at]);
                }
                if (!ok) break;
                mma_commit(&ctl.done[ar.at]);
                if (!kOneX) mma_commit(&ctl.x_free[xr.at]);
            }
            mma_commit(&ctl.drain);
            wait_phase(&ctl.drain, 0, nullptr);
        }
        __syncwarp();
      }
    }
    if (splits > 1 && (warp < kScaleWarp0 || warp >= kXWarp0)) cluster_barrier();      // the scaling warps' first one
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == kMmaWarp) tmem_dealloc(ctl.tmem, kTmemCols);
    if (splits > 1) {
        cluster_barrier();
        const float *in = reinterpret_cast<const float *>(smem);
        for (int x = threadIdx.x; x < NTOK / splits * kRows; x += kThreads) {
            const int t = x / kRows, r = x % kRows;
            float s = 0.f;
            for (int from = 0; from < splits; ++from) s += in[(from * (NTOK / splits) + t) * kRows + r];
            const int token = t * splits + rank;
            if (token < p.T && n0 + r < p.h_out) store(y + (long long)token * p.h_out + n0 + r, s);
        }
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            ptr = nullptr;
        }
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

// A matrix of `rows` rows of `cols` elements in boxes of 128 bytes x box_rows; what lies outside reads as zeros.
bool make_map(CUtensorMap *map, CUtensorMapDataType type, void *base, int cols, int rows, cuuint64_t pitch, int box_cols,
              int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {pitch};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, step[2] = {1, 1};
    return encode_fn()(map, type, 2, base, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaLaunchAttribute cluster_of(int blocks) {
    cudaLaunchAttribute a;
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = blocks;
    a.val.clusterDim.y = 1;
    a.val.clusterDim.z = 1;
    return a;
}

// Clusters of 2^log2 blocks (1 to 3) that run at once on the current device, asked for once
// a device: every form of the kernel has one block an SM.  The SMs that can share a
// cluster come in groups that are no multiples of eight, so there are 76, 36 and 15 here.
int clusters_at_once(const void *func, size_t smem, int log2) {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices][4];          // plus one; 0: not asked yet
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) dev = -1;
    if (dev >= 0 && known[dev][log2].load(std::memory_order_relaxed)) return known[dev][log2].load(std::memory_order_relaxed) - 1;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = cluster_of(1 << log2);
    cfg.gridDim = dim3(1 << log2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, func, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (dev >= 0) known[dev][log2].store(n + 1, std::memory_order_relaxed);
    return n;
}

template <typename E, int GROUP, int NTOK>
int launch(const W4Params &p, const CUtensorMap &map, const CUtensorMap &x_map, cudaStream_t st) {
    using Sh = W4Shape<E, NTOK>;
    const int rows = (p.h_out + kRows - 1) / kRows, tiles = (p.h_in + kCols - 1) / kCols;
    const void *func = reinterpret_cast<const void *>(w4_tc_kernel<E, GROUP, NTOK>);
    if (smem_optin(func, Sh::kSmem)) return LORA_ERR_CUDA;
    // Blocks that share the columns: as many as let all clusters run at once, with two tiles
    // of columns each.  Against one block: 16 x 4096 -> 4096 8.4 for 15.4 us, 64 x 16384 ->
    // 4096 20.8 for 53.6.  Clusters that wait for others cost more than smaller ones: 16 x
    // 4096 -> 2048 (16 row blocks) 8.3 us in fours for 12.0 in eights, 64 x 4096 -> 4736 (37)
    // 13.8 in twos for 18.3 in fours; up to the limit, 16 x 4096 -> 1920 (15) 7.0 in eights
    // for 8.3 in fours, 64 x 4096 -> 4608 (36) 11.0 in fours for 13.7 in twos.
    int log2 = 0;
    while (log2 < 3 && tiles >= 4 << log2 && rows <= clusters_at_once(func, Sh::kSmem, log2 + 1)) ++log2;
    const int splits = 1 << log2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * splits));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Sh::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr = cluster_of(splits);
    cfg.attrs = &attr;
    cfg.numAttrs = splits > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, w4_tc_kernel<E, GROUP, NTOK>, map, x_map, p, splits);
    count_launch();
    return cuda_status(e);
}

template <typename E, int NTOK>
int launch(const W4Params &p, int group, const CUtensorMap &map, cudaStream_t st) {
    CUtensorMap x_map = {};
    if (W4Shape<E, NTOK>::kParts == 1 &&
        !make_map(&x_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, const_cast<void *>(p.x), p.h_in, p.T, (cuuint64_t)p.h_in * 2, 64, NTOK))
        return LORA_ERR_CUDA;
    if (group == 128) return launch<E, 128, NTOK>(p, map, x_map, st);
    return group == 64 ? launch<E, 64, NTOK>(p, map, x_map, st) : launch<E, 32, NTOK>(p, map, x_map, st);
}

}  // namespace

namespace decode {

int launch_w4_tc(int dtype, const W4Params &p, int group, cudaStream_t st) {
    if (!encode_fn()) return LORA_ERR_CUDA;
    CUtensorMap map;        // codes as bytes [h_out][h_in / 2]
    if (!make_map(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<uint8_t *>(p.codes), p.h_in / 2, p.h_out, p.h_in / 2, kCols, kRows))
        return LORA_ERR_CUDA;
    // Few tokens take the narrow tile of x: half the shared memory traffic, products and
    // scaling.  32 x 4096 -> 16384: 17.2 us with 32 columns for 17.7 with 64, in fp32 33.1 for
    // 50.0; 12 x 4096 -> 16384: 16.6 us with 16 columns for 17.0 with 32, groups of 32 34.5 for
    // 37.3, in fp32 27.2 for 31.7.
    if (dtype == LORA_BF16)
        return p.T <= 16 ? launch<__nv_bfloat16, 16>(p, group, map, st) : p.T <= 32 ? launch<__nv_bfloat16, 32>(p, group, map, st) : launch<__nv_bfloat16, 64>(p, group, map, st);
    return p.T <= 16 ? launch<float, 16>(p, group, map, st) : p.T <= 32 ? launch<float, 32>(p, group, map, st) : launch<float, 64>(p, group, map, st);
}

}  // namespace decode
}  // namespace lora
