// Attention of drafted tokens over a paged cache (lora_tree_attention).
//
// For drafted token i of a request with prefix P = kv_len - n:
//   o = sum_c p_c v_c / sum_c p_c,  p_c = 2^(scale log2(e) q . k_c - m),  m the running maximum,
// over the visible c: every c < P, and drafted j (c = P + j) that the token's
// mask row names (or j <= i without a mask).  K and V are read once, which is
// the bound while few query rows share them (2 flops a byte and row).
//
// attention_mma_kernel (bf16): warp MMAs on units of 16 rows.  Few rows share a key,
//   so memory is the bound: one producer warp keeps two to six tiles of K and V on
//   their way, four warps take a quarter of each tile's keys and add up at the unit's
//   end.  128 requests of one token over <= 8192 cached, 32 query and 8 kv heads of
//   128: 240 us, 6.64 TB/s.  One request over 777: 10.7 us, of which the bytes take
//   0.5; the rest is the chain launch -> page ids -> tile -> products -> sums in
//   memory -> join.
// attention_tc_kernel (bf16, attention_tc.cu): tcgen05 on units of 128 or 256 rows.
// attention_few_kernel, attention_simt_kernel (fp32): the same list, fp32
//   multiply-adds.  Few rows: memory, as long as it comes in time (39 requests of one
//   token over <= 6697, 4 heads of 112: 89 us, 4.4 TB/s).  More: instructions (4 trees
//   of 22 over <= 13071, 28 query and 4 kv heads of 128: 362 us, 16.1 TFLOP/s), and for
//   short contexts the chain above (5 requests of up to 7 tokens over <= 300: 13.5 us).
// attention_join_kernel: joins the units that were cut between blocks.  It is
//   launched while the attention still runs, and waits for it.
//
// Probabilities are rounded to bf16 for their product with V, as the tensor cores
// take them (2^-9 relative each, no more than V's own rounding); maximum, sum and
// output stay in fp32.  The error of a bf16 output, root mean square, is then 0.0018 to
// 0.0023 of the outputs' size (long contexts most), of which storing them in bf16 makes
// 0.00165.  A second bf16 part of each probability would take that away, but a part that
// is zero would make NaN of an infinite value (p v is infinite), and large trees, bound by
// their products, would have half as many again.  fp32 caches are not rounded anywhere.
#include <cudaTypedefs.h>

#include <type_traits>

#include "kv_copy.cuh"

namespace lora {
namespace {

using namespace decode;

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 mul_add2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n.reg .b64 a, b, c, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\n"
        "fma.rn.f32x2 d, a, b, c;\nmov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

constexpr int kThreads = 128;      // the join kernel's, the fp32 kernel's, the consumers of the MMA kernel
constexpr int kJoinThreads = 256, kJoinRows = 8;
constexpr int kRows = 16;          // query rows a unit

// This thread's writes to a stage come before the copies that fill it next.
__device__ __forceinline__ void fence_own_writes() { tc::fence_proxy_async(); }

// D: head width padded to 64, 128 or 256.
template <int D, bool TMA>
struct MmaShape {
    static constexpr int kTile = D == 64 ? 128 : 64;       // cached tokens a stage
    static constexpr int kWarpKeys = kTile / 4;
    static constexpr int kHalf = kTile * D * 2;            // K, then V
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kPerSm = TMA && D <= 128 ? 2 : 1;
    static constexpr int kStages = D <= 128 && !TMA ? 6 : 3;
    static constexpr int kThreadsAll = kThreads + (TMA ? 32 : 128);
    static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
};

struct MmaControl {
    uint64_t full[6], empty[6], join;
    volatile int abort;
    float row_max[4][16], row_sum[4][16];
};

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, MmaControl &ctl) {
    for (int i = 0; i < 64; ++i)
        if (tc::mbar_try_wait(bar, parity)) return true;
    if (tc::wait_phase(bar, parity, &ctl.abort)) return true;
    ctl.abort = 1;
    return false;
}
// wait_bar for a whole warp: all lanes go on, or none.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, MmaControl &ctl) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, ctl));
}

// Four consumer warps; each takes kWarpKeys of a stage's tokens for all rows of
// the unit, with a maximum, sum and output of its own (so a tile needs no exchange
// between warps), joined in shared memory when the block leaves the unit.
template <int D, bool TMA>
__device__ void consume(const AttnParams &p, Cursor cur, uint32_t total, uint8_t *smem, MmaControl &ctl) {
    using Sh = MmaShape<D, TMA>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g4 = lane >> 2, t4 = lane & 3, mi = lane >> 3, r8 = lane & 7;
    const uint32_t base = smem_addr(smem);
    const int key0 = warp * Sh::kWarpKeys;
    uint32_t qf[D / 16][4], join_phase = 0;
    float o[D / 8][4], m[2], l[2];
    int start_tile = cur.tile;
    // a new unit: its queries, straight into MMA fragments, and nothing seen yet
    auto load_queries = [&](const Cursor &c) {
        const int rows = min(kRows, c.r.n * p.group - c.row_tile * kRows);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int row = hh * 8 + g4;
            const __nv_bfloat16 *src =
                static_cast<const __nv_bfloat16 *>(p.q) + (row < rows ? row_offset(p, c, c.row_tile * kRows + row) : 0);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    const int col = ks * 16 + kk * 8 + t4 * 2;
                    qf[ks][kk * 2 + hh] = row < rows && col < p.d ? *reinterpret_cast<const uint32_t *>(src + col) : 0u;
                }
        }
    };
    auto clear = [&]() {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            m[hh] = -INFINITY;
            l[hh] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    };
    load_queries(cur);
    clear();
    auto all_warps = [&]() {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl.join);
        return wait_warp(&ctl.join, join_phase++ & 1, ctl);
    };
    for (int it = 0; cur.left > 0; ++it) {
        const int stage = it % Sh::kStages;
        uint8_t *vs = smem + stage * Sh::kStage + Sh::kHalf;
        const uint32_t ks_base = base + stage * Sh::kStage, vs_base = ks_base + Sh::kHalf;
        const int rows = min(kRows, cur.r.n * p.group - cur.row_tile * kRows);
        if (!wait_warp(&ctl.full[stage], (it / Sh::kStages) & 1, ctl)) return;
        const int c0 = cur.tile * Sh::kTile + key0;         // first cached token of this warp's keys
        const int drafted = cur.r.len - cur.r.n - c0;       // the first of them that a mask rules

        if (c0 < cur.r.len) {
            float s[Sh::kWarpKeys / 8][4];
#pragma unroll
            for (int j = 0; j < Sh::kWarpKeys / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                if (ks * 16 >= p.d) break;
#pragma unroll
                for (int kg = 0; kg < Sh::kWarpKeys / 16; ++kg) {
                    uint32_t b[4];
                    ldm4(b, ks_base + panel_off(Sh::kTile, key0 + kg * 16 + (mi >> 1) * 8 + r8, ks * 2 + (mi & 1)));
                    mma16816(s[kg * 2], qf[ks], b[0], b[1]);
                    mma16816(s[kg * 2 + 1], qf[ks], b[2], b[3]);
                }
            }
            uint32_t see[2] = {0u, 0u};       // bit x: row hh * 8 + g4 sees the warp's token x
            if (drafted < Sh::kWarpKeys) {
                // scores that are not visible leave the softmax here, whatever they hold
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
                    if (hh * 8 + g4 < rows) see[hh] = seen_word(p, cur.r, (cur.row_tile * kRows + hh * 8 + g4) / p.group, c0);
#pragma unroll
                for (int j = 0; j < Sh::kWarpKeys / 8; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!((see[e >> 1] >> (j * 8 + t4 * 2 + (e & 1))) & 1)) s[j][e] = -INFINITY;
            }
            // softmax of the warp's keys
            float a[2];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < Sh::kWarpKeys / 8; ++j) top = fmaxf(top, fmaxf(s[j][hh * 2], s[j][hh * 2 + 1]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float m2 = fmaxf(m[hh], top * p.scale_log2);
                const float ref = m2 == -INFINITY ? 0.f : m2;        // nothing visible so far
                a[hh] = exp2_fast(m[hh] - ref);
                m[hh] = m2;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < Sh::kWarpKeys / 8; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float &x = s[j][hh * 2 + e];
                        x = exp2_fast(fmaf(x, p.scale_log2, -ref));
                        sum += x;
                    }
                l[hh] = l[hh] * a[hh] + sum;      // this thread's columns only, joined at the end
            }
            if (__any_sync(0xffffffffu, a[0] != 1.f || a[1] != 1.f)) {
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    o[j][0] *= a[0];
                    o[j][1] *= a[0];
                    o[j][2] *= a[1];
                    o[j][3] *= a[1];
                }
            }
            if (drafted < Sh::kWarpKeys) {
                // values past the request, and drafted ones that are not finite, would enter the product times
                // zero: the latter are added to the rows that see them, and both leave the tile (its rows are
                // this warp's own)
                const int first = max(0, drafted), end = cur.r.len - c0;
                bool bad = false;
                for (int x = lane; x < (Sh::kWarpKeys - first) * (D / 8); x += 32) {
                    const int key = first + x / (D / 8), ch = x % (D / 8);
                    uint4 *at = reinterpret_cast<uint4 *>(vs + panel_off(Sh::kTile, key0 + key, ch));
                    const uint4 u = *at;
                    if (key >= end) *at = make_uint4(0, 0, 0, 0);
                    else bad |= ch * 8 < p.d && (non_finite2(u.x) || non_finite2(u.y) || non_finite2(u.z) || non_finite2(u.w));
                }
                __syncwarp();
                if (__any_sync(0xffffffffu, bad)) {
                    for (int x = first; x < min(end, Sh::kWarpKeys); ++x)
#pragma unroll
                        for (int j = 0; j < D / 8; ++j) {
                            if (j * 8 >= p.d) break;
                            const uint32_t w = *reinterpret_cast<const uint32_t *>(vs + panel_off(Sh::kTile, key0 + x, j) + t4 * 4);
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t bits = e ? w & 0xffff0000u : w << 16;
                                if ((bits & 0x7f800000u) != 0x7f800000u) continue;
#pragma unroll
                                for (int hh = 0; hh < 2; ++hh)
                                    if ((see[hh] >> x) & 1) o[j][hh * 2 + e] += __uint_as_float(bits);
                            }
                        }
                    __syncwarp();
                    for (int x = lane; x < (Sh::kWarpKeys - first) * (D / 8); x += 32)
                        make_finite(reinterpret_cast<uint4 *>(vs + panel_off(Sh::kTile, key0 + first + x / (D / 8), x % (D / 8))));
                    __syncwarp();
                }
                fence_own_writes();
            }
#pragma unroll
            for (int kg = 0; kg < Sh::kWarpKeys / 16; ++kg) {
                const uint32_t pf[4] = {pack_bf16(s[kg * 2][0], s[kg * 2][1]), pack_bf16(s[kg * 2][2], s[kg * 2][3]),
                                        pack_bf16(s[kg * 2 + 1][0], s[kg * 2 + 1][1]),
                                        pack_bf16(s[kg * 2 + 1][2], s[kg * 2 + 1][3])};
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    if (j * 16 >= p.d) break;
                    uint32_t b[4];
                    ldm4t(b, vs_base + panel_off(Sh::kTile, key0 + kg * 16 + (mi & 1) * 8 + r8, j * 2 + (mi >> 1)));
                    mma16816(o[j * 2], pf, b[0], b[1]);
                    mma16816(o[j * 2 + 1], pf, b[2], b[3]);
                }
            }
        }

        const bool unit_ends = cur.tile + 1 == cur.r.tiles;
        if (unit_ends || cur.left == 1) {
            // join the four warps through the stage just used
            const bool whole = unit_ends && start_tile == 0;
            float *dst = partial_of(p, blockIdx.x, start_tile > 0 ? 0 : 1);
            float *scratch = reinterpret_cast<float *>(smem + stage * Sh::kStage);     // [4][16][D]
            Cursor after = cur;
            after.advance(p, 1);
            if (after.left > 0) load_queries(after);      // on their way while this unit is joined
            if (!all_warps()) return;
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int row = hh * 8 + g4;
                float sum = l[hh];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                if (t4 == 0) {
                    ctl.row_max[warp][row] = m[hh];
                    ctl.row_sum[warp][row] = sum;
                }
                if (row < rows) {
#pragma unroll
                    for (int j = 0; j < D / 8; ++j)
                        *reinterpret_cast<float2 *>(scratch + (warp * 16 + row) * D + ((j ^ g4) * 8 + t4 * 2)) =
                            make_float2(o[j][hh * 2], o[j][hh * 2 + 1]);
                }
            }
            if (!all_warps()) return;
            const int shift = rows <= 4 ? 2 : rows <= 8 ? 3 : 4;
            for (int x = tid; x < (D / 4) << shift; x += kThreads) {
                const int row = x & ((1 << shift) - 1), col = (x >> shift) * 4;
                if (row >= rows || col >= p.d) continue;
                float top = ctl.row_max[0][row];
#pragma unroll
                for (int w = 1; w < 4; ++w) top = fmaxf(top, ctl.row_max[w][row]);
                const float ref = top == -INFINITY ? 0.f : top;
                float sum = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float share = exp2_fast(ctl.row_max[w][row] - ref);
                    const float4 u = *reinterpret_cast<const float4 *>(scratch + (w * 16 + row) * D + (col ^ ((row & 7) * 8)));
                    sum += share * ctl.row_sum[w][row];
                    acc.x += share * u.x;
                    acc.y += share * u.y;
                    acc.z += share * u.z;
                    acc.w += share * u.w;
                }
                if (whole) {
                    const float r = sum == 0.f ? 0.f : 1.f / sum;      // a row that saw nothing: zeros
                    uint2 w2;
                    w2.x = pack_bf16(acc.x * r, acc.y * r);
                    w2.y = pack_bf16(acc.z * r, acc.w * r);
                    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) +
                                               row_offset(p, cur, cur.row_tile * kRows + row) + col) = w2;
                } else {
                    *reinterpret_cast<float4 *>(dst + partial_at(p, row, col)) = acc;
                    if (col == 0) {
                        dst[kRows * p.d + row * 2] = top;
                        dst[kRows * p.d + row * 2 + 1] = sum;
                    }
                }
            }
            if (tid == 0 && start_tile == 0 && !unit_ends) record_unit(p, cur, cur.tile, total);
            fence_own_writes();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ctl.empty[stage]);
            clear();
            cur = after;
            start_tile = cur.tile;
            continue;
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl.empty[stage]);
        cur.advance(p, 1);
    }
}

template <int D, bool TMA>
__global__ void __launch_bounds__((MmaShape<D, TMA>::kThreadsAll), (MmaShape<D, TMA>::kPerSm))
    attention_mma_kernel(const __grid_constant__ KvMaps maps, const AttnParams p) {
    using Sh = MmaShape<D, TMA>;
    using Copy = std::conditional_t<TMA, TmaCopy<D, Sh::kTile>, ChunkCopy<D, Sh::kTile, 128>>;
    extern __shared__ uint8_t raw[];
    __shared__ ScanShared scan;
    __shared__ MmaControl ctl;
    uint8_t *smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::kStages; ++i) {
            tc::mbar_init(&ctl.full[i], 2 * Copy::kArrivals);       // K, then V
            tc::mbar_init(&ctl.empty[i], 4);
        }
        tc::mbar_init(&ctl.join, 4);
        ctl.abort = 0;
        tc::mbar_fence_init();
    }
    Cursor cur;
    const uint32_t total = start_block(p, scan, cur);
    if (cur.left <= 0) return;
    if (threadIdx.x < kThreads) {
        consume<D, TMA>(p, cur, total, smem, ctl);
    } else {
        const int tid = threadIdx.x - kThreads;
        const uint32_t base = smem_addr(smem);
        Copy copy;
        copy.fetch(p, cur, cur.tile, tid);
        for (int it = 0; cur.left > 0; ++it) {
            const int stage = it % Sh::kStages;
            if (!wait_warp(&ctl.empty[stage], ((it / Sh::kStages) & 1) ^ 1, ctl)) {
                // tensor copies on their way land before the block leaves
                for (int x = max(0, it - Sh::kStages); TMA && x < it; ++x)
                    tc::wait_phase(&ctl.full[x % Sh::kStages], (x / Sh::kStages) & 1, nullptr);
                break;
            }
            for (int which = 0; which < 2; ++which) {
                copy.copy(p, which ? &maps.v : &maps.k, which ? p.v : p.k, base + stage * Sh::kStage + which * Sh::kHalf,
                          &ctl.full[stage], tid);
                if (!TMA) cp_arrive(&ctl.full[stage]);
            }
            cur.advance(p, 1);
            if (cur.left > 0) copy.fetch(p, cur, cur.tile, tid);
        }
        if (!TMA) cp_wait_all();
    }
    __syncthreads();
    if (threadIdx.x == 0 && ctl.abort) flag_status(p.status, LORA_DEV_WAIT_TIMEOUT);
}

// fp32: four warps of four rows each, over 32 cached tokens a stage.  A lane holds one
// token's score for its warp's rows, then every 32nd output column.  Two multiply-adds
// an instruction; tiles that every row sees whole need neither masks nor a look at
// the values (both steps: 430 -> 362 us for the 4 trees above).
constexpr int kSimtTile = 32;
constexpr int kSimtRows = 16;

template <int D>
__global__ void __launch_bounds__(kThreads) attention_simt_kernel(const AttnParams p) {
    constexpr int kLd = D + 4;            // row pitch: lanes a row apart read different banks
    constexpr int kCols = D / 32;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ ScanShared scan;
    float *qs = reinterpret_cast<float *>(smem);            // [16][D]
    float *ps = qs + kSimtRows * D;                         // [4 warps][32 tokens][4 rows]
    float *ring = ps + 4 * kSimtTile * 4;                   // [2][K, V][32][kLd]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Cursor cur;
    const uint32_t total = start_block(p, scan, cur);
    if (cur.left <= 0) return;
    Cursor ahead = cur;
    // copies: this thread's 16 bytes of rows copy_row + i * kRowsPerPass, whose pages are fetched a tile ahead
    constexpr int kLanes = D / 4, kRowsPerPass = kThreads / kLanes, kPasses = kSimtTile / kRowsPerPass;
    const int chunk = tid % kLanes, copy_row = tid / kLanes, page_mask = (1 << p.page_shift) - 1;
    int pages[kPasses];
    auto fetch = [&]() {
#pragma unroll
        for (int i = 0; i < kPasses; ++i)
            pages[i] = page_of(p, ahead.s, ahead.r, ahead.tile * kSimtTile + copy_row + i * kRowsPerPass);
    };
    auto load = [&](int stage) {
        if (ahead.left > 0) {
            float *dst = ring + stage * 2 * kSimtTile * kLd + copy_row * kLd + chunk * 4;
            if (chunk * 4 < p.d) {
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const int c = ahead.tile * kSimtTile + copy_row + i * kRowsPerPass;
                    const bool real = c < ahead.r.len;
                    const int row = real ? ((checked_page(p, pages[i]) * p.n_kv + ahead.head) << p.page_shift) + (c & page_mask) : 0;
                    const long long off = (long long)row * p.d + chunk * 4;
                    cp_async16(smem_addr(dst + i * kRowsPerPass * kLd), static_cast<const float *>(p.k) + off, real);
                    cp_async16(smem_addr(dst + (kSimtTile + i * kRowsPerPass) * kLd), static_cast<const float *>(p.v) + off, real);
                }
            }
            ahead.advance(p, 1);
            if (ahead.left > 0) fetch();
        }
        cp_commit();
    };
    fetch();
    load(0);
    float2 o2[2][kCols];                  // rows in pairs
    float m[4], l[4];
    auto o = [&](int a, int j) -> float & { return a & 1 ? o2[a >> 1][j].y : o2[a >> 1][j].x; };
    bool fresh = true;
    int start_tile = cur.tile;
    for (int it = 0; cur.left > 0; ++it) {
        const int row0 = warp * 4, rows = min(p.rt, cur.r.n * p.group - cur.row_tile * p.rt);
        if (fresh) {
            fresh = false;
            start_tile = cur.tile;
            __syncthreads();
#pragma unroll
            for (int x = 0; x < kSimtRows / kRowsPerPass; ++x) {
                const int row = copy_row + x * kRowsPerPass;
                float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
                if (row < rows && chunk * 4 < p.d)
                    u = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) +
                                                          row_offset(p, cur, cur.row_tile * p.rt + row) + chunk * 4);
                *reinterpret_cast<float4 *>(qs + row * D + chunk * 4) = u;
            }
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                m[a] = -INFINITY;
                l[a] = 0.f;
#pragma unroll
                for (int j = 0; j < kCols; ++j) o(a, j) = 0.f;
            }
        }
        load((it + 1) & 1);
        cp_wait<1>();
        __syncthreads();
        const float *ks = ring + (it & 1) * 2 * kSimtTile * kLd, *vs = ks + kSimtTile * kLd;
        if (row0 < rows) {
            const bool sure = (cur.tile + 1) * kSimtTile <= cur.r.len - cur.r.n;        // every row sees the whole tile
            float2 s2[4] = {};
            for (int k = 0; k < p.d; k += 4) {
                const float4 kk = *reinterpret_cast<const float4 *>(ks + lane * kLd + k);
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const float4 qq = *reinterpret_cast<const float4 *>(qs + (row0 + a) * D + k);
                    s2[a] = mul_add2(make_float2(kk.x, kk.y), make_float2(qq.x, qq.y), s2[a]);
                    s2[a] = mul_add2(make_float2(kk.z, kk.w), make_float2(qq.z, qq.w), s2[a]);
                }
            }
            uint32_t see[4];
            float w[4];
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                see[a] = sure ? ~0u : 0u;
                if (!sure && row0 + a < rows) see[a] = seen_word(p, cur.r, (cur.row_tile * p.rt + row0 + a) / p.group, cur.tile * kSimtTile);
                const bool on = (see[a] >> lane) & 1;
                const float x = on ? (s2[a].x + s2[a].y) * p.scale_log2 : -INFINITY;
                float top = x;
#pragma unroll
                for (int b = 16; b > 0; b >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, b));
                const float m2 = fmaxf(m[a], top), ref = m2 == -INFINITY ? 0.f : m2;
                const float scale = exp2f(m[a] - ref);
                w[a] = on ? exp2f(x - ref) : 0.f;
                m[a] = m2;
                l[a] = l[a] * scale + warp_sum(w[a]);
#pragma unroll
                for (int j = 0; j < kCols; ++j) o(a, j) *= scale;
            }
            *reinterpret_cast<float4 *>(ps + (warp * kSimtTile + lane) * 4) = make_float4(w[0], w[1], w[2], w[3]);
            __syncwarp();
            // drafted values that are not finite must not meet the zero weights of rows that do not see them: they
            // count as zeros here and are added to the rows that do see them after
            bool bad = false;
            if (sure) {
#pragma unroll 4
                for (int x = 0; x < kSimtTile; ++x) {
                    const float4 pp = *reinterpret_cast<const float4 *>(ps + (warp * kSimtTile + x) * 4);
#pragma unroll
                    for (int j = 0; j < kCols; ++j) {
                        const float v = vs[x * kLd + j * 32 + lane];
                        o2[0][j] = mul_add2(make_float2(pp.x, pp.y), make_float2(v, v), o2[0][j]);
                        o2[1][j] = mul_add2(make_float2(pp.z, pp.w), make_float2(v, v), o2[1][j]);
                    }
                }
            } else {
#pragma unroll 4
                for (int x = 0; x < kSimtTile; ++x) {
                    const float4 pp = *reinterpret_cast<const float4 *>(ps + (warp * kSimtTile + x) * 4);
#pragma unroll
                    for (int j = 0; j < kCols; ++j) {
                        float v = vs[x * kLd + j * 32 + lane];
                        if (!(fabsf(v) < INFINITY)) {
                            bad |= j * 32 + lane < p.d;
                            v = 0.f;
                        }
                        o2[0][j] = mul_add2(make_float2(pp.x, pp.y), make_float2(v, v), o2[0][j]);
                        o2[1][j] = mul_add2(make_float2(pp.z, pp.w), make_float2(v, v), o2[1][j]);
                    }
                }
            }
            if (__any_sync(0xffffffffu, bad)) {
                for (int x = 0; x < kSimtTile; ++x) {
                    const float4 pp = *reinterpret_cast<const float4 *>(ps + (warp * kSimtTile + x) * 4);
                    const float w4[4] = {pp.x, pp.y, pp.z, pp.w};
#pragma unroll
                    for (int j = 0; j < kCols; ++j) {
                        const float v = vs[x * kLd + j * 32 + lane];
#pragma unroll
                        for (int a = 0; a < 4; ++a)
                            if (!(fabsf(v) < INFINITY) && ((see[a] >> x) & 1)) o(a, j) = fmaf(w4[a], v, o(a, j));
                    }
                }
            }
        }
        __syncthreads();
        const bool unit_ends = cur.tile + 1 == cur.r.tiles;
        if (unit_ends || cur.left == 1) {
            const bool whole = unit_ends && start_tile == 0;
            if (tid == 0 && start_tile == 0 && !unit_ends) record_unit(p, cur, cur.tile, total);
            float *dst = partial_of(p, blockIdx.x, start_tile > 0 ? 0 : 1);
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const int ur = row0 + a;
                if (ur >= rows) continue;
                const float r = l[a] == 0.f ? 0.f : 1.f / l[a];
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    const int col = j * 32 + lane;
                    if (col >= p.d) continue;
                    if (whole)
                        static_cast<float *>(p.out)[row_offset(p, cur, cur.row_tile * p.rt + ur) + col] = o(a, j) * r;
                    else
                        dst[partial_at(p, ur, col)] = o(a, j);
                }
                if (!whole && lane == 0) {
                    dst[p.rt * p.d + ur * 2] = m[a];
                    dst[p.rt * p.d + ur * 2 + 1] = l[a];
                }
            }
            fresh = true;
        }
        cur.advance(p, 1);
    }
    cp_wait<0>();
}

constexpr int kFewTile = 64, kFewWarps = 8, kFewRows = 16;
constexpr int kWarpRows = 4;       // query rows a warp

// fp32 for few rows (16 a unit).  Keys and values go from memory straight into
// registers: kLanes lanes have a token (16 bytes of every kLanes * 16), a warp kTokens
// tokens at a time for 4 query rows, the next tokens on their way meanwhile and the page
// ids of those after them.  A unit's rows are dealt to 1, 2 or 4 groups of warps, the
// tokens to the warps of a group in turn, so that a single row has all eight warps.
// Each group of lanes has a maximum, sum and output of its own per row until the block
// leaves the unit; the maximum is raised only when a score passes it by 2^8.  In the
// steps past the prefix, values that a row does not see are left out, whatever they are.
// FULL: d is D.
template <int D, bool FULL>
__global__ void __launch_bounds__(kFewWarps * 32, D == 64 ? 2 : 1) attention_few_kernel(const AttnParams p) {
    constexpr int kLanes = D == 256 ? 16 : 8, kTokens = 32 / kLanes, kVec = D / (4 * kLanes);
    __shared__ ScanShared scan;
    __shared__ float4 sums[kFewWarps][kWarpRows][D / 4];
    __shared__ float2 tops[kFewWarps][kWarpRows];         // maximum, sum
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tok = lane / kLanes, first_chunk = lane % kLanes, chunks = p.d >> 2;
    Cursor cur;
    const uint32_t total = start_block(p, scan, cur);
    while (cur.left > 0) {
        const int tiles = min(cur.left, cur.r.tiles - cur.tile), rows = min(p.rt, cur.r.n * p.group - cur.row_tile * p.rt);
        const int begin = cur.tile * kFewTile, end = min(begin + tiles * kFewTile, cur.r.len);
        const int sure = min(cur.r.len - cur.r.n, end);        // tokens before it are seen by every row
        const int groups = rows <= 4 ? 1 : rows <= 8 ? 2 : 4, parts = kFewWarps / groups;
        const int row0 = (warp % groups) * kWarpRows, step = parts * kTokens;
        float2 q[kWarpRows][2 * kVec], o[kWarpRows][2 * kVec];
        float m[kWarpRows], l[kWarpRows];
#pragma unroll
        for (int a = 0; a < kWarpRows; ++a) {
            const bool live = row0 + a < rows;
            const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) +
                                                                 (live ? row_offset(p, cur, cur.row_tile * p.rt + row0 + a) : 0));
#pragma unroll
            for (int x = 0; x < kVec; ++x) {
                const int c = first_chunk + x * kLanes;
                const float4 u = live && c < chunks ? src[c] : make_float4(0.f, 0.f, 0.f, 0.f);
                q[a][2 * x] = make_float2(u.x, u.y);
                q[a][2 * x + 1] = make_float2(u.z, u.w);
                o[a][2 * x] = o[a][2 * x + 1] = make_float2(0.f, 0.f);
            }
            m[a] = -INFINITY;
            l[a] = 0.f;
        }
        auto load = [&](float4 (&k)[kVec], float4 (&v)[kVec], int c, int page) {
            const bool real = c < end;
            const int row = real ? ((checked_page(p, page) * p.n_kv + cur.head) << p.page_shift) + (c & ((1 << p.page_shift) - 1)) : 0;
            const long long at = (long long)row * chunks + first_chunk;
#pragma unroll
            for (int x = 0; x < kVec; ++x) {
                const bool has = FULL || (real && first_chunk + x * kLanes < chunks);      // FULL: row 0, masked below
                k[x] = has ? __ldg(static_cast<const float4 *>(p.k) + at + x * kLanes) : make_float4(0.f, 0.f, 0.f, 0.f);
                v[x] = has ? __ldg(static_cast<const float4 *>(p.v) + at + x * kLanes) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        };
        auto add = [&](const float4 (&k)[kVec], const float4 (&v)[kVec], int c) {
            float s[kWarpRows];
            bool on[kWarpRows];
#pragma unroll
            for (int a = 0; a < kWarpRows; ++a) {
                float2 t = make_float2(0.f, 0.f);
#pragma unroll
                for (int x = 0; x < kVec; ++x) {
                    t = mul_add2(make_float2(k[x].x, k[x].y), q[a][2 * x], t);
                    t = mul_add2(make_float2(k[x].z, k[x].w), q[a][2 * x + 1], t);
                }
                s[a] = t.x + t.y;
                on[a] = true;
            }
#pragma unroll
            for (int b = kLanes / 2; b > 0; b >>= 1)
#pragma unroll
                for (int a = 0; a < kWarpRows; ++a) s[a] += __shfl_xor_sync(0xffffffffu, s[a], b);
            const bool masked = c - tok + kTokens > sure;
            bool raise = false;
#pragma unroll
            for (int a = 0; a < kWarpRows; ++a) {
                s[a] *= p.scale_log2;
                if (masked) {
                    const uint32_t see = row0 + a < rows ? seen_word(p, cur.r, (cur.row_tile * p.rt + row0 + a) / p.group, c & ~31) : 0u;
                    on[a] = (see >> (c & 31)) & 1;
                    if (!on[a]) s[a] = -INFINITY;
                }
                raise |= s[a] > m[a] + 8.f;        // from -infinity by any score
            }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int a = 0; a < kWarpRows; ++a) {
                    const float top = fmaxf(m[a], s[a]), scale = top == -INFINITY ? 1.f : exp2f(m[a] - top);
                    m[a] = top;
                    l[a] *= scale;
#pragma unroll
                    for (int x = 0; x < 2 * kVec; ++x) o[a][x] = make_float2(o[a][x].x * scale, o[a][x].y * scale);
                }
            }
#pragma unroll
            for (int a = 0; a < kWarpRows; ++a) {
                const float w = on[a] ? exp2f(s[a] - (m[a] == -INFINITY ? 0.f : m[a])) : 0.f;
                l[a] += w;
                const float2 w2 = make_float2(w, w);
                if (masked && !on[a]) continue;
#pragma unroll
                for (int x = 0; x < kVec; ++x) {
                    o[a][2 * x] = mul_add2(w2, make_float2(v[x].x, v[x].y), o[a][2 * x]);
                    o[a][2 * x + 1] = mul_add2(w2, make_float2(v[x].z, v[x].w), o[a][2 * x + 1]);
                }
            }
        };
        if (row0 < rows) {
            float4 k0[kVec], v0[kVec], k1[kVec], v1[kVec];
            int c = begin + (warp / groups) * kTokens + tok;
            int page = page_of(p, cur.s, cur.r, c);
            load(k0, v0, c, page);
            page = page_of(p, cur.s, cur.r, c + step);
            while (c - tok < end) {
                load(k1, v1, c + step, page);
                page = page_of(p, cur.s, cur.r, c + 2 * step);
                add(k0, v0, c);
                c += step;
                if (c - tok >= end) break;
                load(k0, v0, c + step, page);
                page = page_of(p, cur.s, cur.r, c + 2 * step);
                add(k1, v1, c);
                c += step;
            }
        }
        // the warp's groups of lanes join, then the warps of a group of rows
#pragma unroll
        for (int a = 0; a < kWarpRows; ++a) {
            float top = m[a];
#pragma unroll
            for (int b = 16; b >= kLanes; b >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, b));
            const float scale = m[a] == -INFINITY ? 0.f : exp2f(m[a] - top);
            l[a] *= scale;
#pragma unroll
            for (int x = 0; x < 2 * kVec; ++x) o[a][x] = make_float2(o[a][x].x * scale, o[a][x].y * scale);
#pragma unroll
            for (int b = 16; b >= kLanes; b >>= 1) {
                l[a] += __shfl_xor_sync(0xffffffffu, l[a], b);
#pragma unroll
                for (int x = 0; x < 2 * kVec; ++x) {
                    o[a][x].x += __shfl_xor_sync(0xffffffffu, o[a][x].x, b);
                    o[a][x].y += __shfl_xor_sync(0xffffffffu, o[a][x].y, b);
                }
            }
            if (tok == 0) {
#pragma unroll
                for (int x = 0; x < kVec; ++x)
                    sums[warp][a][first_chunk + x * kLanes] = make_float4(o[a][2 * x].x, o[a][2 * x].y, o[a][2 * x + 1].x, o[a][2 * x + 1].y);
                if (lane == 0) tops[warp][a] = make_float2(top, l[a]);
            }
        }
        __syncthreads();
        const bool whole = tiles == cur.r.tiles;
        float *dst = partial_of(p, blockIdx.x, cur.tile > 0 ? 0 : 1);
        for (int x = tid; x < rows * chunks; x += kFewWarps * 32) {
            const int row = x / chunks, c = x - row * chunks, w0 = row / kWarpRows, a = row % kWarpRows;
            float top = -INFINITY, sum = 0.f;
            float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = w0; w < kFewWarps; w += groups) top = fmaxf(top, tops[w][a].x);
            for (int w = w0; w < kFewWarps; w += groups) {
                const float2 t = tops[w][a];
                const float scale = t.x == -INFINITY ? 0.f : exp2f(t.x - top);
                const float4 part = sums[w][a][c];
                sum += t.y * scale;
                u.x += part.x * scale;
                u.y += part.y * scale;
                u.z += part.z * scale;
                u.w += part.w * scale;
            }
            if (whole) {
                const float r = sum == 0.f ? 0.f : 1.f / sum;
                *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + row_offset(p, cur, cur.row_tile * p.rt + row) + c * 4) =
                    make_float4(u.x * r, u.y * r, u.z * r, u.w * r);
            } else {
                *reinterpret_cast<float4 *>(dst + partial_at(p, row, c * 4)) = u;
                if (c == 0) *reinterpret_cast<float2 *>(dst + p.rt * p.d + row * 2) = make_float2(top, sum);
            }
        }
        if (tid == 0 && cur.tile == 0 && !whole) record_unit(p, cur, tiles - 1, total);
        __syncthreads();
        cur.advance(p, tiles);
    }
}

// Block (c, y): if a unit starts in block c's part of the list and goes on after it
// (its record says so), adds up the parts: c's slot 1, then slot 0 of each block
// after it until the unit ends.  A warp has 8 rows x 16 columns at a time: 128-byte
// reads, 32-byte writes.  gridDim.y is a unit's rows / kJoinRows: 16 rows a block made
// 8 trees of 64 take 58.4 us for 56.6 and the small fp32 case 15.9 for 13.2, 4 rows
// gained nothing.
template <typename E>
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(const AttnParams p) {
    const int c = blockIdx.x, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const JoinRecord rec = p.records[c];
    const int across = (p.d + 15) >> 4, pieces = ((rec.rows + 7) >> 3) * across;
    for (int x = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5); x < pieces; x += gridDim.y * (kJoinThreads / 32)) {
        const int row = (x / across) * 8 + (lane & 7), col = (x % across) * 16 + (lane >> 3) * 4;
        if (row >= rec.rows || col >= p.d) continue;
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int i = 0; i < rec.parts; ++i) {
            const float *src = partial_of(p, c + i, i == 0 ? 1 : 0);
            const float2 ml = *reinterpret_cast<const float2 *>(src + p.rt * p.d + row * 2);
            const float4 u = *reinterpret_cast<const float4 *>(src + partial_at(p, row, col));
            const float top = fmaxf(m, ml.x), ref = top == -INFINITY ? 0.f : top;
            const float old = exp2f(m - ref), w = exp2f(ml.x - ref);
            m = top;
            l = l * old + ml.y * w;
            o.x = o.x * old + u.x * w;
            o.y = o.y * old + u.y * w;
            o.z = o.z * old + u.z * w;
            o.w = o.w * old + u.w * w;
        }
        const float r = l == 0.f ? 0.f : 1.f / l;
        const int unit_row = rec.first_row + row, i = unit_row / p.group;
        E *out = static_cast<E *>(p.out) + ((long long)(rec.begin + i) * p.n_q + rec.head * p.group + unit_row - i * p.group) * p.d + col;
        if constexpr (sizeof(E) == 2)
            *reinterpret_cast<uint2 *>(out) = make_uint2(pack_bf16(o.x * r, o.y * r), pack_bf16(o.z * r, o.w * r));
        else
            *reinterpret_cast<float4 *>(out) = make_float4(o.x * r, o.y * r, o.z * r, o.w * r);
    }
}

// What a call runs: rows and cached tokens a unit tile, blocks a SM.
struct Variant {
    bool tc, few;            // tcgen05; fp32 for few rows
    int rt, tk, per_sm, unit_cost;
};

// Pages of whole swizzle atoms (8 rows) come by tensor copies, a page a copy, smaller
// ones by 16-byte copies, whose address arithmetic costs more than the transfer: pages
// of 8, 16, 64 by tensor copies 83, 75, 75 us for 32 requests over <= 8192 and 54 us
// for 8 trees of 64; by 16-byte copies 127, 109, 101 us and 131 us.
constexpr int kTmaMinPage = 8;

// The kernel goes by the rows that share a kv head of a request, on average (lengths
// are on the device).  More than 16 go to tcgen05: with warp MMAs a unit of 16 rows
// reads K and V again for each 16.  Page 16, 4 query heads a kv head, tcgen05 against
// warp MMAs: 8 requests over <= 20000, 16 rows 63 and 57 us, 24 rows 60 and 76, 32 rows
// 56 and 73, 64 rows 66 and 147; 64 requests over <= 900, 16 rows 58 and 32, 32 rows
// 62 and 47, 64 rows 65 and 92; one request over 4000, 32 rows 17.0 and 17.1.
// fp32: up to 8 rows go to the kernel without shared tiles.  It and the other: 39
// requests of one token over <= 6697, 1 row of 112, 89 and 166 us; 48 over <= 25977, 1 row
// of 64, 183 and 491; 48 over <= 421, 8 rows of 256, 77 and 151; 10 over <= 39506, 8 rows
// of 112, 110 and 122; but 75 of 3 tokens over <= 16886, 12 rows of 80, 367 and 247.
// Units of 256 rows when that is more than 128: 8 x 256 rows 53 us against 67 with
// units of 128, 8 x 160 rows 55 against 58, 1 x 256 rows over <= 65536 72 against 99,
// 32 x 160 over <= 2000 the same.
// unit_cost, in tiles, stands for a unit's start and end: 128 requests of one token take
// 305, 240, 242, 248 us with 0, 2, 4, 8; 8 trees of 64 take 81, 62.5, 60.1, 60.2 with 2, 4,
// 6, 8; in fp32 39 requests of one token over <= 6697 take 103, 89, 91 with 1, 2, 4.
Variant variant_of(const lora_kv_pages *kv, int group, int S, int T) {
    const int d = kv->head_dim;
    const long long rows = (long long)T * group;       // against S: rows a request and kv head, on average
    if (kv->dtype == LORA_F32) {
        if (rows <= 8LL * S) return {false, true, kFewRows, kFewTile, d <= 64 ? 2 : 1, 2};
        return {false, false, kSimtRows, kSimtTile, d <= 128 ? 2 : 1, 1};
    }
    if ((d == 64 || d == 128) && rows > (long long)kRows * S) return {true, false, rows > 128LL * S ? 256 : 128, 128, 1, 8};
    const bool tma = kv->page_size >= kTmaMinPage;
    return {false, false, kRows, d <= 64 ? 128 : 64, tma && d <= 128 ? 2 : 1, 2};
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

// Boxes of 64 head elements (columns from head_dim on read as zeros) x `rows` cache rows.
bool make_map(CUtensorMap *map, void *pages, const lora_kv_pages *kv, int rows) {
    if (!encode_fn()) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)kv->head_dim, (cuuint64_t)kv->n_pages * kv->n_kv_heads * kv->page_size};
    const cuuint64_t strides[1] = {(cuuint64_t)kv->head_dim * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)rows}, step[2] = {1, 1};
    return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, pages, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool TMA>
int launch_mma(const KvMaps &maps, const AttnParams &p, cudaStream_t st) {
    using Sh = MmaShape<D, TMA>;
    if (smem_optin(reinterpret_cast<const void *>(attention_mma_kernel<D, TMA>), Sh::kSmem)) return LORA_ERR_CUDA;
    attention_mma_kernel<D, TMA><<<p.grid, Sh::kThreadsAll, Sh::kSmem, st>>>(maps, p);
    count_launch();
    return cuda_status(cudaGetLastError());
}

template <int D>
int launch_simt(const AttnParams &p, cudaStream_t st) {
    const size_t smem = (size_t)(kSimtRows * D + 4 * kSimtTile * 4 + 4 * kSimtTile * (D + 4)) * 4;
    if (smem_optin(reinterpret_cast<const void *>(attention_simt_kernel<D>), smem)) return LORA_ERR_CUDA;
    attention_simt_kernel<D><<<p.grid, kThreads, smem, st>>>(p);
    count_launch();
    return cuda_status(cudaGetLastError());
}

template <int D>
int launch_few(const AttnParams &p, cudaStream_t st) {
    if (p.d == D) attention_few_kernel<D, true><<<p.grid, kFewWarps * 32, 0, st>>>(p);
    else attention_few_kernel<D, false><<<p.grid, kFewWarps * 32, 0, st>>>(p);
    count_launch();
    return cuda_status(cudaGetLastError());
}

int launch_attention(const lora_kv_pages *kv, const AttnParams &p, const Variant &v, cudaStream_t st) {
    if (v.few) return p.d <= 64 ? launch_few<64>(p, st) : p.d <= 128 ? launch_few<128>(p, st) : launch_few<256>(p, st);
    if (kv->dtype == LORA_F32)
        return p.d <= 64 ? launch_simt<64>(p, st) : p.d <= 128 ? launch_simt<128>(p, st) : launch_simt<256>(p, st);
    KvMaps maps = {};
    const bool tma = kv->page_size >= kTmaMinPage;
    if (tma) {
        const int rows = kv->page_size < v.tk ? kv->page_size : v.tk;
        if (!make_map(&maps.k, kv->k, kv, rows) || !make_map(&maps.v, kv->v, kv, rows)) return LORA_ERR_CUDA;
    }
    if (v.tc) return launch_attention_tc(tma ? &maps : nullptr, p, st);
    if (tma)
        return p.d <= 64 ? launch_mma<64, true>(maps, p, st)
               : p.d <= 128 ? launch_mma<128, true>(maps, p, st) : launch_mma<256, true>(maps, p, st);
    return p.d <= 64 ? launch_mma<64, false>(maps, p, st)
           : p.d <= 128 ? launch_mma<128, false>(maps, p, st) : launch_mma<256, false>(maps, p, st);
}

size_t partial_bytes(const Variant &v, int d) {
    return (size_t)num_sms() * v.per_sm * (2 * v.rt * (d + 2) * sizeof(float) + sizeof(JoinRecord));
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" size_t lora_tree_attention_workspace_size(const lora_kv_pages *kv, int n_q_heads, int S, int T) {
    if (decode::check_kv(kv, n_q_heads) || n_q_heads < 1 || S < 0 || T < 0) return 0;
    if (S == 0) return 16;
    // T tokens of one request have the most rows a kv head, and the kernel for more rows never needs less
    return partial_bytes(variant_of(kv, n_q_heads / kv->n_kv_heads, 1, T), kv->head_dim) + 16;
}

extern "C" int lora_tree_attention(const lora_kv_pages *kv, const void *q, int n_q_heads, const int *seg_starts, int S,
                                   int T, const int *kv_lens, const int *page_table, int max_pages,
                                   const long long *tree_mask, int mask_words, float scale, void *out, void *workspace,
                                   size_t ws_bytes, lora_stream stream) {
    int rc = decode::check_kv(kv, n_q_heads);
    if (rc) return rc;
    if (n_q_heads < 1) return LORA_ERR_SHAPE;
    if (!(scale > 0.f) || scale > 1.0e30f) return LORA_ERR_ARG;
    if (S < 0 || T < 0 || (S == 0 && T > 0) || max_pages < 0 || (tree_mask && mask_words < 1)) return LORA_ERR_ARG;
    if ((long long)max_pages * kv->page_size > 0x7fffffffLL - 1024) return LORA_ERR_SHAPE;
    if ((long long)T * n_q_heads > 0x7fffffffLL) return LORA_ERR_SHAPE;
    if (T == 0) return LORA_OK;
    if (!q || !out || !seg_starts || !kv_lens || !page_table || !workspace || max_pages < 1) return LORA_ERR_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || ((uintptr_t)tree_mask & 7u) ||
        (((uintptr_t)seg_starts | (uintptr_t)kv_lens | (uintptr_t)page_table) & 3u))
        return LORA_ERR_ARG;
    if (num_sms() < 1) return LORA_ERR_CUDA;
    const Variant variant = variant_of(kv, n_q_heads / kv->n_kv_heads, S, T);
    if (ws_bytes < partial_bytes(variant, kv->head_dim) + 16) return LORA_ERR_ARG;
    decode::AttnParams p;
    p.q = q;
    p.k = kv->k;
    p.v = kv->v;
    p.n_q = n_q_heads;
    p.n_kv = kv->n_kv_heads;
    p.group = n_q_heads / kv->n_kv_heads;
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
    p.scale_log2 = scale * 1.44269504088896340736f;
    p.out = out;
    p.status = kv->status;
    cudaStream_t st = (cudaStream_t)stream;
    p.rt = variant.rt;
    p.tk = variant.tk;
    p.tk_shift = decode::log2_of(variant.tk);
    p.unit_cost = variant.unit_cost;
    const long long tiles = (long long)max_pages * kv->page_size / variant.tk + 1 + variant.unit_cost;
    const long long units = (long long)T * p.group / variant.rt + S;       // a kv head
    if (tiles * units > 0x7fffffffLL / p.n_kv) return LORA_ERR_SHAPE;
    p.max_places = (uint32_t)(tiles * units * p.n_kv);
    p.grid = num_sms() * variant.per_sm;
    p.records = static_cast<JoinRecord *>(workspace);
    p.partial = reinterpret_cast<float *>(p.records + p.grid);
    if ((rc = launch_attention(kv, p, variant, st))) return rc;
    // the join starts while the last blocks run; it waits for them before it reads their sums
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.grid, p.rt / kJoinRows);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = kv->dtype == LORA_BF16 ? cudaLaunchKernelEx(&cfg, attention_join_kernel<__nv_bfloat16>, p)
                                                 : cudaLaunchKernelEx(&cfg, attention_join_kernel<float>, p);
    count_launch();
    return cuda_status(e);
}
