// Weights of cached tokens on the tensor cores (tcgen05), for a bf16 cache and many query rows.
//
// S = K Q^T with a key a lane of tensor memory and a row a column: a thread owns a cached
// token, and its weight is the sum along its lane of 2^(s - lse(column)) - no exchange
// between threads, and one order of addition whatever the split.  A block takes pairs of
// key tiles of 128, one a group of four warps, against the same tiles of 128 rows; each
// group has two tiles of scores in tensor memory, so that products run under the
// exponentials.  Rows that fit in the ring of query tiles stay in it for all key tiles of
// a kv head.  Keys are copied while the attention's last kernel runs; what reads its sums
// waits for it.
//
// 8 requests of 64 tokens over <= 16384 (256 rows, 8 kv heads of 128): about 27 us of the
// call's 85, where the products would take 8 and the exponentials, at the 25 a cycle and SM
// that attention_tc.cu measures, 10.  Neither is the bound: the tensor pipe is active for 32 %
// of the time and the exponentials' for 27 %.  A pair of key tiles against 128 rows takes some
// 2200 cycles, for 1024 of products and 1300 of exponentials that run beside them; what the
// summing warps wait for in the other 900 is not known.  To that come the start (scan, first
// copies, 4 us) and the cut into whole key tiles: 16.4 such pairs a block.  Exponentials on
// the multiply-add pipe for a quarter of the columns were slower (90 us), as were twice the
// summing warps (89) and loads of 32 columns that nothing ran under (89).
#include <type_traits>

#include "kv_copy.cuh"
#include "packed.cuh"
#include "tmem.cuh"
#include "weigh.cuh"

namespace lora {
namespace {

using namespace decode;
using namespace tc;

constexpr int kTile = 128;                          // keys a group, rows a query tile
constexpr int kConsumers = 8, kThreads = 16 * 32;   // warps 8 and 9 copy keys, 10 issues products, 12 to 15 copy queries
constexpr int kKeyWarp = 8, kMmaWarp = 10, kQueryWarp = 12;
constexpr uint32_t kTmemCols = 512;

// D: head width padded to 64, 128 or 256.
template <int D>
struct Shape {
    static constexpr int kBytes = kTile * D * 2;            // a tile of keys or queries
    static constexpr int kKeys = D == 256 ? 1 : 2;          // pairs of key tiles
    static constexpr int kQueries = D == 64 ? 6 : D == 128 ? 3 : 1;
    static constexpr size_t kSmem = (size_t)(2 * kKeys + kQueries) * kBytes + 1024;
};

template <int D>
struct Control {
    uint64_t k_full[2][2], k_empty[2], q_full[6], q_empty[6], s_full[2][2], s_empty[2][2], drain;
    volatile int abort;
    uint32_t tmem;
    __align__(16) float lse[Shape<D>::kQueries][kTile];
};

template <int D>
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, Control<D> &ctl) {
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    if (wait_phase(bar, parity, &ctl.abort)) return true;
    ctl.abort = 1;
    return false;
}
template <int D>
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, Control<D> &ctl) {
    return __all_sync(0xffffffffu, wait_bar<D>(bar, parity, ctl));
}

// The block's key tiles of one kv head, and how its query tiles pass through the ring: tile `rows` of key tile t is
// number q0 + (stays ? rows : t * row_tiles + rows).
struct Run {
    int tiles;
    bool stays;
    __device__ __forceinline__ Run(const KeyCursor &c, int ring) : tiles(c.run()), stays(c.r.row_tiles <= ring) {}
    __device__ __forceinline__ uint32_t number(const KeyCursor &c, int t, int row_tile) const {
        return stays ? row_tile : (uint32_t)t * c.r.row_tiles + row_tile;
    }
    __device__ __forceinline__ uint32_t total(const KeyCursor &c) const { return (stays ? 1u : (uint32_t)tiles) * c.r.row_tiles; }
    __device__ __forceinline__ bool last_use(int t) const { return !stays || t + 1 == tiles; }
};

template <int D, bool TMA>
__device__ void copy_keys(const AttnParams &p, const KvMaps &maps, KeyCursor cur, uint8_t *ring, Control<D> &ctl) {
    using Sh = Shape<D>;
    using Copy = std::conditional_t<TMA, TmaCopy<D, kTile>, ChunkCopy<D, kTile, 64>>;
    const int tid = threadIdx.x - kKeyWarp * 32;
    if (TMA && tid >= 32) return;
    const uint32_t base = smem_u32(ring);
    Copy copy[TMA ? 2 : 1];      // page ids of a tile ahead (of ordinary copies, whose rows take many registers, of the next half)
    auto fetch = [&](int w) {
        Cursor at;
        at.r = cur.r;
        at.s = cur.s;
        at.head = cur.head;
        copy[TMA ? w : 0].fetch(p, at, cur.tile * 2 + w, tid);
    };
    uint32_t seq = 0;
    if (TMA) {
        fetch(0);
        fetch(1);
    }
    while (cur.left > 0) {
        const uint32_t stage = seq % Sh::kKeys, use = seq / Sh::kKeys;
        if (TMA ? !wait_warp<D>(&ctl.k_empty[stage], (use & 1) ^ 1, ctl) : !wait_bar<D>(&ctl.k_empty[stage], (use & 1) ^ 1, ctl)) {
            // tensor copies on their way land before the block leaves
            for (uint32_t x = seq < Sh::kKeys ? 0 : seq - Sh::kKeys; TMA && x < seq; ++x)
                for (int w = 0; w < 2; ++w) wait_phase(&ctl.k_full[x % Sh::kKeys][w], (x / Sh::kKeys) & 1, nullptr);
            return;
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            if (!TMA) fetch(w);
            copy[TMA ? w : 0].copy(p, &maps.k, p.k, base + (stage * 2 + w) * Sh::kBytes, &ctl.k_full[stage][w], tid);
            if (!TMA) cp_arrive(&ctl.k_full[stage][w]);
        }
        ++seq;
        cur.advance(p);
        if (TMA && cur.left > 0) {
            fetch(0);
            fetch(1);
        }
    }
    if (TMA) {       // also where others gave up: no copy outlives the block
        for (uint32_t x = seq < Sh::kKeys ? 0 : seq - Sh::kKeys; x < seq; ++x)
            for (int w = 0; w < 2; ++w) wait_phase(&ctl.k_full[x % Sh::kKeys][w], (x / Sh::kKeys) & 1, nullptr);
    }
}

// Four warps of 32 rows, D / 8 lanes a row; rows past the request become zeros.
template <int D>
__device__ void copy_queries(const AttnParams &p, KeyCursor cur, uint8_t *ring, Control<D> &ctl) {
    using Sh = Shape<D>;
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
    const int lane = threadIdx.x & 31, chunk = lane % kLanes, row0 = (threadIdx.x >> 5) * 32 - kQueryWarp * 32;
    const bool inside = chunk * 8 < ((p.d + 15) & ~15), real_chunk = chunk * 8 < p.d;
    uint32_t seq = 0;
    while (cur.left > 0) {
        const Run run(cur, Sh::kQueries);
        const int rows = cur.r.n * p.group;
        const uint32_t total = run.total(cur);
        const long long first = (long long)cur.r.begin * p.n_q + cur.head * p.group;
        int row_tile = 0;
        for (uint32_t x = 0; x < total; ++x, ++seq) {
            const uint32_t slot = seq % Sh::kQueries, use = seq / Sh::kQueries;
            if (!wait_warp<D>(&ctl.q_empty[slot], (use & 1) ^ 1, ctl)) return;
            const uint32_t dst = smem_u32(ring) + slot * Sh::kBytes, sums = smem_u32(ctl.lse[slot]);
            const int row = row_tile * kTile + row0 + lane, i = row / p.group;
            const long long line = row < rows ? first + (long long)i * (p.n_q - p.group) + row : -1;
#pragma unroll
            for (int j = 0; j < 32; j += kRows) {
                const int r = j + lane / kLanes;
                const long long from = __shfl_sync(0xffffffffu, line, r);
                const bool real = from >= 0 && real_chunk;
                if (inside)
                    cp_async16(dst + panel_off(kTile, row0 + r, chunk), static_cast<const __nv_bfloat16 *>(p.q) + (real ? from * p.d + chunk * 8 : 0),
                               real);
            }
            if (seq == 0) asm volatile("griddepcontrol.wait;\n" ::: "memory");       // the attention's sums
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(sums + (row0 + lane) * 4), "l"(p.lse + max(line, 0ll)),
                         "r"(line >= 0 ? 4 : 0)
                         : "memory");
            cp_arrive(&ctl.q_full[slot]);
            if (++row_tile == cur.r.row_tiles) row_tile = 0;
        }
        cur.advance(p, run.tiles);
    }
}

template <int D, bool TMA>
__device__ void issue(const AttnParams &p, KeyCursor cur, uint8_t *keys, uint8_t *queries, Control<D> &ctl) {
    using Sh = Shape<D>;
    constexpr uint32_t kIdesc = idesc_bf16_f32(kTile, kTile);
    constexpr uint32_t kSwizzled = (1024u >> 4) | (1u << 14) | (2u << 29);      // descriptor bits 32..63
    const uint32_t k_lo = (uint32_t)desc_kmajor_sw128(smem_u32(keys)), q_lo = (uint32_t)desc_kmajor_sw128(smem_u32(queries));
    const int steps = (p.d + 15) >> 4;
    uint32_t k_seq = 0, q0 = 0, s_seq[2] = {0, 0};
    while (cur.left > 0) {
        const Run run(cur, Sh::kQueries);
        for (int t = 0; t < run.tiles; ++t, ++k_seq) {
            const uint32_t stage = k_seq % Sh::kKeys;
            const int groups = (cur.tile + t) * kWeighTile + kTile < cur.r.len ? 2 : 1;
            for (int w = 0; w < 2; ++w)
                if (!wait_bar<D>(&ctl.k_full[stage][w], (k_seq / Sh::kKeys) & 1, ctl)) return;
            if (!TMA) fence_proxy_async();
            for (int row_tile = 0; row_tile < cur.r.row_tiles; ++row_tile) {
                const uint32_t q = q0 + run.number(cur, t, row_tile), slot = q % Sh::kQueries;
                if (!run.stays || t == 0) {
                    if (!wait_bar<D>(&ctl.q_full[slot], (q / Sh::kQueries) & 1, ctl)) return;
                    fence_proxy_async();     // ordinary copies; the products read through the async proxy
                }
                fence_after_sync();
                for (int w = 0; w < groups; ++w) {
                    const uint32_t b = s_seq[w] & 1;
                    if (!wait_bar<D>(&ctl.s_empty[w][b], ((s_seq[w] >> 1) & 1) ^ 1, ctl)) return;
                    ++s_seq[w];
                    fence_after_sync();
                    // descriptors: 32-bit sums of 16-byte units to a constant upper half
                    const uint32_t k = k_lo + (stage * 2 + w) * (Sh::kBytes / 16), q_at = q_lo + slot * (Sh::kBytes / 16);
                    const uint32_t d = ctl.tmem + (w * 2 + b) * kTile;
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        if (ks >= steps) break;
                        const uint32_t step = ((ks >> 2) * (kTile * 128) + (ks & 3) * 32) >> 4;
                        asm volatile(
                            "{\n.reg .pred p;\n.reg .b64 a, b;\nsetp.ne.b32 p, %5, 0;\nmov.b64 a, {%1, %3};\nmov.b64 b, {%2, %3};\n"
                            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}\n" ::"r"(d),
                            "r"(k + step), "r"(q_at + step), "n"(kSwizzled), "n"(kIdesc), "r"(ks > 0 ? 1u : 0u)
                            : "memory");
                    }
                    mma_commit(&ctl.s_full[w][b]);
                }
                if (run.last_use(t)) mma_commit(&ctl.q_empty[slot]);
            }
            mma_commit(&ctl.k_empty[stage]);
        }
        q0 += run.total(cur);
        cur.advance(p, run.tiles);
    }
}

// A group of four warps: each thread sums up the weight of one cached token of each of the group's key tiles.
template <int D>
__device__ void consume(const AttnParams &p, KeyCursor cur, float *weights, float decay, Control<D> &ctl) {
    using Sh = Shape<D>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp >> 2;
    const uint32_t tmem = ctl.tmem + ((uint32_t)((warp & 3) * 32) << 16) + w * 2 * kTile;
    uint32_t q0 = 0, s_seq = 0;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const bool computed = *p.computed != 0;
    while (cur.left > 0) {
        const Run run(cur, Sh::kQueries);
        const int rows = cur.r.n * p.group, prefix = cur.r.len - cur.r.n;
        for (int t = 0; t < run.tiles; ++t) {
            const int g0 = (cur.tile + t) * kWeighTile + w * kTile;        // first token of the group
            const int c0 = g0 + (warp & 3) * 32, c = c0 + lane;
            const bool active = g0 < cur.r.len;
            long long slot = -1;
            float old = 0.f;
            if (c < cur.r.len && computed) slot = weight_at(p, cur.s, cur.r, cur.head, c);
            if (slot >= 0 && decay > 0.f && c < prefix) old = weights[slot];
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            for (int row_tile = 0; row_tile < cur.r.row_tiles; ++row_tile) {
                const uint32_t q = q0 + run.number(cur, t, row_tile), at = q % Sh::kQueries;
                // the sums' logarithms; without this wait a group without tokens would be ahead of the ring
                if (!wait_warp<D>(&ctl.q_full[at], (q / Sh::kQueries) & 1, ctl)) return;
                if (active) {
                    const uint32_t b = s_seq & 1;
                    if (!wait_warp<D>(&ctl.s_full[w][b], (s_seq >> 1) & 1, ctl)) return;
                    ++s_seq;
                    fence_after_sync();
                    const int columns = min(kTile, rows - row_tile * kTile);
                    const uint32_t from = tmem + b * kTile;
                    const float *lse = ctl.lse[at];
                    const int seen = c0 + 32 > prefix ? 0 : columns & ~31;        // columns that see all of the warp's tokens
                    auto add = [&](const float (&s)[32], int x0) {
                        const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
#pragma unroll
                        for (int x = 0; x < 32; x += 4) {
                            const float4 l = *reinterpret_cast<const float4 *>(lse + x0 + x);
                            const float2 e0 = fma2(make_float2(s[x], s[x + 1]), scale2, make_float2(-l.x, -l.y));
                            const float2 e1 = fma2(make_float2(s[x + 2], s[x + 3]), scale2, make_float2(-l.z, -l.w));
                            sum[0].x += exp2_fast(e0.x);
                            sum[0].y += exp2_fast(e0.y);
                            sum[1].x += exp2_fast(e1.x);
                            sum[1].y += exp2_fast(e1.y);
                        }
                    };
                    // 32 columns are on their way while the 32 before are summed up
                    int x0 = 0;
#pragma unroll 1
                    for (; x0 + 64 <= seen; x0 += 64) {
                        float s0[32], s1[32];
                        tmem_ld32_start(from + x0, s0);
                        tmem_wait_ld();
                        tmem_arrived(s0);
                        tmem_ld32_start(from + x0 + 32, s1);
                        add(s0, x0);
                        tmem_wait_ld();
                        tmem_arrived(s1);
                        add(s1, x0 + 32);
                    }
#pragma unroll 1
                    for (; x0 < columns && c0 < cur.r.len; x0 += 32) {
                        // drafted tokens, or columns without a row: what is not seen counts nothing, whatever it is
                        float s[32];
                        tmem_ld32(from + x0, s);
                        const int row = row_tile * kTile + x0 + lane;
                        const uint32_t word = row < rows ? seen_word(p, cur.r, row / p.group, c0) : 0u;
#pragma unroll
                        for (int x = 0; x < 32; ++x) {
                            const bool on = (__shfl_sync(0xffffffffu, word, x) >> lane) & 1;
                            const float e = exp2_fast(fmaf(s[x], p.scale_log2, -lse[x0 + x]));
                            if (on) sum[x & 1].x += e;
                        }
                    }
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl.s_empty[w][b]);
                }
                if (run.last_use(t) && lane == 0) mbar_arrive(&ctl.q_empty[at]);
            }
            if (slot >= 0) weights[slot] = old * decay + ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
        }
        q0 += run.total(cur);
        cur.advance(p, run.tiles);
    }
}

template <int D, bool TMA>
__global__ void __launch_bounds__(kThreads, 1)
    weigh_tc_kernel(const __grid_constant__ KvMaps maps, const AttnParams p, float *weights, float decay) {
    using Sh = Shape<D>;
    extern __shared__ uint8_t raw[];
    __shared__ ScanShared scan;
    __shared__ Control<D> ctl;
    uint8_t *keys = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023), *queries = keys + 2 * Sh::kKeys * Sh::kBytes;
    const int warp = threadIdx.x >> 5;
    if (TMA && threadIdx.x == kKeyWarp * 32) prefetch_tmap(&maps.k);
    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::kKeys; ++i) {
            for (int w = 0; w < 2; ++w) mbar_init(&ctl.k_full[i][w], TMA ? 1 : 64);
            mbar_init(&ctl.k_empty[i], 1);
        }
        for (int i = 0; i < Sh::kQueries; ++i) {
            mbar_init(&ctl.q_full[i], 128);
            mbar_init(&ctl.q_empty[i], 1 + kConsumers);
        }
        for (int w = 0; w < 2; ++w)
            for (int b = 0; b < 2; ++b) {
                mbar_init(&ctl.s_full[w][b], 1);
                mbar_init(&ctl.s_empty[w][b], 4);
            }
        mbar_init(&ctl.drain, 1);
        ctl.abort = 0;
        mbar_fence_init();
    }
    Cursor at;
    KeyCursor cur;
    cur.start(p, scan, start_block<kPlain, false>(p, scan, at));
    if (cur.left <= 0) {                // the whole block; no grid ends before those it depends on
        asm volatile("griddepcontrol.wait;\n" ::: "memory");
        return;
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&ctl.tmem, kTmemCols);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp < kConsumers) {
        consume<D>(p, cur, weights, decay, ctl);
    } else if (warp < kMmaWarp) {
        copy_keys<D, TMA>(p, maps, cur, keys, ctl);
        if (!TMA) cp_wait_all();
    } else if (warp == kMmaWarp) {
        if (elect_lane()) {
            issue<D, TMA>(p, cur, keys, queries, ctl);
            mma_commit(&ctl.drain);
            wait_phase(&ctl.drain, 0, nullptr);
        }
        __syncwarp();
    } else if (warp >= kQueryWarp) {
        copy_queries<D>(p, cur, queries, ctl);
        cp_wait_all();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (threadIdx.x == 0 && ctl.abort) flag_status(p.status, LORA_DEV_WAIT_TIMEOUT);
    if (warp == kMmaWarp) tmem_dealloc(ctl.tmem, kTmemCols);
}

template <int D, bool TMA>
int launch(const KvMaps &maps, const AttnParams &p, float *weights, float decay, cudaStream_t st) {
    if (smem_optin(reinterpret_cast<const void *>(weigh_tc_kernel<D, TMA>), Shape<D>::kSmem)) return LORA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Shape<D>::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, weigh_tc_kernel<D, TMA>, maps, p, weights, decay);
    count_launch();
    return launch_status(e);
}

template <int D>
int launch(const KvMaps *maps, const AttnParams &p, float *weights, float decay, cudaStream_t st) {
    return maps ? launch<D, true>(*maps, p, weights, decay, st) : launch<D, false>(KvMaps{}, p, weights, decay, st);
}

}  // namespace

namespace decode {

int launch_weigh_tc(const KvMaps *maps, const AttnParams &p, float *weights, float decay, cudaStream_t st) {
    return p.d <= 64 ? launch<64>(maps, p, weights, decay, st)
           : p.d <= 128 ? launch<128>(maps, p, weights, decay, st) : launch<256>(maps, p, weights, decay, st);
}

}  // namespace decode
}  // namespace lora
