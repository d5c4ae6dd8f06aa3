// Norm, rotation with several axes and append of many tokens (lora_kv_append_axes).
//
// The formulas are append.cu's.  Each token's heads are read and written once, so memory is
// the bound, if enough is on its way: a block keeps a ring of whole tokens in shared memory
// (queries, keys and values by bulk copies; the cosines and sines that its axes choose by
// 4-byte copies, once for all heads), eight warps turn one token in place, and bulk stores
// take its queries to q_out and each key and value head to its slot.  Values never pass
// through registers.
//
// 8192 tokens of 48 heads of 128 with norms, three axes in turn: 34.7 us, 5.9 TB/s, 0.88
// of the measured copy (append.cu's kernel, whose halves are read in 8-byte pieces and
// whose blocks end with their loads: 71 us).  Instructions come next: schedulers issue in
// two cycles of three.  Four stages and three blocks a SM; 5 stages 35.1 us, 3 stages and
// four blocks 39.1, 6 stages and two blocks 37.2.  Several small tokens a stage gained
// little (12 heads 20.5 -> 16.9 us, 48 heads of 64 29.0 -> 27.9) and cost the larger ones
// (37.4 -> 41.0).
#include "append.cuh"
#include "packed.cuh"
#include "tc_common.cuh"

namespace lora {
namespace {

using namespace decode;
using namespace tc;

constexpr int kConsumers = 8, kWork = kConsumers * 32, kAll = kWork + 64;       // a warp copies, a warp stores
constexpr int kStages = 4;
constexpr int kPerSm = 3;
constexpr int kThird = 75 << 10;          // of a SM's shared memory
constexpr int kMaxToken = 26 << 10;       // bytes of a token's heads: two blocks a SM
// Bytes of all heads from which on this kernel takes a call.  It and append.cu's, bf16, halves, norms, three axes in turn:
// 48 heads of 128, 512 tokens (6 MB) 6.2 and 6.0 us, 1024 tokens 7.3 and 10.3, 8192 tokens 34.7 and 71.3; neighbours, 608
// tokens (7.3 MB) 6.1 and 5.4, 1024 tokens 7.6 and 8.5, 8192 tokens 35.6 and 54.5; 12 heads of 128, 2048 tokens (6 MB)
// 7.0 and 7.0, 4096 tokens 11.6 and 12.1, 8192 tokens 19.8 and 24.5; 48 heads of 64, 1024 tokens (6 MB) 6.7 and 6.5, 2048
// tokens 8.8 and 11.1; 48 heads of 80, 1024 tokens (8 MB) 7.2 and 9.6; fp32, 48 heads of 128, 512 tokens (12 MB) 6.2 and
// 6.4, 8192 tokens 68 and 87.  One limit for all of them: neighbours, which append.cu reads in 16-byte pieces, break even
// between 700 and 800 tokens of 48 heads of 128 (9 MB), and lose about a microsecond between the limit and that.
constexpr long long kMinBytes = 7 << 20;

struct StreamParams {
    AppendParams a;
    int T, q_bytes, k_bytes, stage, table_at;      // bytes of a token's queries, of its keys; of a stage; where its table lies
};

struct Control {
    uint64_t full[kStages], done[kStages], empty[kStages];
    volatile int abort;
};

__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, Control &ctl) {
    bool ok = false;
    for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait(bar, parity);
    if (!ok) {
        ok = wait_phase(bar, parity, &ctl.abort);
        if (!ok) ctl.abort = 1;
    }
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void copy_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async8(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(dst), "l"(src) : "memory");
}

// One warp: token by token into the ring.
template <typename E>
__device__ void copy_tokens(const StreamParams &sp, uint8_t *ring, Control &ctl) {
    const AppendParams &p = sp.a;
    const int lane = threadIdx.x & 31, half = p.rot >> 1;
    uint32_t axes = 0;                     // of this lane's table entries lane, lane + 32, ..: two bits each
    for (int x = 0; x * 32 + lane < p.rot; ++x) {
        const int at = x * 32 + lane, i = at < half ? at : at - half;
        axes |= (uint32_t)((p.axes[i >> 2] >> (2 * (i & 3))) & 3) << (2 * x);
    }
    auto position = [&](long long t) {     // lane a: of axis a
        if (t >= sp.T || lane >= p.n_axes || !((p.used_axes >> lane) & 1)) return 0;
        return __ldg(p.positions + t * p.n_axes + lane);
    };
    int pos = position(blockIdx.x), it = 0;
    for (long long t = blockIdx.x; t < sp.T; t += gridDim.x, ++it) {
        const int stage = it % kStages, ahead = position(t + gridDim.x);
        if (pos < 0 || pos >= p.n_pos) {
            if (p.rot) flag_status(p.status, LORA_DEV_BAD_POSITION);
            pos = pos < 0 ? 0 : p.n_pos - 1;
        }
        if (!wait_warp(&ctl.empty[stage], ((it / kStages) & 1) ^ 1, ctl)) break;
        uint8_t *to = ring + stage * sp.stage;
        if (lane == 0) {
            mbar_arrive_expect_tx(&ctl.full[stage], sp.q_bytes + 2 * sp.k_bytes);
            if (sp.q_bytes) bulk_g2s(to, static_cast<const E *>(p.q) + t * p.ld_q, sp.q_bytes, &ctl.full[stage]);
            bulk_g2s(to + sp.q_bytes, static_cast<const E *>(p.k) + t * p.ld_k, sp.k_bytes, &ctl.full[stage]);
            bulk_g2s(to + sp.q_bytes + sp.k_bytes, static_cast<const E *>(p.v) + t * p.ld_v, sp.k_bytes, &ctl.full[stage]);
            copy_async8(smem_u32(to + sp.table_at - 16), p.slots + t);
        }
        const uint32_t table = smem_u32(to + sp.table_at);
        for (int x = 0; x * 32 < p.rot; ++x) {
            const int row = __shfl_sync(0xffffffffu, pos, (axes >> (2 * x)) & 3), at = x * 32 + lane;
            if (at < p.rot) copy_async4(table + at * 4, p.cos_sin + (long long)row * p.rot + at);
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(smem_u32(&ctl.full[stage])) : "memory");
        pos = ahead;
    }
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    // bulk copies on their way land before the block leaves, also where others gave up
    for (int x = max(0, it - kStages); x < it; ++x) wait_phase(&ctl.full[x % kStages], (x / kStages) & 1, nullptr);
}

// Eight warps: LANES threads a head, its norm and rotation in place.
template <typename E, int LANES, int PAIRS>
__device__ void turn_tokens(const StreamParams &sp, uint8_t *ring, Control &ctl) {
    constexpr int kGroups = kWork / LANES;
    constexpr bool kApart = PAIRS == kFar;
    const AppendParams &p = sp.a;
    const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES, half = p.rot >> 1, heads = p.n_q + p.n_kv;
    const unsigned mask = group_mask<LANES>();
    const int at = lane * 8;
    const bool inside = at < p.d, turns = at < p.rot;
    const int o0 = kApart && turns ? lane * 4 : at, o1 = kApart && turns ? half + lane * 4 : at + 4;
    float2 q_norm[4] = {}, k_norm[4] = {};
    auto load_norm = [&](const void *norm, float2 (&to)[4]) {
        if (!norm || !inside) return;
        Quads<E> n;
        float w[8];
        load_quads<E, kApart>(n, static_cast<const E *>(norm), o0, o1);
        n.a.get(w);
        n.b.get(w + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) to[e] = make_float2(w[2 * e], w[2 * e + 1]);
    };
    load_norm(p.q_norm, q_norm);
    load_norm(p.k_norm, k_norm);
    int it = 0;
    for (long long t = blockIdx.x; t < sp.T; t += gridDim.x, ++it) {
        const int stage = it % kStages;
        if (!wait_warp(&ctl.full[stage], (it / kStages) & 1, ctl)) return;
        uint8_t *token = ring + stage * sp.stage;
        float c[4] = {}, s[4] = {};
        if (turns) {
            const float *table = reinterpret_cast<const float *>(token + sp.table_at) + lane * 4;
            *reinterpret_cast<float4 *>(c) = *reinterpret_cast<const float4 *>(table);
            *reinterpret_cast<float4 *>(s) = *reinterpret_cast<const float4 *>(table + half);
        }
        const float2 c2[2] = {make_float2(c[0], c[1]), make_float2(c[2], c[3])}, s2[2] = {make_float2(s[0], s[1]), make_float2(s[2], s[3])};
        auto turn = [&](E *row, const float2 (&norm)[4], bool normed) {
            Quads<E> held;
            float h[8] = {};
            if (inside) {
                load_quads<E, kApart>(held, row, o0, o1);
                held.a.get(h);
                held.b.get(h + 4);
            }
            float2 x[4];
            float r = 1.f;
            if (normed) {
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum += h[e] * h[e];
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(mask, sum, o);
                r = rsqrtf(fmaf(sum, p.inv_d, p.eps));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = make_float2(h[2 * e], h[2 * e + 1]);
                if (normed) x[e] = mul2(mul2(x[e], make_float2(r, r)), norm[e]);
            }
            if (turns) {
                if (PAIRS == kFar) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 m = x[e], n = x[2 + e], t = mul2(n, s2[e]);
                        x[e] = fma2(m, c2[e], make_float2(-t.x, -t.y));
                        x[2 + e] = fma2(m, s2[e], mul2(n, c2[e]));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float m = x[e].x, n = x[e].y;
                        x[e].x = m * c[e] - n * s[e];
                        x[e].y = m * s[e] + n * c[e];
                    }
                }
            }
            if (inside) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    h[2 * e] = x[e].x;
                    h[2 * e + 1] = x[e].y;
                }
                held.a.set(h);
                held.b.set(h + 4);
                store_quads<E, kApart>(held, row, o0, o1);
            }
        };
        int head = group;
        E *row = reinterpret_cast<E *>(token) + head * p.d;
        const int step = kGroups * p.d;
        for (; head < p.n_q; head += kGroups, row += step) turn(row, q_norm, p.q_norm != nullptr);
        for (; head < heads; head += kGroups, row += step) turn(row, k_norm, p.k_norm != nullptr);
        fence_proxy_async();               // the stores read through the async proxy
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&ctl.done[stage]);
    }
}

// One warp: the turned token to q_out and its slot.
template <typename E>
__device__ void store_tokens(const StreamParams &sp, uint8_t *ring, Control &ctl) {
    const AppendParams &p = sp.a;
    const int lane = threadIdx.x & 31, bytes = p.d * (int)sizeof(E);
    int it = 0;
    for (long long t = blockIdx.x; t < sp.T; t += gridDim.x, ++it) {
        const int stage = it % kStages;
        if (!wait_warp(&ctl.full[stage], (it / kStages) & 1, ctl) || !wait_warp(&ctl.done[stage], (it / kStages) & 1, ctl)) break;
        const uint8_t *token = ring + stage * sp.stage;
        const long long slot = *reinterpret_cast<const long long *>(token + sp.table_at - 16);
        if (slot >= p.n_slots && lane == 0) flag_status(p.status, LORA_DEV_BAD_SLOT);
        if (lane == 0 && sp.q_bytes) bulk_s2g(static_cast<E *>(p.q_out) + t * p.n_q * p.d, token, sp.q_bytes);
        if (slot >= 0 && slot < p.n_slots) {
            const long long page = slot >> p.page_shift, off = slot & ((1 << p.page_shift) - 1);
            for (int x = lane; x < 2 * p.n_kv; x += 32) {
                const bool is_v = x >= p.n_kv;
                const long long row = ((page * p.n_kv + (is_v ? x - p.n_kv : x)) << p.page_shift) + off;
                bulk_s2g(static_cast<E *>(is_v ? p.v_pages : p.k_pages) + row * p.d, token + sp.q_bytes + x * bytes, bytes);
            }
        }
        bulk_commit();
        // the stage before has been read by its stores
        asm volatile("cp.async.bulk.wait_group.read 1;\n" ::: "memory");
        __syncwarp();
        if (lane == 0 && it > 0) mbar_arrive(&ctl.empty[(it - 1) % kStages]);
    }
    bulk_wait_all();
}

template <typename E, int LANES, int PAIRS>
__global__ void __launch_bounds__(kAll, kPerSm) append_stream_kernel(const __grid_constant__ StreamParams sp) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ Control ctl;
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&ctl.full[i], 33);
            mbar_init(&ctl.done[i], kConsumers);
            mbar_init(&ctl.empty[i], 1);
        }
        ctl.abort = 0;
        mbar_fence_init();
    }
    __syncthreads();
    if (warp < kConsumers) turn_tokens<E, LANES, PAIRS>(sp, ring, ctl);
    else if (warp == kConsumers) copy_tokens<E>(sp, ring, ctl);
    else store_tokens<E>(sp, ring, ctl);
    __syncthreads();
    if (threadIdx.x == 0 && ctl.abort) flag_status(sp.a.status, LORA_DEV_WAIT_TIMEOUT);
}

template <typename E, int LANES, int PAIRS>
int launch(const StreamParams &sp, cudaStream_t st) {
    const size_t smem = (size_t)kStages * sp.stage;
    if (smem_optin(reinterpret_cast<const void *>(append_stream_kernel<E, LANES, PAIRS>), smem)) return LORA_ERR_CUDA;
    const int per_sm = smem <= (size_t)kThird ? kPerSm : 2, places = num_sms() * per_sm, grid = sp.T < places ? sp.T : places;
    append_stream_kernel<E, LANES, PAIRS><<<grid, kAll, smem, st>>>(sp);
    count_launch();
    return cuda_status(cudaGetLastError());
}

template <typename E, int PAIRS>
int launch(const StreamParams &sp, cudaStream_t st) {
    return sp.a.d <= 64 ? launch<E, 8, PAIRS>(sp, st) : sp.a.d <= 128 ? launch<E, 16, PAIRS>(sp, st) : launch<E, 32, PAIRS>(sp, st);
}

}  // namespace

namespace decode {

bool streams(const AppendParams &p, int T, int esize) {
    const long long token = (p.n_q + 2LL * p.n_kv) * p.d * esize;
    return p.rot % 8 == 0 && token <= kMaxToken && token * T >= kMinBytes;
}

int launch_append_stream(const AppendParams &p, int T, bool bf16, bool near, cudaStream_t st) {
    StreamParams sp;
    sp.a = p;
    sp.T = T;
    const int esize = bf16 ? 2 : 4;
    sp.q_bytes = p.n_q * p.d * esize;
    sp.k_bytes = p.n_kv * p.d * esize;
    sp.table_at = sp.q_bytes + 2 * sp.k_bytes + 16;         // after the slot
    sp.stage = (sp.table_at + p.rot * 4 + 127) & ~127;
    if (bf16) return near ? launch<__nv_bfloat16, kNear>(sp, st) : launch<__nv_bfloat16, kFar>(sp, st);
    return near ? launch<float, kNear>(sp, st) : launch<float, kFar>(sp, st);
}

}  // namespace decode
}  // namespace lora
