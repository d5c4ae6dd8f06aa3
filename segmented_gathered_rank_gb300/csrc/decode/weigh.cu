// Weights that cached tokens get from an attention (lora_tree_attention_weights):
//
//   w_c <- decay w_c (prefix; a drafted token starts from 0) + sum over the request's rows
//          of 2^(scale log2(e) q . k_c - lse),  lse = log2 sum_c 2^(..) of the row,
//
// over the rows that see c.  The attention's kernels leave lse.
//
// weigh_scores_kernel: with few rows they leave the scores too (4 bytes a row and token,
//   written and read, against 2 d for reading a bf16 key again), and a thread sums up four
//   tokens.  128 requests over <= 8192, 4 rows, 8 kv heads: about 18 us of the call's 269, for
//   50 MB of scores that are still in L2 and 25 MB of weights; the bound is instructions and
//   the chain page id -> weight -> store, which is why both are requested a tile ahead.  One
//   request over 777: 13.6 us, of which the attention is 10.8.  Its exponentials are the fast
//   ones for an fp32 cache as well (2^-22 relative, as exp2f's; a weight below 2^-126 is 0).
// weigh_tc_kernel (weigh_tc.cu; bf16), weigh_kernel (fp32): else the scores are computed
//   once more, keys at rest and rows going by, so that a key's sum stays in one block and
//   its order is fixed.  weigh_kernel has fp32 multiply-adds for its bound, two tokens and
//   eight rows a thread.
#include "packed.cuh"
#include "weigh.cuh"

namespace lora {
namespace {

using namespace decode;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kTile = 64;              // cached tokens a tile, two a lane
constexpr int kWarpRows = 8, kRows = kWarps * kWarpRows;

__global__ void __launch_bounds__(kThreads) weigh_kernel(const AttnParams p, float *weights, float decay) {
    static_assert(kThreads >= kScanThreads, "start_block");
    extern __shared__ __align__(16) float smem[];
    __shared__ ScanShared scan;
    __shared__ float sums[kWarps][kTile], lse[kRows];
    __shared__ int slots[kTile];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, pitch = p.d + 4;
    float *ks = smem, *qs = smem + kTile * pitch;
    Cursor at;
    KeyCursor cur;
    cur.start(p, scan, start_block<kPlain, false>(p, scan, at));
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    if (!*p.computed) return;
    for (; cur.left > 0; cur.advance(p)) {
        const int c0 = cur.tile * kTile, rows = cur.r.n * p.group;
        const long long first = (long long)cur.r.begin * p.n_q + cur.head * p.group;
        __syncthreads();
        if (tid < kTile) slots[tid] = c0 + tid < cur.r.len ? (int)weight_at(p, cur.s, cur.r, cur.head, c0 + tid) : -1;
        __syncthreads();
        for (int j = tid >> 3; j < kTile; j += kThreads / 8)
            for (int e = (tid & 7) * 4; e < p.d; e += 32)
                *reinterpret_cast<float4 *>(ks + j * pitch + e) =
                    slots[j] >= 0 ? *reinterpret_cast<const float4 *>(static_cast<const float *>(p.k) + (long long)slots[j] * p.d + e)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
        float acc[2] = {0.f, 0.f};
        for (int r0 = 0; r0 < rows; r0 += kRows) {
            __syncthreads();
            for (int j = tid >> 3; j < kRows; j += kThreads / 8) {
                const int row = r0 + j, i = row / p.group;
                const long long line = first + (long long)i * (p.n_q - p.group) + row;
                for (int e = (tid & 7) * 4; e < p.d; e += 32)
                    *reinterpret_cast<float4 *>(qs + j * pitch + e) =
                        row < rows ? *reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + line * p.d + e)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
                if ((tid & 7) == 0) lse[j] = row < rows ? p.lse[line] : INFINITY;
            }
            __syncthreads();
            if (r0 + warp * kWarpRows >= rows) continue;
            float2 dot[2][kWarpRows] = {};
            for (int e = 0; e < p.d; e += 4) {
                const float4 k = *reinterpret_cast<const float4 *>(ks + lane * pitch + e);
                const float4 l = *reinterpret_cast<const float4 *>(ks + (lane + 32) * pitch + e);
#pragma unroll
                for (int a = 0; a < kWarpRows; ++a) {
                    const float4 q = *reinterpret_cast<const float4 *>(qs + (warp * kWarpRows + a) * pitch + e);
                    dot[0][a] = fma2(make_float2(k.z, k.w), make_float2(q.z, q.w), fma2(make_float2(k.x, k.y), make_float2(q.x, q.y), dot[0][a]));
                    dot[1][a] = fma2(make_float2(l.z, l.w), make_float2(q.z, q.w), fma2(make_float2(l.x, l.y), make_float2(q.x, q.y), dot[1][a]));
                }
            }
#pragma unroll
            for (int a = 0; a < kWarpRows; ++a) {
                const int row = r0 + warp * kWarpRows + a;
                if (row >= rows) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t see = seen_word(p, cur.r, row / p.group, c0 + h * 32);
                    if ((see >> lane) & 1) acc[h] += exp2f((dot[h][a].x + dot[h][a].y) * p.scale_log2 - lse[warp * kWarpRows + a]);
                }
            }
        }
        sums[warp][lane] = acc[0];
        sums[warp][lane + 32] = acc[1];
        __syncthreads();
        if (tid < kTile && slots[tid] >= 0) {
            float w = c0 + tid < cur.r.len - cur.r.n && decay > 0.f ? weights[slots[tid]] * decay : 0.f;
            for (int x = 0; x < kWarps; ++x) w += sums[x][tid];
            weights[slots[tid]] = w;
        }
    }
}

constexpr int kScoreThreads = 128, kScorePerSm = 7;
constexpr int kScoreTile = kScoreThreads * 4;       // cached tokens a tile
// Rows on their way at once: 8 for 4 gain a microsecond where a small call has more (5 fp32 trees of 7 over <= 300, 21 rows,
// 19.0 us for 19.7) and lose one in large ones (32 over <= 8192, 8 rows, 88.5 for 87.5).
constexpr int kScoreRows = 4;
// Rows a place of the list: a tile of more is as many places, so that one long request among short ones is dealt out over
// the blocks as well.  With any number of rows a place, 63 requests of one token and one of 190 over 8192 (4 query heads a
// kv head) took 1564 us for 741, 127 and one of 300 4344 for 1333.
constexpr int kPlaceRows = 16;

struct ScoreTile {
    int s, head, tile;
};

// The sums of a thread's four tokens where the sum of one of the rows is NaN (a score of it is, or is infinite): what the
// row sees gets NaN, and what it does not see is left alone.  Sums that do not look at the mask cannot tell minus infinity
// for a token that is not seen from a score.
__device__ __noinline__ float4 sum_seen(const AttnParams &p, const ScoreTile &at) {
    const Request r = request_of(p, at.s);
    const int c = at.tile * kScoreTile + threadIdx.x * 4;
    float w[4] = {};
    for (int row = 0; row < r.n * p.group; ++row) {
        const int i = row / p.group;
        const long long line = (long long)(r.begin + i) * p.n_q + at.head * p.group + row - i * p.group;
        const float4 s = *reinterpret_cast<const float4 *>(p.scores + line * p.ld_scores + c);
        const float lse = p.lse[line], scores[4] = {s.x, s.y, s.z, s.w};
        const uint32_t see = seen_word(p, r, i, c & ~31) >> (c & 31);
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if ((see >> x) & 1) w[x] += exp2_fast(scores[x] - lse);
    }
    return make_float4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(kScoreThreads, kScorePerSm) weigh_scores_kernel(const AttnParams p, float *weights, float decay) {
    static_assert(kScoreThreads >= kScanThreads, "start_block");
    __shared__ ScanShared scan;
    __shared__ ScoreTile tiles[kScoreThreads / 32];       // each warp's, for sum_seen
    Cursor at;
    KeyCursor cur;
    const uint32_t total = start_block<kPlain, false>(p, scan, at);
    cur.start(p, scan, total);
    const bool drop = total > (uint32_t)p.grid;
    // A tile's page ids, then its slots (-1: none) and what its weights were: two round trips, both a tile ahead and the
    // first before the attention's last kernel is done.
    int page[4], slot[4];
    float old[4];
    const bool whole = p.page_shift >= 2;        // a thread's four tokens are in one page
    auto fetch_pages = [&](const KeyCursor &c) {
        const int c0 = c.tile * kScoreTile + threadIdx.x * 4;
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if ((x == 0 || !whole) && c.left > 0 && c0 + x < c.r.len) page[x] = page_of(p, c.s, c.r, c0 + x);
    };
    auto fetch_weights = [&](const KeyCursor &c) {
        const int c0 = c.tile * kScoreTile + threadIdx.x * 4, prefix = c.r.len - c.r.n;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            slot[x] = -1;
            old[x] = 0.f;
            const int at = whole ? page[0] : page[x];
            if (c.left <= 0 || c0 + x >= c.r.len) continue;
            if (at >= 0 && at < p.n_pages) slot[x] = ((at * p.n_kv + c.head) << p.page_shift) + ((c0 + x) & ((1 << p.page_shift) - 1));
            else flag_status(p.status, LORA_DEV_BAD_PAGE);
        }
        if (!(decay > 0.f)) return;
        if (whole && slot[3] >= 0 && c0 + 4 <= prefix) {
            *reinterpret_cast<float4 *>(old) = *reinterpret_cast<const float4 *>(weights + slot[0]);
            return;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (slot[x] >= 0 && c0 + x < prefix) old[x] = weights[slot[x]];
    };
    fetch_pages(cur);
    fetch_weights(cur);
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    if (!*p.computed) return;
    while (cur.left > 0) {
        const int c = cur.tile * kScoreTile + threadIdx.x * 4;
        const int rows = c - (int)(threadIdx.x & 31) * 4 < cur.r.len ? cur.r.n * p.group : 0;       // of the whole warp
        const bool inside = c < cur.r.len;
        // rows of a kv head lie group by group of n_q rows: the place of the next one, and its head in the group
        struct Place {
            const float *scores, *sums;
            int g;
            __device__ __forceinline__ void next(const AttnParams &p) {
                scores += p.ld_scores;
                ++sums;
                if (++g == p.group) {
                    g = 0;
                    scores += (p.n_q - p.group) * p.ld_scores;
                    sums += p.n_q - p.group;
                }
            }
        } ahead = {p.scores + ((long long)cur.r.begin * p.n_q + cur.head * p.group) * p.ld_scores + c,
                   p.lse + (long long)cur.r.begin * p.n_q + cur.head * p.group, 0};
        Place done = ahead;
        float4 s[kScoreRows] = {};
        float lse[kScoreRows] = {}, w[4] = {};
        auto load = [&](int row0) {
#pragma unroll
            for (int x = 0; x < kScoreRows; ++x) {
                if (row0 + x >= rows) break;
                if (inside) s[x] = *reinterpret_cast<const float4 *>(ahead.scores);
                lse[x] = *ahead.sums;
                ahead.next(p);
            }
        };
        load(0);
        // drafted tokens among the warp's: rows differ in what they see of them
        const bool drafted = c + 128 - (int)(threadIdx.x & 31) * 4 > cur.r.len - cur.r.n;
        if (drafted) {
            __syncwarp();
            if ((threadIdx.x & 31) == 0) tiles[threadIdx.x >> 5] = {cur.s, cur.head, cur.tile};
            __syncwarp();
        }
        cur.advance(p);
        fetch_pages(cur);
        for (int row0 = 0; row0 < rows; row0 += kScoreRows) {
#pragma unroll
            for (int x = 0; x < kScoreRows; ++x) {
                if (row0 + x >= rows) break;
                w[0] += exp2_fast(s[x].x - lse[x]);
                w[1] += exp2_fast(s[x].y - lse[x]);
                w[2] += exp2_fast(s[x].z - lse[x]);
                w[3] += exp2_fast(s[x].w - lse[x]);
            }
            if (row0 + kScoreRows < rows) load(row0 + kScoreRows);
            // the scores are not needed again: their lines leave L2 without being written to memory (2 over 131072: 142 ->
            // 135 us; one over 777 would take 15.0 us for 14.2)
            if (drop && !drafted) {
                __syncwarp();
#pragma unroll
                for (int x = 0; x < kScoreRows; ++x) {
                    if (row0 + x >= rows) break;
                    if (inside && (threadIdx.x & 7) == 0) asm volatile("discard.global.L2 [%0], 128;\n" ::"l"(done.scores) : "memory");
                    done.next(p);
                }
            }
        }
        if (drafted && w[0] != w[0] && inside) {         // such a row makes NaN of any token's sum
            const float4 seen = sum_seen(p, tiles[threadIdx.x >> 5]);
            w[0] = seen.x;
            w[1] = seen.y;
            w[2] = seen.z;
            w[3] = seen.w;
        }
        int to[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            w[x] += old[x] * decay;
            to[x] = slot[x];
        }
        fetch_weights(cur);
        if (whole && to[3] >= 0) {
            *reinterpret_cast<float4 *>(weights + to[0]) = make_float4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (to[x] >= 0) weights[to[x]] = w[x];
        }
    }
}

}  // namespace

namespace decode {

int plan_weigh(const lora_kv_pages *kv, const AttnParams &attention, AttnParams &p) {
    p = attention;
    const bool tc = !p.scores && kv->dtype == LORA_BF16;
    p.rt = p.scores ? kPlaceRows : tc ? kWeighRows : kRows;
    p.tk = p.scores ? kScoreTile : tc ? kWeighTile : kTile;
    p.tk_shift = log2_of(p.tk);
    p.unit_cost = tc ? kWeighUnitCost : 0;
    const long long tiles = (long long)p.max_pages * kv->page_size / p.tk + 1 + p.unit_cost, units = (long long)p.T * p.group / p.rt + p.S;
    if (tiles * units > 0x7fffffffLL / p.n_kv) return LORA_ERR_SHAPE;
    p.max_places = (uint32_t)(tiles * units * p.n_kv);
    p.grid = num_sms() * (p.scores ? kScorePerSm : tc ? 1 : 2);
    return LORA_OK;
}

int launch_weigh(const lora_kv_pages *kv, const KvMaps *maps, const AttnParams &p, float *weights, float decay, cudaStream_t st) {
    if (!p.scores && kv->dtype == LORA_BF16) return launch_weigh_tc(maps, p, weights, decay, st);
    void (*const kernel)(AttnParams, float *, float) = p.scores ? weigh_scores_kernel : weigh_kernel;
    const size_t smem = p.scores ? 0 : (size_t)(kTile + kRows) * (p.d + 4) * sizeof(float);
    if (smem && smem_optin(reinterpret_cast<const void *>(kernel), smem)) return LORA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.grid);
    cfg.blockDim = dim3(p.scores ? kScoreThreads : kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p, weights, decay);
    count_launch();
    return launch_status(e);
}

}  // namespace decode
}  // namespace lora
