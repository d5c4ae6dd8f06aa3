// Eviction from a paged cache by accumulated attention weight (lora_kv_evict).
//
// Per request and kv head, of len cached tokens with scores f_c: the first `first` and the
// last `recent` stay, and of those between the k = keep - first - recent with the greatest
// (f_c, -c); the kept ones move, in order, to places 0 .. keep - 1.
//
// One cluster of blocks a (request, kv head):
//   select   scores become whole numbers that order as they do (NaN lowest), 4 bytes a token
//            in shared memory; the k-th greatest is found 11 bits at a time from the top, by
//            counts that the cluster's blocks add up; ties are cut by their rank in the row.
//   list     a warp counts its tokens that stay, the cluster scans the counts, and the
//            sources of the kept tokens are written in order.
//   move     a token's source is never before its destination, so a round of destinations
//            [j, j + n) is read whole, the cluster waits, and it is written: what a round
//            overwrites, no later round reads.  Tokens before the first evicted one stay.
#include "decode.cuh"

namespace lora {
namespace {

using namespace decode;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBits = 11, kBins = 1 << kBits;
constexpr int kMaxCluster = 8;
constexpr int kMaxHeld = 16384;       // scores a block keeps in shared memory; more are read again

struct EvictParams {
    char *k, *v;
    const float *scores;
    float *weights;
    int S, n_kv, n_pages, page_shift, max_pages, row_bytes;
    const int *lens, *table, *keep;
    int first, recent, ld_kept, held;
    int *kept, *new_lens, *status;
};

struct Shared {
    uint32_t bins[kBins];             // this block's counts, read by its cluster
    uint32_t scan[kWarps];
    uint32_t sure[kWarps], equal[kWarps];     // tokens of each warp above the cut, and at it
    uint32_t block_sure, block_equal, bad, hole;
    uint32_t cut, wanted;             // key of the last kept token; how many of that key are kept
};

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm("mov.u32 %0, %%cluster_nctaid.x;\n" : "=r"(n));
    return n;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}
// Every thread of the cluster; orders shared and global memory.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_load(const uint32_t *mine, uint32_t rank) {
    uint32_t addr, value;
    asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(addr) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(value) : "r"(addr) : "memory");
    return value;
}

// Orders as the scores do; -0 is 0, a NaN is below everything.
__device__ __forceinline__ uint32_t key_of(float f) {
    if (f != f) return 0u;
    const uint32_t u = __float_as_uint(f + 0.f);
    return u >> 31 ? ~u : u | 0x80000000u;
}

struct Row {                          // one request and kv head
    const int *table;
    int head;
    __device__ __forceinline__ int slot(const EvictParams &p, int c) const {
        return ((__ldg(table + (c >> p.page_shift)) * p.n_kv + head) << p.page_shift) + (c & ((1 << p.page_shift) - 1));
    }
};

__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictParams p) {
    extern __shared__ uint32_t keys[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t blocks = cluster_size(), rank = cluster_rank();
    const int unit = blockIdx.x / blocks, s = unit / p.n_kv, head = unit - s * p.n_kv;
    const long long cap = (long long)p.max_pages << p.page_shift;
    const int len = p.lens[s], keep = p.keep[s];
    if (len < 0 || len > cap || (keep >= 0 && len > keep && keep > p.ld_kept)) {
        // a length that the table does not hold, a budget that `kept` does not: the request stays as it is
        if (head == 0 && rank == 0 && tid == 0) {
            flag_status(p.status, LORA_DEV_BAD_LENGTH);
            p.new_lens[s] = len;
        }
        return;
    }
    if (keep < 0 || len <= keep) {
        if (head == 0 && rank == 0 && tid == 0) p.new_lens[s] = len;
        return;
    }
    const Row row = {p.table + (long long)s * p.max_pages, head};
    const int recent = min(p.recent, keep), first = min(p.first, keep - recent);
    const int last = len - recent;                                  // tokens from here on stay
    // this block's tokens, and of those this warp's
    const int each = (((len + blocks - 1) / blocks) + 31) & ~31;
    const int lo = min(len, (int)rank * each), hi = min(len, lo + each);
    const int per_warp = ((each / 32 + kWarps - 1) / kWarps) * 32;
    const int w_lo = min(hi, lo + warp * per_warp), w_hi = min(hi, w_lo + per_warp);

    // a page outside the cache: the request stays as it is
    if (tid == 0) sh.bad = 0;
    __syncthreads();
    const int pages = (len + (1 << p.page_shift) - 1) >> p.page_shift;
    bool bad = false;
    for (int x = tid; x < pages; x += kThreads) {
        const int page = __ldg(row.table + x);
        bad |= page < 0 || page >= p.n_pages;
    }
    if (__syncthreads_or(bad)) {            // every block of every head of the request finds the same
        if (head == 0 && rank == 0 && tid == 0) {
            flag_status(p.status, LORA_DEV_BAD_PAGE);
            p.new_lens[s] = len;
        }
        return;
    }
    for (int c = lo + tid; c < min(hi, lo + p.held); c += kThreads) keys[c - lo] = key_of(p.scores[row.slot(p, c)]);
    auto key_at = [&](int c) { return c - lo < p.held ? keys[c - lo] : key_of(p.scores[row.slot(p, c)]); };

    // the k-th greatest key of the tokens that compete
    uint32_t wanted = keep - first - recent, known = 0, mask = 0;
    if (wanted == 0) {
        known = mask = ~0u;                 // nobody: no key is above, and of those equal none is wanted
        __syncthreads();
    }
    for (int shift = 32 - kBits; wanted && mask != ~0u; shift = max(0, shift - kBits)) {
        const int width = shift == 0 ? 32 - 2 * kBits : kBits, bins = 1 << width;
        for (int x = tid; x < bins; x += kThreads) sh.bins[x] = 0;
        if (tid == 0) {
            sh.cut = known;
            sh.wanted = wanted;
        }
        __syncthreads();
        for (int c = max(lo, first) + tid; c < min(hi, last); c += kThreads) {
            const uint32_t key = key_at(c);
            if ((key & mask) == known) atomicAdd(&sh.bins[(key >> shift) & (bins - 1)], 1u);
        }
        cluster_sync();
        // from the top bin down: the bin in which the count passes `wanted`
        const int per = bins / kThreads;    // 4 or 2 bins a thread, from the top
        uint32_t mine[kBins / kThreads], sum = 0;
#pragma unroll
        for (int x = 0; x < kBins / kThreads; ++x) {
            mine[x] = 0;
            if (x < per)
                for (uint32_t r = 0; r < blocks; ++r) mine[x] += peer_load(&sh.bins[bins - 1 - (tid * per + x)], r);
            sum += mine[x];
        }
        uint32_t upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t other = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += other;
        }
        if (lane == 31) sh.scan[warp] = upto;
        __syncthreads();
        uint32_t before = upto - sum;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            if (w < warp) before += sh.scan[w];
#pragma unroll
        for (int x = 0; x < kBins / kThreads; ++x) {
            if (x < per && before < wanted && before + mine[x] >= wanted) {
                sh.cut = known | (uint32_t)(bins - 1 - (tid * per + x)) << shift;
                sh.wanted = wanted - before;
            }
            before += mine[x];
        }
        cluster_sync();                     // also: the peers have read this block's bins
        known = sh.cut;
        wanted = sh.wanted;
        mask |= (uint32_t)(bins - 1) << shift;
    }
    const uint32_t cut = known;

    // how many stay before each warp's tokens
    uint32_t sure = 0, equal = 0;
    for (int c0 = w_lo; c0 < w_hi; c0 += 32) {
        const int c = c0 + lane;
        const bool in = c < w_hi, safe = in && (c < first || c >= last);
        const uint32_t key = in ? key_at(c) : 0u;
        sure += __popc(__ballot_sync(0xffffffffu, safe || (in && key > cut)));
        equal += __popc(__ballot_sync(0xffffffffu, in && !safe && key == cut));
    }
    if (lane == 0) {
        sh.sure[warp] = sure;
        sh.equal[warp] = equal;
    }
    if (tid == 0) sh.hole = 0xffffffffu;
    __syncthreads();
    if (tid == 0) {
        uint32_t a = 0, b = 0;
        for (int w = 0; w < kWarps; ++w) {
            a += sh.sure[w];
            b += sh.equal[w];
        }
        sh.block_sure = a;
        sh.block_equal = b;
    }
    cluster_sync();
    uint32_t sure_before = 0, equal_before = 0;
    for (uint32_t r = 0; r < rank; ++r) {
        sure_before += peer_load(&sh.block_sure, r);
        equal_before += peer_load(&sh.block_equal, r);
    }
    for (int w = 0; w < warp; ++w) {
        sure_before += sh.sure[w];
        equal_before += sh.equal[w];
    }
    // the sources of the kept tokens, in order
    int *kept = p.kept + ((long long)s * p.n_kv + head) * p.ld_kept;
    uint32_t hole = 0xffffffffu;
    for (int c0 = w_lo; c0 < w_hi; c0 += 32) {
        const int c = c0 + lane;
        const bool in = c < w_hi, safe = in && (c < first || c >= last);
        const uint32_t key = in ? key_at(c) : 0u;
        const uint32_t above = __ballot_sync(0xffffffffu, safe || (in && key > cut));
        const uint32_t at = __ballot_sync(0xffffffffu, in && !safe && key == cut), before = (1u << lane) - 1;
        const uint32_t rank_at = equal_before + __popc(at & before);
        const uint32_t place = sure_before + __popc(above & before) + min(rank_at, wanted);
        if (((above >> lane) & 1) || (((at >> lane) & 1) && rank_at < wanted)) {
            if (place < (uint32_t)keep) kept[place] = c;       // always, unless scores change under the call
        } else if (in) hole = min(hole, (uint32_t)c);
        sure_before += __popc(above);
        equal_before += __popc(at);
    }
    hole = __reduce_min_sync(0xffffffffu, hole);
    if (lane == 0 && hole != 0xffffffffu) atomicMin(&sh.hole, hole);
    cluster_sync();                          // the list is complete, and the scores have been read
    uint32_t from = 0xffffffffu;
    for (uint32_t r = 0; r < blocks; ++r) from = min(from, peer_load(&sh.hole, r));
    cluster_sync();                          // no block leaves while its shared memory is read
    if (rank == 0 && head == 0 && tid == 0) p.new_lens[s] = keep;

    // the move, up to 32 KB of keys and as much of values a block and round
    auto source = [&](int j) { return (int)min((uint32_t)kept[j], (uint32_t)len - 1); };
    constexpr int kPieces = 4;
    const int chunks = p.row_bytes >> 4, rows = min(kThreads, kThreads * kPieces / chunks);
    for (long long j0 = from; j0 < keep; j0 += (long long)rows * blocks) {
        uint4 k[kPieces], v[kPieces];
        float w = 0.f;
        const int begin = (int)min((long long)keep, j0 + (long long)rank * rows), count = min(rows, keep - begin);
#pragma unroll
        for (int x = 0; x < kPieces; ++x) {
            const int piece = x * kThreads + tid, j = piece / chunks;
            if (j < count) {
                const long long at = (long long)row.slot(p, source(begin + j)) * p.row_bytes + (piece - j * chunks) * 16;
                k[x] = *reinterpret_cast<const uint4 *>(p.k + at);
                v[x] = *reinterpret_cast<const uint4 *>(p.v + at);
            }
        }
        if (p.weights && tid < count) w = p.weights[row.slot(p, source(begin + tid))];
        cluster_sync();
#pragma unroll
        for (int x = 0; x < kPieces; ++x) {
            const int piece = x * kThreads + tid, j = piece / chunks;
            if (j < count) {
                const long long at = (long long)row.slot(p, begin + j) * p.row_bytes + (piece - j * chunks) * 16;
                *reinterpret_cast<uint4 *>(p.k + at) = k[x];
                *reinterpret_cast<uint4 *>(p.v + at) = v[x];
            }
        }
        if (p.weights && tid < count) p.weights[row.slot(p, begin + tid)] = w;
    }
}

// Blocks of a cluster: as many as let every block have a place on the SMs at once.
int cluster_of(int S, int n_kv) {
    int n = kMaxCluster;
    while (n > 1 && (long long)S * n_kv * n > 2LL * num_sms()) n >>= 1;
    return n;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" int lora_kv_evict(const lora_kv_pages *kv, const float *scores, float *weights, int S, const int *kv_lens,
                             const int *page_table, int max_pages, const int *keep, int first, int recent, int *kept,
                             int ld_kept, int *new_lens, lora_stream stream) {
    const int rc = decode::check_kv(kv, 0);
    if (rc) return rc;
    if (S < 0 || max_pages < 0 || first < 0 || recent < 0 || ld_kept < 0) return LORA_ERR_ARG;
    if ((long long)max_pages * kv->page_size > 0x7fffffffLL - 4096) return LORA_ERR_SHAPE;
    if ((long long)S * kv->n_kv_heads > 0x7fffffffLL / kMaxCluster) return LORA_ERR_SHAPE;
    if (S == 0) return LORA_OK;
    if (!scores || !kv_lens || !page_table || max_pages < 1 || !keep || !new_lens || (ld_kept && !kept)) return LORA_ERR_ARG;
    if (((uintptr_t)scores | (uintptr_t)weights | (uintptr_t)kv_lens | (uintptr_t)page_table | (uintptr_t)keep |
         (uintptr_t)kept | (uintptr_t)new_lens) & 3u)
        return LORA_ERR_ARG;
    const size_t plane = (size_t)kv->n_pages * kv->n_kv_heads * kv->page_size * sizeof(float), row = (size_t)S * sizeof(int);
    if (weights && weights != scores && overlap(weights, plane, scores, plane)) return LORA_ERR_ARG;
    if (overlap(new_lens, row, kv_lens, row) || overlap(new_lens, row, keep, row)) return LORA_ERR_ARG;
    if (num_sms() < 1) return LORA_ERR_CUDA;
    EvictParams p;
    p.k = static_cast<char *>(kv->k);
    p.v = static_cast<char *>(kv->v);
    p.scores = scores;
    p.weights = weights;
    p.S = S;
    p.n_kv = kv->n_kv_heads;
    p.n_pages = kv->n_pages;
    p.page_shift = decode::log2_of(kv->page_size);
    p.max_pages = max_pages;
    p.row_bytes = kv->head_dim * (kv->dtype == LORA_BF16 ? 2 : 4);
    p.lens = kv_lens;
    p.table = page_table;
    p.keep = keep;
    p.first = first;
    p.recent = recent;
    p.ld_kept = ld_kept;
    p.kept = kept;
    p.new_lens = new_lens;
    p.status = kv->status;
    const int blocks = cluster_of(S, p.n_kv);
    const long long most = ((((long long)max_pages * kv->page_size + blocks - 1) / blocks) + 31) & ~31LL;     // tokens a block
    p.held = (int)(most < kMaxHeld ? most : kMaxHeld);
    if (smem_optin(reinterpret_cast<const void *>(evict_kernel), kMaxHeld * sizeof(uint32_t))) return LORA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)S * p.n_kv * blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = p.held * sizeof(uint32_t);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_kernel, p);
    count_launch();
    return cuda_status(e);
}
