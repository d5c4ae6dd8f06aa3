// Eviction from a paged cache by accumulated attention weight (lora_kv_evict).
//
// Per request and kv head, of len cached tokens with scores f_c: the first `first` and the
// last `recent` stay, and of those between the k = keep - first - recent with the greatest
// (f_c, -c); the kept ones move, in order, to places 0 .. keep - 1.
//
// evict_select_kernel, a cluster (or one block) a (request, kv head) that loses tokens:
//   scores become whole numbers that order as they do (NaN lowest), 4 bytes a token in shared
//   memory; the k-th greatest is found 11 bits at a time from the top.  Up to kSolo tokens
//   one block does that, as waiting for one another costs more than it saves; of more, each
//   block has its share, and counts are added up.  Then a warp counts its tokens that stay,
//   the counts are scanned, and the sources of the kept tokens are written in order (ties by
//   their rank in the row).
// evict_move_kernel, a block a column range of one plane (keys, values, weights) of a pair:
//   a token's source is never before its destination, so a round of destinations
//   [j, j + n) is read whole before it is written: what a round overwrites, no later round
//   reads.  Column ranges move apart from one another, so blocks never wait for one another,
//   and the next rounds are on their way while one is written.
//
// Memory is the bound of large calls: 64 requests over <= 4352, 4096 kept, 8 heads of 128,
// 81 us for 388 MB (4.8 TB/s); the select is 17 of them (a block goes from barrier to barrier
// and from load to load), the rest the ranges' last rounds.  Small calls are chains: one
// request 1088 -> 1024 10.2 us, half of them the select's: lengths, page ids, scores, two or
// three passes of 0.7 to 1.4, the list.  Four of 32768 -> 2048: 36.7 us, half of them for
// passes over scores in clusters of four blocks.  In one kernel, a cluster a unit, the three
// took 117, 13.7 and 116 us: whole units are too large a piece to spread evenly.
#include "kv_copy.cuh"

namespace lora {
namespace {

using namespace decode;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBits = 11, kBins = 1 << kBits, kCoarse = 8;      // kCoarse bins side by side are counted together as well
constexpr int kMaxCluster = 8;
// Alone and in clusters of four, four requests, 8 heads of 128, 2048 kept: 2100 tokens 28.7 and 29.7 us, 4200 31.7 and
// 30.7, 8100 36.9 and 32.0, 16000 47.1 and 34.8; half of the tokens kept: 2100 22.5 and 24.4, 4200 32.8 and 30.7, 8100 51.2
// and 45.1, 16000 86.0 and 73.7 (events around a call, L2 flushed before it).
constexpr int kSolo = 4096;
constexpr int kMaxHeld = 16384;       // scores a block keeps in shared memory; more are read again

constexpr int kMoveThreads = 256;
constexpr int kStages = 3;            // rounds in shared memory
constexpr int kAhead = kStages - 1, kSlotRounds = kStages + 1;
constexpr int kSliceChunks = 8;       // at most, of 16 bytes
// 16-byte pieces a thread and round, and blocks a SM: long rounds where all ranges there can be run at once, else more
// blocks.  Four 32768 -> 2048 (128 ranges) 37.6 us with 8 pieces and two blocks, 43.4 with 5 and three; 64 requests over
// <= 4352 (368 ranges of 2048 that there could be) 99.6 and 81.
struct Few {
    static constexpr int kPieces = 8, kPerSm = 2;
};
struct Many {
    static constexpr int kPieces = 5, kPerSm = 3;
};
template <typename M>
constexpr size_t kMoveSmem = (size_t)kStages * M::kPieces * kMoveThreads * 16;

struct EvictParams {
    char *k, *v;
    const float *scores;
    float *weights;
    int S, n_kv, n_pages, page_shift, max_pages, row_bytes;
    const int *lens, *table, *keep;
    int first, recent, ld_kept, held;
    int slices;                       // column ranges of a row of keys (and of values)
    int places;                       // blocks that move at once
    int *kept, *new_lens, *status;
};

struct __align__(16) Shared {
    uint32_t bins[2][kBins], coarse[2][kBins / kCoarse];      // this block's counts, of two passes, read by its cluster
    uint32_t scan[kWarps];
    uint32_t sure[kWarps], equal[kWarps];     // tokens of each warp above the cut, and at it
    uint32_t block_sure, block_equal, bad;
    uint32_t cut, wanted, inside, group;      // a pass's bin: its keys' upper bits, how many are wanted of it, how many it has
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
__device__ __forceinline__ uint32_t peer_addr(const uint32_t *mine, uint32_t rank) {
    uint32_t addr;
    asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(addr) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(rank));
    return addr;
}
// Each lane's peer has a value (lanes from `blocks` on: 0); volatile, so that loads are on their way together.
__device__ __forceinline__ uint32_t peer_values(const uint32_t *mine, uint32_t blocks) {
    const uint32_t lane = threadIdx.x & 31;
    uint32_t value = 0;
    if (lane < blocks) asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(value) : "r"(peer_addr(mine, lane)));
    __syncwarp();
    return value;
}
// Sum over the blocks.
__device__ __forceinline__ uint32_t peer_sum(const uint32_t *mine, uint32_t blocks) {
    uint32_t part[kMaxCluster], sum = 0;
#pragma unroll
    for (uint32_t r = 0; r < kMaxCluster; ++r) {
        part[r] = 0;
        if (r < blocks) asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(part[r]) : "r"(peer_addr(mine, r)));
    }
#pragma unroll
    for (uint32_t r = 0; r < kMaxCluster; ++r) sum += part[r];
    return sum;
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

// Inclusive sum over the warp.
__device__ __forceinline__ uint32_t warp_scan(uint32_t v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t other = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += other;
    }
    return v;
}

// Whether a request loses tokens; bad: its length or budget is beyond its table.
__device__ __forceinline__ bool loses(const EvictParams &p, int len, int keep, bool &bad) {
    const bool shorter = keep >= 0 && len > keep;
    bad = len < 0 || len > ((long long)p.max_pages << p.page_shift) || (shorter && keep > p.ld_kept);
    return shorter && !bad;
}

// The sources of one request and kv head.
__device__ void select(const EvictParams &p, Shared &sh, uint32_t *keys, int s, int head, uint32_t blocks, uint32_t rank) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int len = p.lens[s], keep = p.keep[s];
    const Row row = {p.table + (long long)s * p.max_pages, head};
    const int recent = min(p.recent, keep), first = min(p.first, keep - recent);
    const int last = len - recent;                                  // tokens from here on stay
    const bool solo = len <= kSolo || blocks == 1;
    if (solo && rank) return;
    // this block's tokens, and of those this warp's
    const int each = solo ? len : (((len + blocks - 1) / blocks) + 31) & ~31;
    const int lo = solo ? 0 : min(len, (int)rank * each), hi = min(len, lo + each), held = min(hi, lo + p.held);
    const int per_warp = (((each + 31) / 32 + kWarps - 1) / kWarps) * 32;
    const int w_lo = min(hi, lo + warp * per_warp), w_hi = min(hi, w_lo + per_warp);

    // a page outside the cache counts as 0 here, and in the end the request stays as it is
    bool bad = false;
    auto place = [&](int c, bool &outside) {
        const int page = __ldg(row.table + (c >> p.page_shift));
        outside = page < 0 || page >= p.n_pages;
        return (((outside ? 0 : page) * p.n_kv + head) << p.page_shift) + (c & ((1 << p.page_shift) - 1));
    };
    __syncthreads();                  // the unit before has read what is written here
    if (p.page_shift >= 2) {
#pragma unroll 4
        for (int c = lo + tid * 4; c < held; c += kThreads * 4) {
            bool outside;
            const int at = place(c, outside);
            bad |= outside;
            if (c + 4 <= held) {
                const float4 f = *reinterpret_cast<const float4 *>(p.scores + at);
                *reinterpret_cast<uint4 *>(keys + (c - lo)) = make_uint4(key_of(f.x), key_of(f.y), key_of(f.z), key_of(f.w));
            } else {
                for (int x = 0; c + x < held; ++x) keys[c + x - lo] = key_of(p.scores[at + x]);
            }
        }
    } else {
#pragma unroll 4
        for (int c = lo + tid; c < held; c += kThreads) {
            bool outside;
            keys[c - lo] = key_of(p.scores[place(c, outside)]);
            bad |= outside;
        }
    }
    for (int x = (held >> p.page_shift) + tid; held < hi && x < (hi + (1 << p.page_shift) - 1) >> p.page_shift; x += kThreads) {
        bool outside;
        place(min(x << p.page_shift, hi - 1), outside);
        bad |= outside;
    }
    auto key_at = [&](int c) {
        bool outside;
        return c < held ? keys[c - lo] : key_of(p.scores[place(c, outside)]);
    };
    bad = __syncthreads_or(bad);

    // the k-th greatest key of the tokens that compete: its upper bits as far as they are needed
    uint32_t wanted = keep - first - recent, cut = 0, mask = 0;
    if (wanted == 0) cut = mask = ~0u;       // nobody: no key is above, and of those equal none is wanted
    for (int shift = 32 - kBits, turn = 0; mask != ~0u; shift = max(0, shift - kBits), turn ^= 1) {
        // the buffer of the pass before the last: a cluster's barrier later, its peers have read it
        uint32_t *all_bins = sh.bins[turn], *coarse = sh.coarse[turn];
        const int width = shift == 0 ? 32 - 2 * kBits : kBits, bins = 1 << width;
        for (int x = tid; x < bins; x += kThreads) all_bins[x] = 0;
        if (tid == 0) {
            sh.cut = cut;
            sh.wanted = sh.inside = wanted;
            sh.group = 0;
        }
        __syncthreads();
        for (int c = max(lo, first) + tid; c < min(hi, last); c += kThreads) {
            const uint32_t key = key_at(c);
            if ((key & mask) == cut) atomicAdd(&all_bins[(key >> shift) & (bins - 1)], 1u);
        }
        __syncthreads();
        const int groups = bins / kCoarse;
        uint32_t sum = 0;
        if (tid < groups) {                 // a group of bins a thread, from the top
            const uint4 *bin = reinterpret_cast<const uint4 *>(all_bins + (groups - 1 - tid) * kCoarse);
            const uint4 u = bin[0], v = bin[1];
            sum = ((u.x + u.y) + (u.z + u.w)) + ((v.x + v.y) + (v.z + v.w));
        }
        if (!solo) {
            if (tid < groups) coarse[tid] = sum;
            cluster_sync();
            if (tid < groups) sum = peer_sum(coarse + tid, blocks);
        }
        // from the top down: the group, then its bin, in which the count passes `wanted`
        const uint32_t upto = warp_scan(sum);
        if (lane == 31) sh.scan[warp] = upto;
        __syncthreads();
        uint32_t before = upto - sum;
        for (int w = 0; w < warp && w < (groups + 31) / 32; ++w) before += sh.scan[w];
        if (tid < groups && before < wanted && before + sum >= wanted) {
            sh.group = groups - 1 - tid;
            sh.wanted = wanted - before;
        }
        __syncthreads();
        if (warp == 0) {
            const int bin = sh.group * kCoarse + kCoarse - 1 - (lane & (kCoarse - 1));
            const uint32_t left = sh.wanted, n = solo ? all_bins[bin] : peer_sum(all_bins + bin, blocks);
            uint32_t to = n;
#pragma unroll
            for (int o = 1; o < kCoarse; o <<= 1) {
                const uint32_t other = __shfl_up_sync(0xffffffffu, to, o, kCoarse);
                if ((lane & (kCoarse - 1)) >= o) to += other;
            }
            __syncwarp();
            if (lane < kCoarse && to - n < left && to >= left) {
                sh.cut = cut | (uint32_t)bin << shift;
                sh.wanted = left - (to - n);
                sh.inside = n;
            }
        }
        __syncthreads();
        cut = sh.cut;
        wanted = sh.wanted;
        mask |= (uint32_t)(bins - 1) << shift;
        const bool all = sh.inside == wanted;       // the whole bin stays: its keys need no order
        __syncthreads();
        if (all) break;
    }

    // how many stay before each warp's tokens
    uint32_t sure = 0, equal = 0;
    for (int c0 = w_lo; c0 < w_hi; c0 += 32) {
        const int c = c0 + lane;
        const bool in = c < w_hi, safe = in && (c < first || c >= last);
        const uint32_t key = in ? key_at(c) & mask : 0u;
        sure += __popc(__ballot_sync(0xffffffffu, safe || (in && key > cut)));
        equal += __popc(__ballot_sync(0xffffffffu, in && !safe && key == cut));
    }
    if (lane == 0) {
        sh.sure[warp] = sure;
        sh.equal[warp] = equal;
    }
    __syncthreads();
    uint32_t sure_before = 0, equal_before = 0;
    if (!solo) {
        if (warp == 0) {
            const uint32_t a = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.sure[lane] : 0u);
            const uint32_t b = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.equal[lane] : 0u);
            if (lane == 0) {
                sh.block_sure = a;
                sh.block_equal = b;
                sh.bad = bad;
            }
        }
        cluster_sync();
        sure_before = __reduce_add_sync(0xffffffffu, peer_values(&sh.block_sure, rank));
        equal_before = __reduce_add_sync(0xffffffffu, peer_values(&sh.block_equal, rank));
        bad = __any_sync(0xffffffffu, peer_values(&sh.bad, blocks) != 0);
        cluster_sync();                      // no block leaves while its shared memory is read
    }
    if (bad) {
        if (head == 0 && rank == 0 && tid == 0) {
            flag_status(p.status, LORA_DEV_BAD_PAGE);
            p.new_lens[s] = len;
        }
        return;
    }
    for (int w = 0; w < warp; ++w) {
        sure_before += sh.sure[w];
        equal_before += sh.equal[w];
    }
    // the sources of the kept tokens, in order
    int *kept = p.kept + ((long long)s * p.n_kv + head) * p.ld_kept;
    for (int c0 = w_lo; c0 < w_hi; c0 += 32) {
        const int c = c0 + lane;
        const bool in = c < w_hi, safe = in && (c < first || c >= last);
        const uint32_t key = in ? key_at(c) & mask : 0u;
        const uint32_t above = __ballot_sync(0xffffffffu, safe || (in && key > cut));
        const uint32_t at = __ballot_sync(0xffffffffu, in && !safe && key == cut), before = (1u << lane) - 1;
        const uint32_t rank_at = equal_before + __popc(at & before);
        const uint32_t place = sure_before + __popc(above & before) + min(rank_at, wanted);
        const bool stays = ((above >> lane) & 1) || (((at >> lane) & 1) && rank_at < wanted);
        if (stays && place < (uint32_t)keep) kept[place] = c;       // below keep always, unless scores change under the call
        sure_before += __popc(above);
        equal_before += __popc(at);
    }
    if (rank == 0 && head == 0 && tid == 0) p.new_lens[s] = keep;
}

// Calls f(request, unit) for the units, n a request, of the requests for which active(s) holds: the one `turn` units
// from here and every `workers`-th after it.  Returns what is left of `turn`.
template <int THREADS, typename A, typename F>
__device__ __forceinline__ long long in_turn(int S, int n, long long turn, int workers, A active, F f) {
    __shared__ int requests[THREADS], counts[THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int s0 = 0; s0 < S; s0 += THREADS) {
        const int s = s0 + tid;
        const bool mine = s < S && active(s);
        const uint32_t on = __ballot_sync(0xffffffffu, mine);
        __syncthreads();
        if (lane == 0) counts[warp] = __popc(on);
        __syncthreads();
        int at = __popc(on & ((1u << lane) - 1)), count = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) at += counts[w];
            count += counts[w];
        }
        if (mine) requests[at] = s;
        __syncthreads();
        for (; turn < (long long)count * n; turn += workers) f(requests[turn / n], (int)(turn % n));
        turn -= (long long)count * n;
    }
    return turn;
}

__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictParams p) {
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ Shared sh;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const uint32_t blocks = cluster_size(), rank = cluster_rank();
    const int cluster = blockIdx.x / blocks;
    if ((long long)p.S * p.n_kv <= gridDim.x / blocks) {       // a cluster for every unit there can be
        const int s = cluster / p.n_kv, head = cluster - s * p.n_kv, len = p.lens[s];
        bool bad = false;
        if (loses(p, len, p.keep[s], bad)) {
            select(p, sh, keys, s, head, blocks, rank);
        } else if (head == 0 && rank == 0 && threadIdx.x == 0) {
            p.new_lens[s] = len;
            if (bad) flag_status(p.status, LORA_DEV_BAD_LENGTH);
        }
        return;
    }
    // more units than clusters: blocks by themselves
    in_turn<kThreads>(
        p.S, p.n_kv, blockIdx.x, gridDim.x,
        [&](int s) {
            bool bad = false;
            const int len = p.lens[s];
            const bool active = loses(p, len, p.keep[s], bad);
            if (!active && blockIdx.x == 0) {
                p.new_lens[s] = len;
                if (bad) flag_status(p.status, LORA_DEV_BAD_LENGTH);
            }
            return active;
        },
        [&](int s, int head) { select(p, sh, keys, s, head, 1, 0); });
}

// What evict_select_kernel left, once it is done.
__device__ __forceinline__ int new_len(const EvictParams &p, int s) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    return *(volatile int *)(p.new_lens + s);
}

// Moves a column range of `width` 16-byte chunks of one plane of a request and kv head.  A thread looks up one row of
// a round: its source's index two rounds before its slots, those a round before the copies, which are two rounds ahead
// of the stores.
template <int kPieces>
__device__ void move_range(const EvictParams &p, int s, char *plane, const Row &row, const int *kept, int keep, int len, int first, int width,
                           uint4 *ring, int2 (*slots)[kMoveThreads]) {
    const int tid = threadIdx.x, per_pass = kMoveThreads / width, pieces = min(kPieces, kMoveThreads / per_pass), round = per_pass * pieces;
    const int rounds = (keep + round - 1) / round;
    const int my_row = tid < per_pass * width ? tid / width : -1;
    char *column = plane + (first + tid % width) * 16;
    uint4 *mine = ring + tid;
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(mine);
    auto index = [&](int i) {                            // source of this thread's row of round i, -1: none
        const int j = i * round + tid;
        return tid < round && j < keep ? (int)min((uint32_t)kept[j], (uint32_t)len - 1) : -1;
    };
    auto places = [&](int i, int src) {                  // slots it moves between; .x -1: it does not
        const int j = i * round + tid;
        return src < 0 || src == j ? make_int2(-1, 0) : make_int2(row.slot(p, src), row.slot(p, j));
    };
    auto load = [&](int i) {
        const int2 *at = slots[i % kSlotRounds];
        const uint32_t dst = base + (i % kStages) * (kPieces * kMoveThreads * 16);
        if (i < rounds && my_row >= 0)
#pragma unroll
            for (int x = 0; x < kPieces; ++x)
                if (x < pieces) {
                    const int from = at[x * per_pass + my_row].x;
                    if (from >= 0) cp_async16(dst + x * (kMoveThreads * 16), column + (long long)from * p.row_bytes, true);
                }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
    __syncthreads();                                     // the range before has read its slots
    int2 next;
    int src;
    {
        int at[kAhead + 1];
        const int now = new_len(p, s);
#pragma unroll
        for (int i = 0; i <= kAhead; ++i) at[i] = index(i);
        if (now != keep) return;                         // a page outside the cache: there are no sources
#pragma unroll
        for (int i = 0; i < kAhead; ++i) slots[i][tid] = places(i, at[i]);
        next = places(kAhead, at[kAhead]);
        src = index(kAhead + 1);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i);
    for (int i = 0; i < rounds; ++i) {
        slots[(i + kAhead) % kSlotRounds][tid] = next;
        next = places(i + kAhead + 1, src);
        src = index(i + kAhead + 2);
        asm volatile("cp.async.wait_group %0;\n" ::"n"(kAhead - 1) : "memory");
        __syncthreads();                                 // round i has been read
        if (my_row >= 0) {
            const int2 *at = slots[i % kSlotRounds];
            const uint4 *data = mine + (i % kStages) * (kPieces * kMoveThreads);
#pragma unroll
            for (int x = 0; x < kPieces; ++x)
                if (x < pieces) {
                    const int2 to = at[x * per_pass + my_row];
                    if (to.x >= 0) *reinterpret_cast<uint4 *>(column + (long long)to.y * p.row_bytes) = data[x * kMoveThreads];
                }
        }
        load(i + kAhead);
    }
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
}

template <int kPieces>
__device__ void move_weights(const EvictParams &p, int s, const Row &row, const int *kept, int keep, int len) {
    const int tid = threadIdx.x;
    if (new_len(p, s) != keep) return;
    for (int j0 = 0; j0 < keep; j0 += kMoveThreads * kPieces) {
        float w[kPieces];
        int src[kPieces];
#pragma unroll
        for (int x = 0; x < kPieces; ++x) {
            const int j = j0 + x * kMoveThreads + tid;
            src[x] = j < keep ? (int)min((uint32_t)kept[j], (uint32_t)len - 1) : -1;
        }
#pragma unroll
        for (int x = 0; x < kPieces; ++x) w[x] = src[x] >= 0 ? p.weights[row.slot(p, src[x])] : 0.f;
        __syncthreads();
#pragma unroll
        for (int x = 0; x < kPieces; ++x) {
            const int j = j0 + x * kMoveThreads + tid;
            if (src[x] >= 0) p.weights[row.slot(p, j)] = w[x];
        }
    }
}

template <typename M>
__global__ void __launch_bounds__(kMoveThreads, M::kPerSm) evict_move_kernel(const EvictParams p) {
    extern __shared__ __align__(16) uint4 ring[];         // [kStages][M::kPieces][kMoveThreads]: each thread's own
    __shared__ int2 slots[kSlotRounds][kMoveThreads];
    const int chunks = p.row_bytes >> 4, workers = gridDim.x;
    // which requests is known before the sources are; that all pages of one are in the cache, with them
    auto active = [&](int s) {
        bool bad;
        return loses(p, p.lens[s], p.keep[s], bad);
    };
    // 128 bytes a range; where that would leave half of the blocks without one, 64 (if both halves are whole sectors): one
    // request 1088 -> 1024, 8 heads of 128, 10.2 us for 11.4, four 32768 -> 2048 36.7 for 37.6; but 64 over <= 4352 102 for
    // 93, as memory is read in smaller pieces
    long long units = (long long)p.S * p.n_kv;
    const int more = p.weights ? 1 : 0;
    bool direct = units * (2 * p.slices + more) <= p.places;       // a block for every range there can be
    if (!direct) {
        units = 0;
        for (int s0 = 0; s0 < p.S; s0 += kMoveThreads) units += __syncthreads_count(s0 + (int)threadIdx.x < p.S && active(s0 + threadIdx.x));
        units *= p.n_kv;
    }
    const int slices = chunks == p.slices * kSliceChunks && units * p.slices * 4 <= p.places ? 2 * p.slices : p.slices;
    const int parts = 2 * slices;
    direct = direct && units * (parts + more) <= workers;
    auto range = [&](int s, int unit) {
        const int head = unit / parts, part = unit - head * parts;
        const Row row = {p.table + (long long)s * p.max_pages, head};
        const int slice = part % slices, first = chunks * slice / slices, width = chunks * (slice + 1) / slices - first;
        move_range<M::kPieces>(p, s, part < slices ? p.k : p.v, row, p.kept + ((long long)s * p.n_kv + head) * p.ld_kept, p.keep[s], p.lens[s],
                               first, width, ring, slots);
    };
    auto weights = [&](int s, int head) {
        move_weights<8>(p, s, {p.table + (long long)s * p.max_pages, head}, p.kept + ((long long)s * p.n_kv + head) * p.ld_kept, p.keep[s],
                        p.lens[s]);
    };
    if (direct) {
        const int each = p.n_kv * (parts + more), s = blockIdx.x / each, unit = blockIdx.x - s * each;
        if (s < p.S && active(s)) {
            if (unit < p.n_kv * parts) range(s, unit);
            else weights(s, unit - p.n_kv * parts);
        }
    } else {
        const long long turn = in_turn<kMoveThreads>(p.S, p.n_kv * parts, blockIdx.x, workers, active, range);
        if (p.weights) in_turn<kMoveThreads>(p.S, p.n_kv, turn, workers, active, weights);
    }
    asm volatile("griddepcontrol.wait;\n" ::: "memory");       // no grid ends before the one it depends on
}

template <typename M>
cudaError_t launch_move(EvictParams p, long long units, cudaStream_t st) {
    if (smem_optin(reinterpret_cast<const void *>(evict_move_kernel<M>), kMoveSmem<M>)) return cudaErrorInvalidValue;
    p.places = num_sms() * M::kPerSm;
    const long long tasks = units * (4 * p.slices + 1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tasks < p.places ? tasks : p.places));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.dynamicSmemBytes = kMoveSmem<M>;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_move_kernel<M>, p);
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" int lora_kv_evict(const lora_kv_pages *kv, const lora_eviction *a, lora_stream stream) {
    if (!a) return LORA_ERR_ARG;
    const float *const scores = a->scores;
    float *const weights = a->weights;
    const int *const kv_lens = a->kv_lens, *const page_table = a->page_table, *const keep = a->keep;
    int *const kept = a->kept, *const new_lens = a->new_lens;
    const int S = a->S, max_pages = a->max_pages, first = a->first, recent = a->recent, ld_kept = a->ld_kept;
    const int rc = decode::check_kv(kv, 0);
    if (rc) return rc;
    if (S < 0 || max_pages < 0 || first < 0 || recent < 0 || ld_kept < 0) return LORA_ERR_ARG;
    if ((long long)max_pages * kv->page_size > 0x7fffffffLL - 4096) return LORA_ERR_SHAPE;
    if ((long long)S * kv->n_kv_heads > 0x7fffffffLL / kMaxCluster) return LORA_ERR_SHAPE;
    if (S == 0) return LORA_OK;
    if (!scores || !kv_lens || !page_table || max_pages < 1 || !keep || !new_lens || (ld_kept && !kept)) return LORA_ERR_ARG;
    if (!aligned16(scores) || !aligned16(weights)) return LORA_ERR_ARG;
    if (((uintptr_t)kv_lens | (uintptr_t)page_table | (uintptr_t)keep | (uintptr_t)kept | (uintptr_t)new_lens) & 3u) return LORA_ERR_ARG;
    const size_t plane = (size_t)kv->n_pages * kv->n_kv_heads * kv->page_size * sizeof(float), row = (size_t)S * sizeof(int);
    if (weights && weights != scores && overlap(weights, plane, scores, plane)) return LORA_ERR_ARG;
    if (overlap(new_lens, row, kv_lens, row) || overlap(new_lens, row, keep, row)) return LORA_ERR_ARG;
    const size_t list = (size_t)S * kv->n_kv_heads * ld_kept * sizeof(int), table = (size_t)S * max_pages * sizeof(int);
    if (overlap(kept, list, kv_lens, row) || overlap(kept, list, keep, row) || overlap(kept, list, new_lens, row) ||
        overlap(kept, list, page_table, table) || overlap(new_lens, row, page_table, table) || overlap(kept, list, scores, plane) ||
        (weights && overlap(kept, list, weights, plane)))
        return LORA_ERR_ARG;
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
    const long long cap = (long long)max_pages * kv->page_size, units = (long long)S * p.n_kv;
    // clusters of several blocks only where all units there can be run at once: S and the table are what the host knows.
    // So one long request among many short ones has a block a head: of 131072 tokens, 8 heads, 2048 kept, by itself 45 us,
    // beside 7 of 1000 tokens 287 (two blocks), beside 15 574.
    int blocks = 1;
    while (cap > kSolo && blocks < kMaxCluster && units * blocks * 2 <= num_sms()) blocks *= 2;
    const long long share = ((cap + blocks - 1) / blocks + 31) & ~31LL, solo = ((cap < kSolo ? cap : kSolo) + 3) & ~3LL;
    p.held = (int)(share < solo ? solo : share < kMaxHeld ? share : kMaxHeld);
    const long long clusters = units < 4LL * num_sms() / blocks ? units : 4LL * num_sms() / blocks;
    const int chunks = p.row_bytes >> 4;
    p.slices = (chunks + kSliceChunks - 1) / kSliceChunks;
    const bool few = units * 2 * p.slices <= num_sms() * Few::kPerSm;
    if (smem_optin(reinterpret_cast<const void *>(evict_select_kernel), kMaxHeld * sizeof(uint32_t))) return LORA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = p.held * sizeof(uint32_t);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
    count_launch();
    if (e != cudaSuccess) return launch_status(e);
    e = few ? launch_move<Few>(p, units, (cudaStream_t)stream) : launch_move<Many>(p, units, (cudaStream_t)stream);
    count_launch();
    return launch_status(e);
}
