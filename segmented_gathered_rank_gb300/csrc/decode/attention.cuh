// The work list of lora_tree_attention, shared by its kernels.
//
// The rows of a unit are up to `rt` of the n * (n_q / n_kv) query rows that
// share one kv head of one request (row r: drafted token r / group, head r %
// group), so a cached key and value are loaded once for the whole group.  A unit
// is cut into tiles of `tk` cached tokens, and all tiles of all units, in
// order (request, kv head, row tile, key tile), form one list that is cut into
// `grid` equal parts.  A unit's first tile has `unit_cost` empty places before it,
// for what starting and ending a unit takes (measured, in tiles): every block gets
// the same work whatever the lengths are, and a unit cut between blocks
// is joined afterwards from the blocks' partial sums.
#pragma once

#include "decode.cuh"

namespace lora {
namespace decode {

// What the join reads of a block: the unit that starts in its part and goes on after it.
struct __align__(16) JoinRecord {
    int parts, rows, begin, head, first_row, unused[3];      // rows 0: nothing to join
};

struct AttnParams {
    const void *q, *k, *v;
    int n_q, n_kv, group, d, page_shift, n_pages;
    const int *starts, *lens, *table;
    int S, T, max_pages;
    const long long *mask;
    int words;
    float scale_log2;        // scale * log2(e): the softmax works in powers of two
    void *out;
    int *status;
    JoinRecord *records;     // [grid]
    float *partial;          // [grid][2]: sums [d / 4][rt][4], then the rows' maximum and sum [rt][2]
    int rt, tk, grid;        // rows a unit, tokens a tile (a power of two), blocks
    int tk_shift, unit_cost;
    uint32_t max_places;     // of the list of any table that keeps the rules; below 2^31
    float *lse;              // [T][n_q]: log2 of each row's sum, infinity where it saw nothing; or NULL
    int *computed;           // with lse: whether the list held anything
    float *scores;           // [T][n_q][ld_scores]: the rows' scores in powers of two (-infinity: not seen); or NULL
    long long ld_scores;     // a multiple of 32, as scores is of 128 bytes
};

struct Request {
    int begin, n, len, tiles, row_tiles;   // tokens; drafted; cached; key tiles; row tiles
    __device__ __forceinline__ uint32_t places(const AttnParams &p) const {
        return (uint32_t)(tiles + p.unit_cost) * row_tiles * p.n_kv;
    }
};

// Request s with everything clamped into the arrays.  bad: LORA_DEV_* bits.
__device__ __forceinline__ Request request_of(const AttnParams &p, int s, int *bad = nullptr) {
    Request r;
    const int b = p.starts[s], e = p.starts[s + 1], len = p.lens[s];
    const long long cap = (long long)p.max_pages << p.page_shift;
    r.begin = min(max(b, 0), p.T);
    r.n = min(max(e, r.begin), p.T) - r.begin;
    r.len = (int)min((long long)max(len, r.n), cap);
    if (bad && (len < r.n || len > cap)) *bad |= LORA_DEV_BAD_LENGTH;
    r.tiles = (r.len + p.tk - 1) >> p.tk_shift;
    r.row_tiles = (int)(((uint32_t)r.n * p.group + p.rt - 1) / (uint32_t)p.rt);
    return r;
}

// One block's place in the list: at key tile `tile` of a unit, with `left` places
// to go (none or fewer: done).
struct Cursor {
    Request r;
    int s, head, row_tile, tile, left;

    // Past `count` tiles of the unit.
    __device__ __forceinline__ void advance(const AttnParams &p, int count) {
        left -= count;
        tile += count;
        if (tile < r.tiles || left <= 0) return;
        tile = 0;
        left -= p.unit_cost;
        if (++row_tile < r.row_tiles) return;
        row_tile = 0;
        if (++head < p.n_kv) return;
        head = 0;
        do {
            if (++s >= p.S) {
                left = 0;
                return;
            }
            r = request_of(p, s);
        } while (r.row_tiles == 0);
    }
};

constexpr int kScanThreads = 128;

struct ScanShared {
    uint32_t sums[kScanThreads / 32];
    uint32_t residual;
    int request;
    Request r;
};

// Sum of places, at most 2^31 - 1: segments that overlap can name any number of them.
__device__ __forceinline__ uint32_t add_places(uint32_t a, uint32_t b) { return min(a + b, 0x7fffffffu); }

// The list has up to max_places places.  The first place of block c: total / grid places
// each, one more for the first total % grid.
__device__ __forceinline__ uint32_t block_begin(uint32_t total, uint32_t c, uint32_t grid) {
    const uint32_t each = total / grid;
    return each * c + min(c, total - each * grid);
}
// The block that has place x.
__device__ __forceinline__ int block_of(uint32_t total, uint32_t x, uint32_t grid) {
    const uint32_t each = total / grid, more = total - each * grid, edge = more * (each + 1);
    return (int)(x < edge ? x / (each + 1) : more + (x - edge) / each);
}

// What a kernel leaves beside its outputs: nothing; p.lse and p.computed; those and p.scores.
enum { kPlain, kSums, kScores };

// Called by every thread of the block (kScanThreads at least): the block's first tile, and the length of
// the list.  Lets the join launch; block 0 reports bad tables.  A table whose segments
// overlap until they name more places than the T tokens can have has an empty list.
// RECORDS: the block's record is cleared (the weights' kernels have none).
template <int MODE = kPlain, bool RECORDS = true>
__device__ __forceinline__ uint32_t start_block(const AttnParams &p, ScanShared &sh, Cursor &c) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.S + kScanThreads - 1) / kScanThreads;
    const int s0 = tid < kScanThreads ? min(p.S, tid * per) : p.S, s1 = min(p.S, s0 + per);
    const bool flags = blockIdx.x == 0;
    uint32_t mine = 0;
    int bad = 0;
    Request r = {};
    for (int s = s0; s < s1; ++s) {
        r = request_of(p, s, &bad);
        mine = add_places(mine, r.places(p));
        if (flags && (p.starts[s + 1] < p.starts[s] || (s == 0 && p.starts[0] != 0) || (s + 1 == p.S && p.starts[p.S] != p.T)))
            bad |= LORA_DEV_BAD_SEGMENTS;
    }
    if (flags && bad) flag_status(p.status, bad);
    uint32_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t other = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto = add_places(upto, other);
    }
    if (lane == 31 && warp < kScanThreads / 32) sh.sums[warp] = upto;
    if (tid == 0) {
        sh.request = -1;
        if (RECORDS) p.records[blockIdx.x] = JoinRecord{};
    }
    __syncthreads();
    uint32_t total = 0, before = upto - mine;
#pragma unroll
    for (int w = 0; w < kScanThreads / 32; ++w) {
        if (w < warp) before = add_places(before, sh.sums[w]);
        total = add_places(total, sh.sums[w]);
    }
    if (total > p.max_places) total = 0;
    if (MODE != kPlain && flags && tid == 0) *p.computed = total > 0;
    const uint32_t pos = block_begin(total, blockIdx.x, p.grid);
    if (total > 0 && pos >= before && pos < before + mine) {
        uint32_t rest = pos - before;
        for (int s = s0; s < s1; ++s) {
            if (s1 - s0 > 1) r = request_of(p, s);
            const uint32_t w = r.places(p);
            if (rest < w) {
                sh.request = s;
                sh.residual = rest;
                sh.r = r;
                break;
            }
            rest -= w;
        }
    }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    c.s = sh.request;
    c.left = 0;
    if (c.s >= 0) {
        c.r = sh.r;
        const uint32_t each = c.r.tiles + p.unit_cost, unit = sh.residual / each;
        const int place = (int)(sh.residual - unit * each) - p.unit_cost;       // below 0: before the first tile
        c.head = unit / (uint32_t)c.r.row_tiles;
        c.row_tile = unit - c.head * c.r.row_tiles;
        c.tile = max(place, 0);
        c.left = (int)(block_begin(total, blockIdx.x + 1, p.grid) - pos) + min(place, 0);
    }
    return total;
}

// Thread 0, where a unit started in the block and goes on after the block's last
// tile, at which the cursor is.  Its parts stay inside the grid also when the lengths change
// under the call, between one read and the next.
__device__ __forceinline__ void record_unit(const AttnParams &p, const Cursor &cur, int tile, uint32_t total) {
    JoinRecord rec = {};
    const uint32_t last = block_begin(total, blockIdx.x + 1, p.grid) - 1 + (cur.r.tiles - 1 - tile);
    rec.parts = (int)min((uint32_t)block_of(total, last, p.grid), (uint32_t)p.grid - 1) - (int)blockIdx.x + 1;
    rec.begin = cur.r.begin;
    rec.head = cur.head;
    rec.first_row = cur.row_tile * p.rt;
    rec.rows = min(p.rt, cur.r.n * p.group - rec.first_row);
    p.records[blockIdx.x] = rec;
}

// Which of the 32 cached tokens from c0 on drafted token i sees, one bit each.
__device__ __forceinline__ uint32_t seen_word(const AttnParams &p, const Request &r, int i, int c0) {
    const int j0 = c0 - (r.len - r.n);       // drafted index of bit 0
    if (j0 <= -32) return ~0u;
    if (j0 >= r.n) return 0u;
    uint32_t bits;
    if (!p.mask) {
        const int count = i + 1 - j0;        // tokens up to i itself
        bits = count >= 32 ? ~0u : count <= 0 ? 0u : (1u << count) - 1;
    } else {
        const unsigned long long *row = reinterpret_cast<const unsigned long long *>(p.mask) + (long long)(r.begin + i) * p.words;
        const int at = max(j0, 0), q = at >> 6, sh = at & 63;
        unsigned long long w = q < p.words ? __ldg(row + q) >> sh : 0ull;
        if (sh > 32 && q + 1 < p.words) w |= __ldg(row + q + 1) << (64 - sh);
        bits = (uint32_t)w;
        if (j0 < 0) bits = (bits << -j0) | ((1u << -j0) - 1);      // the prefix
    }
    const int valid = r.n - j0;              // tokens up to the request's end
    return valid < 32 ? bits & ((1u << valid) - 1) : bits;
}

// Page of cached token c, clamped into the cache (flagged); -1 beyond the request.
__device__ __forceinline__ int page_of(const AttnParams &p, int s, const Request &r, int c) {
    return c < r.len ? __ldg(p.table + (long long)s * p.max_pages + (c >> p.page_shift)) : -1;
}
__device__ __forceinline__ int checked_page(const AttnParams &p, int page) {
    if (page >= 0 && page < p.n_pages) return page;
    flag_status(p.status, LORA_DEV_BAD_PAGE);
    return 0;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// Row `row` of the unit at cursor c among the T x n_q rows of q and out, and its element offset.
__device__ __forceinline__ long long row_index(const AttnParams &p, const Cursor &c, int row) {
    const int i = row / p.group, g = row - i * p.group;
    return (long long)(c.r.begin + i) * p.n_q + c.head * p.group + g;
}
__device__ __forceinline__ long long row_offset(const AttnParams &p, const Cursor &c, int row) { return row_index(p, c, row) * p.d; }

// For p.lse: of a row's maximum and sum.
__device__ __forceinline__ float log_sum(float top, float sum) { return sum == 0.f ? INFINITY : top + log2f(sum); }

// Place of element (row, col) in a block's sums: neighbouring rows' groups of four columns lie side by side.
__device__ __forceinline__ int partial_at(const AttnParams &p, int row, int col) { return ((col >> 2) * p.rt + row) * 4 + (col & 3); }

// Sums of block `block`: slot 0 when its part of the unit does not start it, else 1.
__device__ __forceinline__ float *partial_of(const AttnParams &p, int block, int slot) {
    return p.partial + ((long long)block * 2 + slot) * p.rt * (p.d + 2);
}

struct KvMaps;

// attention_tc.cu: p.rt (128 or 256 rows), p.tk (128), p.grid and p.partial set; p.d is 64
// or 128.  maps: tensor maps with boxes of min(page, 128) rows, or NULL (pages below 8 tokens).
int launch_attention_tc(const KvMaps *maps, const AttnParams &p, cudaStream_t st);

// weigh.cu: the weights of the cached tokens from p.lse, after the attention's kernels on the stream.  plan_weigh makes
// launch_weigh's parameters of the attention's, or refuses.
int plan_weigh(const lora_kv_pages *kv, const AttnParams &attention, AttnParams &p);
int launch_weigh(const lora_kv_pages *kv, const KvMaps *maps, const AttnParams &p, float *weights, float decay, cudaStream_t st);

}  // namespace decode
}  // namespace lora
