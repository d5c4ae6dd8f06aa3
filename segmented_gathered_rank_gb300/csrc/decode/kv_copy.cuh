// Copies of key and value tiles from the paged cache into shared memory.
//
// A tile is TILE cached tokens of one kv head, as D/64 panels of TILE rows of 128
// bytes (64 head elements), 16-byte chunks XORed with the row: the layout that
// tensor copies with 128-byte swizzling write, that tcgen05 reads and that
// ldmatrix reads without bank conflicts.
//
//   tma = true   pages of 8 tokens or more (8 rows are one swizzle atom): one
//                copy a page and panel, by one warp, a lane a page.  Rows past
//                the request hold whatever the page holds.
//   tma = false  smaller pages: 16-byte copies by several warps; rows past the
//                request become zeros.
#pragma once

#include <cuda.h>

#include "attention.cuh"
#include "tc_common.cuh"

namespace lora {
namespace decode {

// K and V as matrices of n_pages * n_kv_heads * page_size rows of head_dim.
struct KvMaps {
    CUtensorMap k, v;
};

__device__ __forceinline__ uint32_t panel_off(int tile_rows, int row, int chunk) {
    return (uint32_t)((chunk >> 3) * (tile_rows * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool real) {
    const int bytes = real ? 16 : 0;        // 0: the 16 bytes become zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Arrives on `bar` once this thread's copies so far are complete.
__device__ __forceinline__ void cp_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(tc::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;\n" ::: "memory"); }

__device__ __forceinline__ bool non_finite2(uint32_t w) {      // either bf16 half
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t finite2(uint32_t w) {      // halves that are not finite become 0
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
    return w;
}

// Takes bf16 values that are not finite out of 16 bytes; whether there were any.
__device__ __forceinline__ bool make_finite(uint4 *at) {
    const uint4 u = *at;
    if (!(non_finite2(u.x) || non_finite2(u.y) || non_finite2(u.z) || non_finite2(u.w))) return false;
    *at = make_uint4(finite2(u.x), finite2(u.y), finite2(u.z), finite2(u.w));
    return true;
}

// One warp's tensor copies.  fetch() starts the load of this lane's page id of a
// tile, copy() uses it: fetched a tile ahead, its latency is hidden.
template <int D, int TILE>
struct TmaCopy {
    static constexpr int kThreads = 32;
    static constexpr int kArrivals = 1;     // on the tile's barrier
    int page, offset, head;                 // offset: in the page, -1 without a page

    __device__ __forceinline__ void fetch(const AttnParams &p, const Cursor &c, int tile, int lane) {
        const int per = min(1 << p.page_shift, TILE), at = tile * TILE + lane * per;
        const bool has = lane * per < TILE && at < c.r.len;
        offset = has ? at & ((1 << p.page_shift) - 1) : -1;
        page = has ? page_of(p, c.s, c.r, at) : 0;
        head = c.head;
    }
    __device__ __forceinline__ void copy(const AttnParams &p, const CUtensorMap *map, const void *, uint32_t dst,
                                         uint64_t *bar, int lane) const {
        const int per = min(1 << p.page_shift, TILE), panels = (p.d + 63) >> 6;
        const int pages = __popc(__ballot_sync(0xffffffffu, offset >= 0));
        if (lane == 0) tc::mbar_arrive_expect_tx(bar, (uint32_t)(pages * per * panels * 128));
        __syncwarp();
        if (offset < 0) return;
        const int row = ((checked_page(p, page) * p.n_kv + head) << p.page_shift) + offset;
        for (int h = 0; h < panels; ++h)
            asm volatile(
                "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::
                    "r"(dst + h * (TILE * 128) + lane * per * 128),
                "l"(map), "r"(h * 64), "r"(row), "r"(tc::smem_u32(bar))
                : "memory");
    }
    // Rows `first` on of a landed V tile: rows from `end` on become zeros, values that are not finite
    // too; returns whether there were any such (masked, they would enter the product times zero).
    __device__ __forceinline__ bool clean(const AttnParams &p, uint8_t *tile, int first, int end, int lane) const {
        for (int x = lane; x < (TILE - end) * (D / 8); x += 32)
            *reinterpret_cast<uint4 *>(tile + panel_off(TILE, end + x / (D / 8), x % (D / 8))) = make_uint4(0, 0, 0, 0);
        const int last = min(end, TILE), count = (last - first) * (D / 8);
        bool found = false;
#pragma unroll 4
        for (int x = lane; x < count; x += 32) {
            const uint4 u = *reinterpret_cast<const uint4 *>(tile + panel_off(TILE, first + x / (D / 8), x % (D / 8)));
            found |= non_finite2(u.x) || non_finite2(u.y) || non_finite2(u.z) || non_finite2(u.w);
        }
        if (found)
            for (int x = lane; x < count; x += 32)
                make_finite(reinterpret_cast<uint4 *>(tile + panel_off(TILE, first + x / (D / 8), x % (D / 8))));
        return found;
    }
};

// 16-byte copies by THREADS threads.
template <int D, int TILE, int THREADS>
struct ChunkCopy {
    static constexpr int kThreads = THREADS;
    static constexpr int kArrivals = THREADS;
    static constexpr int kLanes = D / 8, kRows = THREADS / kLanes, kPasses = TILE / kRows;
    int row[kPasses];                       // cache rows, -1 past the request

    __device__ __forceinline__ void fetch(const AttnParams &p, const Cursor &c, int tile, int tid) {
        const int page_mask = (1 << p.page_shift) - 1;
        int bad = 0;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int at = tile * TILE + tid / kLanes + i * kRows;
            int page = at < c.r.len ? __ldg(p.table + (long long)c.s * p.max_pages + (at >> p.page_shift)) : 0;
            const bool in = page >= 0 && page < p.n_pages;
            bad |= !in;
            page = in ? page : 0;
            row[i] = at < c.r.len ? ((page * p.n_kv + c.head) << p.page_shift) + (at & page_mask) : -1;
        }
        if (bad) flag_status(p.status, LORA_DEV_BAD_PAGE);
    }
    __device__ __forceinline__ void copy(const AttnParams &p, const CUtensorMap *, const void *src, uint32_t dst,
                                         uint64_t *, int tid) const {
        const int chunk = tid % kLanes, r0 = tid / kLanes;
        if (chunk * 8 >= ((p.d + 15) & ~15)) return;
        const bool pad = chunk * 8 >= p.d;          // the products read whole 16-element steps
        const char *at = static_cast<const char *>(src) + chunk * 16;
        const long long pitch = p.d * 2;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const bool real = row[i] >= 0 && !pad;
            cp_async16(dst + panel_off(TILE, r0 + i * kRows, chunk), real ? at + row[i] * pitch : src, real);
        }
    }
    // As above, each thread in the chunks it copied itself (rows past the request are zeros already).
    __device__ __forceinline__ bool clean(const AttnParams &p, uint8_t *tile, int first, int, int tid) const {
        bool found = false;
        const int chunk = tid % kLanes;
        if (chunk * 8 >= p.d) return false;
        for (int r = tid / kLanes; r < TILE; r += kRows)
            if (r >= first) found |= make_finite(reinterpret_cast<uint4 *>(tile + panel_off(TILE, r, chunk)));
        return found;
    }
};

}  // namespace decode
}  // namespace lora
