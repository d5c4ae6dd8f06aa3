// Shared by the kernels that sum up cached tokens' weights.
#pragma once

#include "attention.cuh"

namespace lora {
namespace decode {

// A block's part of the list whose places are (request, kv head, key tile, row tile): the key tiles that begin in it.
// A kv head has unit_cost * row_tiles empty places before its first.
struct KeyCursor {
    Request r;
    int s, head, tile, left;
    __device__ __forceinline__ void start(const AttnParams &p, const ScanShared &sh, uint32_t total) {
        s = sh.request;
        left = 0;
        if (s < 0) return;
        r = sh.r;
        left = (int)(block_begin(total, blockIdx.x + 1, p.grid) - block_begin(total, blockIdx.x, p.grid));
        const uint32_t each = (uint32_t)(r.tiles + p.unit_cost) * r.row_tiles, h = sh.residual / each;
        const int place = (int)(sh.residual - h * each) - p.unit_cost * r.row_tiles;       // below 0: before the first tile
        head = h;
        tile = max(place, 0) / r.row_tiles;
        left += min(place, 0);
        const int into = max(place, 0) - tile * r.row_tiles;
        if (into) {                    // the tile began in an earlier block
            left -= r.row_tiles - into;
            next(p);
        }
    }
    __device__ __forceinline__ void next(const AttnParams &p) {
        if (++tile < r.tiles || left <= 0) return;
        tile = 0;
        if (++head >= p.n_kv) {
            head = 0;
            do {
                if (++s >= p.S) {
                    left = 0;
                    return;
                }
                r = request_of(p, s);
            } while (r.row_tiles == 0 || r.tiles == 0);
        }
        left -= p.unit_cost * r.row_tiles;
    }
    __device__ __forceinline__ void advance(const AttnParams &p) { advance(p, 1); }
    // Past `count` key tiles of the kv head.
    __device__ __forceinline__ void advance(const AttnParams &p, int count) {
        left -= count * r.row_tiles;
        tile += count - 1;
        next(p);
    }
    // The block's tiles of this kv head.
    __device__ __forceinline__ int run() const { return min(r.tiles - tile, (left + r.row_tiles - 1) / r.row_tiles); }
};

// The weight's place of cached token c, -1 where its page is outside the cache (flagged).
__device__ __forceinline__ long long weight_at(const AttnParams &p, int s, const Request &r, int head, int c) {
    const int page = page_of(p, s, r, c);
    if (page < 0 || page >= p.n_pages) {
        flag_status(p.status, LORA_DEV_BAD_PAGE);
        return -1;
    }
    return (((long long)page * p.n_kv + head) << p.page_shift) + (c & ((1 << p.page_shift) - 1));
}

constexpr int kWeighTile = 256, kWeighRows = 128;      // of weigh_tc_kernel: cached tokens a tile, rows a place of the list

// In places of all rows: what starting a kv head costs (8 requests of 64 tokens over <= 16384: 0, 1, 2 places 94.7, 85.9, 86.3 us).
constexpr int kWeighUnitCost = 1;

// weigh_tc.cu: a bf16 cache; maps as for launch_attention_tc.
int launch_weigh_tc(const KvMaps *maps, const AttnParams &p, float *weights, float decay, cudaStream_t st);

}  // namespace decode
}  // namespace lora
