// Tree attention on the tensor cores (tcgen05) for units of many query rows.
//
// With R rows a kv head the products cost 4 R flops for every 2 bytes of K and
// V: from R = 64 on, warp MMAs (about a quarter of the tcgen05 rate) bound the
// kernel instead of memory.  Here S = Q K^T and O += P V are tcgen05 products
// of 128 rows x 128 cached tokens with S, P and O in tensor memory.
//
// Two softmax streams of four warps each (one thread a row) share the tensor
// cores, so that one's products run under the other's exponentials:
//   NQ = 2   units of up to 256 rows; stream w has rows w * 128 .. + 127 and both
//            take every key tile, so a tile in shared memory serves 256 rows;
//   NQ = 1   units of up to 128 rows; stream w takes every other key tile, with
//            a maximum, sum and output of its own, joined when the unit ends.
// Two producer warps (keys and values) keep a ring of K and V tiles filled; one
// thread issues all MMAs.  P overwrites the columns of S that it was
// computed from.
//
// 8 trees of 64 tokens over <= 16384 (256 rows a kv head): 55.6 us, 586 TFLOP/s, 0.30 of
// the measured rate.  A tile of keys takes about 3450 cycles, of which the products are
// 2048: a stream goes from its scores to its probabilities in 1870 (650 of them the
// exponentials) and waits 1580 for its two products of 512 and the hand-overs.
// 2 requests of 16 tokens over 131072 (64 rows): 155 us, 6.1 TB/s, the bytes' bound.
//
// A row keeps the maximum it last scaled by until a score passes it by 2^8
// (sums stay far inside fp32), so the output is rescaled in a few tiles only.
#include <type_traits>

#include "kv_copy.cuh"

namespace lora {
namespace {

using namespace decode;
using namespace tc;

constexpr int kTile = 128;                 // cached tokens a tile, rows a stream
constexpr int kThreadsTc = 12 * 32;        // four warps each: streams 0 and 1; copies and MMAs
constexpr int kProducer0 = 8, kMmaWarp = 11;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 8.f;

template <int D>
struct TcShape {
    static constexpr int kSlot = kTile * D * 2;              // a K or V tile (or a stream's queries)
    static constexpr int kSlots = D == 128 ? 5 : 10;
    static constexpr int kControl = 1536;
    static constexpr size_t kSmem = (size_t)(2 + kSlots) * kSlot + kControl + 1024;
};

struct Control {
    uint64_t full[10], empty[10], s_full[2], p_ready[2], o_full[2], q_ready[2], landed, pair, drain;
    int bad[10];              // sequence number + 1 of a V tile that held values that are not finite
    int accumulate[2];        // the stream wrote its output itself before the unit's first product
    volatile int abort;
    uint32_t tmem;
    float row_max[kTile], row_sum[kTile];       // stream 1's, for the join
};

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, Control *ctl) {
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    if (wait_phase(bar, parity, &ctl->abort)) return true;
    ctl->abort = 1;
    return false;
}

// wait_bar for a whole warp: all lanes go on, or none.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, Control *ctl) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, ctl));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n" ::"r"(taddr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
        "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]),
        "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]),
        "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
        : "memory");
}
// 32 columns without a wait; tmem_arrived() below orders the reads of `r` after it.
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, float *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
          "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
          "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tmem_arrived(float *r) {
    asm volatile(""
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                   "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]),
                   "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]),
                   "+f"(r[23]), "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]),
                   "+f"(r[30]), "+f"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
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
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nadd.rn.f32x2 d, a, b;\nmov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};\n" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// V as the B operand of O += P V: rows of 64 head elements (128 bytes, swizzled),
// one row a cached token, so the token (K) axis runs along the rows.  lbo: bytes
// between the two halves of the head; 1024 bytes between groups of 8 tokens.
__device__ __forceinline__ uint64_t desc_rows_sw128(uint32_t smem_addr, uint32_t lbo) {
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(lbo >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
constexpr uint32_t kTransposeB = 1u << 16;

// The tiles of one unit that a block takes.
struct Segment {
    int first, tiles;
    bool whole;              // the block has the unit to itself
};
__device__ __forceinline__ Segment segment_at(const Cursor &c) {
    Segment s;
    s.first = c.tile;
    s.tiles = min(c.left, c.r.tiles - c.tile);
    s.whole = c.tile == 0 && s.tiles == c.r.tiles;
    return s;
}

// Ring positions 2 t (keys) and 2 t + 1 (values) of the block's tile t.  Tensor
// copies: one warp the keys, one the values; else both warps copy both.
template <int D, bool TMA>
__device__ void produce(const AttnParams &p, const KvMaps &maps, Cursor cur, uint8_t *ring, Control *ctl) {
    using Sh = TcShape<D>;
    using Copy = std::conditional_t<TMA, TmaCopy<D, kTile>, ChunkCopy<D, kTile, 64>>;
    const int warp = (threadIdx.x >> 5) - kProducer0;
    const int tid = TMA ? threadIdx.x & 31 : threadIdx.x - kProducer0 * 32;
    if (warp >= 2) return;
    const uint32_t base = smem_u32(ring);
    Copy copy;
    uint32_t seq0 = 0, landed = 0;
    copy.fetch(p, cur, cur.tile, tid);
    while (cur.left > 0) {
        const Segment seg = segment_at(cur);
        Cursor after = cur;
        after.advance(p, seg.tiles);
        for (int t = 0; t < seg.tiles; ++t, seq0 += 2) {
            const int tile = seg.first + t;
            const int drafted = max(0, cur.r.len - cur.r.n - tile * kTile);      // first row that a mask rules
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                if (TMA && which != warp) continue;
                const uint32_t seq = seq0 + which, slot = seq % Sh::kSlots, use = seq / Sh::kSlots;
                if (TMA ? !wait_warp(&ctl->empty[slot], (use & 1) ^ 1, ctl) : !wait_bar(&ctl->empty[slot], (use & 1) ^ 1, ctl)) {
                    // this warp's tensor copies on their way land before the block leaves
                    for (uint32_t x = 2; TMA && x < Sh::kSlots && seq >= x; x += 2)
                        wait_phase(&ctl->full[(seq - x) % Sh::kSlots], ((seq - x) / Sh::kSlots) & 1, nullptr);
                    return;
                }
                const bool clean = which && drafted < kTile;     // before the products see the tile
                copy.copy(p, which ? &maps.v : &maps.k, which ? p.v : p.k, base + slot * Sh::kSlot,
                          TMA && clean ? &ctl->landed : &ctl->full[slot], tid);
                if (which || TMA) {
                    if (t + 1 < seg.tiles) copy.fetch(p, cur, tile + 1, tid);
                    else if (after.left > 0) copy.fetch(p, after, after.tile, tid);
                }
                if (!clean) {
                    if (!TMA) cp_arrive(&ctl->full[slot]);
                    continue;
                }
                if (TMA) {
                    if (!wait_warp(&ctl->landed, landed & 1, ctl)) {
                        wait_phase(&ctl->landed, landed & 1, nullptr);
                        return;
                    }
                    ++landed;
                } else {
                    cp_wait_all();
                }
                if (copy.clean(p, ring + slot * Sh::kSlot, drafted, cur.r.len - tile * kTile, tid)) ctl->bad[slot] = (int)seq + 1;
                fence_proxy_async();
                if (TMA) {
                    __syncwarp();
                    if (tid == 0) mbar_arrive(&ctl->full[slot]);
                } else {
                    mbar_arrive(&ctl->full[slot]);
                }
            }
        }
        cur = after;
    }
}

// A position of the ring, without divisions on the way.
template <int SLOTS>
struct Place {
    uint32_t slot, parity;
    __device__ __forceinline__ explicit Place(uint32_t seq) : slot(seq % SLOTS), parity((seq / SLOTS) & 1) {}
    __device__ __forceinline__ Place next(int n) const {        // n <= SLOTS
        Place to = *this;
        to.slot += n;
        if (to.slot >= SLOTS) {
            to.slot -= SLOTS;
            to.parity ^= 1;
        }
        return to;
    }
};

// One thread issues every MMA.  At 64 cycles a product of 128 x 128 x 16 its own
// instructions are what can starve the tensor cores (its warp shares scheduler and
// instruction cache with softmax warps), so the loop over a segment is a function of
// its own whose state is in registers: descriptors are 32-bit additions (16-byte
// units) to a constant upper half.
template <int D, int NQ, bool TMA>
struct Issuer {
    using Sh = TcShape<D>;
    using At = Place<Sh::kSlots>;
    static constexpr uint32_t kSwizzled = (1024u >> 4) | (1u << 14) | (2u << 29);      // descriptor bits 32..63
    static constexpr uint32_t kIdescS = idesc_bf16_f32(kTile, kTile);
    static constexpr uint32_t kIdescO = idesc_bf16_f32(kTile, D) | kTransposeB;

    static __device__ __forceinline__ bool slot_full(Control *ctl, const At &at) {
        if (!wait_bar(&ctl->full[at.slot], at.parity, ctl)) return false;
        if (!TMA) fence_proxy_async();          // ordinary writes; the MMAs read through the async proxy
        fence_after_sync();
        return true;
    }
    static __device__ __forceinline__ void release(Control *ctl, const At &at) { mma_commit(&ctl->empty[at.slot]); }
    static __device__ __forceinline__ bool probabilities(Control *ctl, int w, uint32_t &phases) {
        if (!wait_bar(&ctl->p_ready[w], (phases >> w) & 1, ctl)) return false;
        phases ^= 1u << w;
        fence_after_sync();
        return true;
    }
    // S_w = Q_w K^T
    static __device__ __forceinline__ void scores(Control *ctl, uint32_t tmem, uint32_t q_lo, uint32_t k_lo, int w, const At &at) {
        uint32_t q = q_lo + w * (Sh::kSlot / 16), k = k_lo + at.slot * (Sh::kSlot / 16);
        const uint32_t d = tmem + w * kTile;
#pragma unroll 1
        for (int panel = 0; panel < D / 64; ++panel, q += kTile * 128 / 16, k += kTile * 128 / 16) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                asm volatile(
                    "{\n.reg .pred p;\n.reg .b64 a, b;\nsetp.ne.b32 p, %5, 0;\nmov.b64 a, {%1, %3};\nmov.b64 b, {%2, %3};\n"
                    "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}\n" ::"r"(d),
                    "r"(q + ks * 2), "r"(k + ks * 2), "n"(kSwizzled), "n"(kIdescS), "r"(ks > 0 || panel > 0 ? 1u : 0u)
                    : "memory");
            }
        }
        mma_commit(&ctl->s_full[w]);
    }
    // O_w += P_w V
    static __device__ __forceinline__ void output(uint32_t tmem, uint32_t v_lo, int w, const At &at, bool accumulate) {
        uint32_t v = v_lo + at.slot * (Sh::kSlot / 16), pr = tmem + w * kTile, acc = accumulate ? 1u : 0u;
        const uint32_t d = tmem + 2 * kTile + w * D;
#pragma unroll 1
        for (int half = 0; half < 2; ++half, v += 4 * 2048 / 16, pr += 32) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                asm volatile(
                    "{\n.reg .pred p;\n.reg .b64 b;\nsetp.ne.b32 p, %5, 0;\nmov.b64 b, {%2, %3};\n"
                    "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}\n" ::"r"(d),
                    "r"(pr + ks * 8), "r"(v + ks * (2048 / 16)), "n"(kSwizzled), "n"(kIdescO), "r"(acc)
                    : "memory");
                acc = 1u;
            }
        }
    }
    // The tiles of a segment; tile t has its keys at ring position seq0 + 2 t, its values right
    // after them.  phases: bit w, the parity of stream w's next probabilities; returns them, or
    // kGaveUp.
    static constexpr uint32_t kGaveUp = 4;
    static __device__ __noinline__ uint32_t segment(Control *ctl, uint32_t tmem, uint32_t q_lo, uint32_t k_lo, uint32_t v_lo,
                                                    uint32_t seq0, uint32_t phases, int tiles, int streams) {
        At k(seq0);
        if (NQ == 2) {
            if (!slot_full(ctl, k)) return kGaveUp;
            for (int w = 0; w < streams; ++w) scores(ctl, tmem, q_lo, k_lo, w, k);
            release(ctl, k);
#pragma unroll 1
            for (int t = 0; t < tiles; ++t) {
                const At v = k.next(1);
                const bool more = t + 1 < tiles;
                k = k.next(2);
#pragma unroll 1
                for (int w = 0; w < streams; ++w) {
                    if (!probabilities(ctl, w, phases)) return kGaveUp;
                    if (w == 0 && !slot_full(ctl, v)) return kGaveUp;
                    output(tmem, v_lo, w, v, t > 0 || ctl->accumulate[w]);
                    if (!more) mma_commit(&ctl->o_full[w]);
                    if (w == streams - 1) release(ctl, v);
                    if (more) {
                        if (w == 0 && !slot_full(ctl, k)) return kGaveUp;
                        scores(ctl, tmem, q_lo, k_lo, w, k);
                    }
                }
                if (more) release(ctl, k);
            }
        } else {
#pragma unroll 1
            for (int w = 0; w < streams; ++w, k = k.next(2)) {
                if (!slot_full(ctl, k)) return kGaveUp;
                scores(ctl, tmem, q_lo, k_lo, w, k);
                release(ctl, k);
            }
            At v(seq0 + 1);
#pragma unroll 1
            for (int t = 0; t < tiles; ++t, v = v.next(2), k = k.next(2)) {
                const int w = t & 1;
                if (!probabilities(ctl, w, phases) || !slot_full(ctl, v)) return kGaveUp;
                output(tmem, v_lo, w, v, t > 1 || ctl->accumulate[w]);
                release(ctl, v);
                if (t + 2 < tiles) {
                    if (!slot_full(ctl, k)) return kGaveUp;
                    scores(ctl, tmem, q_lo, k_lo, w, k);
                    release(ctl, k);
                } else {
                    mma_commit(&ctl->o_full[w]);
                }
            }
        }
        return phases;
    }
};

template <int D, int NQ, bool TMA>
__device__ void issue(const AttnParams &p, Cursor cur, uint8_t *queries, uint8_t *ring, Control *ctl) {
    using Is = Issuer<D, NQ, TMA>;
    const uint32_t tmem = ctl->tmem;
    const uint32_t q_lo = (uint32_t)desc_kmajor_sw128(smem_u32(queries));
    const uint32_t k_lo = (uint32_t)desc_kmajor_sw128(smem_u32(ring));
    const uint32_t v_lo = (uint32_t)desc_rows_sw128(smem_u32(ring), kTile * 128);
    uint32_t seq0 = 0, phases = 0, q_phase[2] = {0, 0};
    while (cur.left > 0) {
        const Segment seg = segment_at(cur);
        const int rows = cur.r.n * p.group - cur.row_tile * p.rt;
        const int streams = NQ == 2 ? (rows > kTile ? 2 : 1) : (seg.tiles > 1 ? 2 : 1);
        for (int w = 0; w < streams; ++w) {
            if (!wait_bar(&ctl->q_ready[w], q_phase[w] & 1, ctl)) return;
            ++q_phase[w];
        }
        fence_after_sync();
        phases = Is::segment(ctl, tmem, q_lo, k_lo, v_lo, seq0, phases, seg.tiles, streams);
        if (phases == Is::kGaveUp) return;
        seq0 += 2 * seg.tiles;
        cur.advance(p, seg.tiles);
    }
}

// 64 scores of the thread's row; those that it does not see become -infinity, whatever they are.
__device__ __forceinline__ void load_scores(float *s, uint32_t taddr, bool masked, const uint32_t *see) {
    tmem_ld32_start(taddr, s);
    tmem_ld32_start(taddr + 32, s + 32);
    tmem_wait_ld();
    tmem_arrived(s);
    tmem_arrived(s + 32);
    if (masked) {
#pragma unroll
        for (int x = 0; x < 64; ++x)
            if (!((see[x >> 5] >> (x & 31)) & 1)) s[x] = -INFINITY;
    }
}

// One thread a row: its queries into shared memory, the softmax of its scores,
// and at the end of the segment its output.
// A softmax thread's row of its stream, and where the unit's row lies in q and out (-1: none).
template <int NQ>
__device__ __forceinline__ long long row_at(const AttnParams &p, const Cursor &cur) {
    const int warp = threadIdx.x >> 5, row = (warp & 3) * 32 + (threadIdx.x & 31) + (NQ == 2 ? (warp >> 2) * kTile : 0);
    return row < cur.r.n * p.group - cur.row_tile * p.rt ? row_offset(p, cur, cur.row_tile * p.rt + row) : -1;
}
// Whether stream w has a part in the segment at the cursor: rows of its own, or key tiles.
template <int NQ>
__device__ __forceinline__ bool takes_part(const AttnParams &p, const Cursor &cur, int w) {
    return w == 0 || (NQ == 2 ? cur.r.n * p.group - cur.row_tile * p.rt > kTile : segment_at(cur).tiles > 1);
}
// Starts the copies of the queries of a warp's 32 rows, D / 8 lanes a row (no row: zeros).  A stream
// without a part in the segment copies nothing: it would not wait for its copies, which have no
// order against those of the next segment to the same place.
template <int D, int NQ>
__device__ __forceinline__ void load_queries(const AttnParams &p, const Cursor &cur, uint8_t *queries) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (!takes_part<NQ>(p, cur, warp >> 2)) return;
    const long long my_off = row_at<NQ>(p, cur);
    const uint32_t dst = smem_u32(queries) + (warp >> 2) * TcShape<D>::kSlot;
#pragma unroll
    for (int x = 0; x < D / 8; ++x) {
        const int rr = x * (256 / D) + lane / (D / 8), c = lane % (D / 8);
        const long long off = __shfl_sync(0xffffffffu, my_off, rr);
        cp_async16(dst + panel_off(kTile, (warp & 3) * 32 + rr, c), static_cast<const __nv_bfloat16 *>(p.q) + (off >= 0 ? off + c * 8 : 0),
                   off >= 0);
    }
}

// The first unit's queries are on their way.
template <int D, int NQ>
__device__ void attend(const AttnParams &p, Cursor cur, uint32_t total, uint8_t *queries, Control *ctl) {
    using Sh = TcShape<D>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w = warp >> 2;                                  // stream
    const int row = (warp & 3) * 32 + lane;                   // of the stream, and its lane of tensor memory
    const uint32_t quad = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_tmem = ctl->tmem + quad + w * kTile, o_tmem = ctl->tmem + quad + 2 * kTile + w * D;
    uint8_t *my_q = queries + w * Sh::kSlot;
    uint32_t s_phase = 0, o_phase = 0, pair_phase = 0, seq0 = 0;
    auto both_streams = [&]() {                               // a barrier of the eight softmax warps
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->pair);
        return wait_warp(&ctl->pair, pair_phase++ & 1, ctl);
    };
    while (cur.left > 0) {
        const Segment seg = segment_at(cur);
        const int rows = cur.r.n * p.group - cur.row_tile * p.rt;
        const int ur = row + (NQ == 2 ? w * kTile : 0);       // row of the unit
        const bool live = ur < rows, warp_live = ur - lane < rows;
        const bool active = takes_part<NQ>(p, cur, w);
        float m = -INFINITY, l = 0.f;
        const long long my_off = row_at<NQ>(p, cur);
        if (active) {
            cp_wait_all();
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                if ((warp & 3) == 0) ctl->accumulate[w] = 0;
                mbar_arrive(&ctl->q_ready[w]);
            }
            const int token = (cur.row_tile * p.rt + ur) / p.group;
            for (int t = NQ == 2 ? 0 : w; t < seg.tiles; t += NQ == 2 ? 1 : 2) {
                const int tile = seg.first + t;
                const bool first = t < (NQ == 2 ? 1 : 2);
                if (!wait_warp(&ctl->s_full[w], s_phase & 1, ctl)) return;
                ++s_phase;
                fence_after_sync();
                const int c0 = tile * kTile;
                const bool masked = c0 + kTile > cur.r.len - cur.r.n;
                uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
                if (warp_live) {
                    if (masked) {
#pragma unroll
                        for (int b = 0; b < 4; ++b) see[b] = live ? seen_word(p, cur.r, token, c0 + b * 32) : 0u;
                    }
                    // the scores are read twice, 64 columns at a time: all of them would take most registers
                    float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float s[64];
                        load_scores(s, s_tmem + h * 64, masked, see + 2 * h);
#pragma unroll
                        for (int x = 0; x < 64; x += 8)
#pragma unroll
                            for (int b = 0; b < 4; ++b) tops[b] = max3(tops[b], s[x + 2 * b], s[x + 2 * b + 1]);
                    }
                    float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                    top *= p.scale_log2;
                    if (__any_sync(0xffffffffu, top > m + kRescaleLog2 || (m == -INFINITY && top > m))) {
                        const float m2 = fmaxf(m, top);
                        const float a = m2 == -INFINITY ? 1.f : exp2_fast(m - m2);
                        m = m2;
                        l *= a;
                        if (!first) {
#pragma unroll
                            for (int b = 0; b < D / 32; ++b) {
                                float o[32];
                                tmem_ld32(o_tmem + b * 32, o);
#pragma unroll
                                for (int x = 0; x < 32; ++x) o[x] *= a;
                                tmem_st32(o_tmem + b * 32, o);
                            }
                        }
                    }
                    const float ref = m == -INFINITY ? 0.f : m;
                    const float2 scale2 = make_float2(p.scale_log2, p.scale_log2), ref2 = make_float2(-ref, -ref);
                    float2 sums[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float s[64];
                        load_scores(s, s_tmem + h * 64, masked, see + 2 * h);
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            uint32_t pk[16];
#pragma unroll
                            for (int x = 0; x < 16; ++x) {
                                float2 e = fma2(make_float2(s[b * 32 + 2 * x], s[b * 32 + 2 * x + 1]), scale2, ref2);
                                e = make_float2(exp2_fast(e.x), exp2_fast(e.y));
                                sums[x & 1] = add2(sums[x & 1], e);
                                const __nv_bfloat162 v = __floats2bfloat162_rn(e.x, e.y);
                                pk[x] = *reinterpret_cast<const uint32_t *>(&v);
                            }
                            tmem_st16(s_tmem + h * 32 + b * 16, pk);
                        }
                    }
                    const float sum = (sums[0].x + sums[0].y) + (sums[1].x + sums[1].y);
                    l += sum;
                    tmem_wait_st();
                }
                if (masked) {
                    // values that the producers took out of the tile, for the rows that see them
                    const uint32_t v = seq0 + 2 * t + 1, slot = v % Sh::kSlots;
                    if (!wait_warp(&ctl->full[slot], (v / Sh::kSlots) & 1, ctl)) return;
                    if (*(volatile int *)&ctl->bad[slot] == (int)v + 1) {
                        if ((warp & 3) == 0 && lane == 0) ctl->accumulate[w] = 1;
                        for (int b = 0; b < D / 32; ++b) {
                            float o[32];
                            tmem_ld32(o_tmem + b * 32, o);
                            if (first) {
#pragma unroll
                                for (int x = 0; x < 32; ++x) o[x] = 0.f;
                            }
                            for (int x = max(0, cur.r.len - cur.r.n - c0); x < kTile; ++x) {
                                if (!live || !((see[x >> 5] >> (x & 31)) & 1)) continue;
                                const int c = c0 + x;
                                const int page = checked_page(p, page_of(p, cur.s, cur.r, c));
                                const __nv_bfloat16 *vr =
                                    static_cast<const __nv_bfloat16 *>(p.v) +
                                    ((((long long)page * p.n_kv + cur.head) << p.page_shift) + (c & ((1 << p.page_shift) - 1))) * D + b * 32;
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    const float f = __bfloat162float(vr[e]);
                                    if ((__float_as_uint(f) & 0x7f800000u) == 0x7f800000u) o[e] += f;
                                }
                            }
                            tmem_st32(o_tmem + b * 32, o);
                        }
                        tmem_wait_st();
                    }
                }
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->p_ready[w]);
            }
            if (!wait_warp(&ctl->o_full[w], o_phase & 1, ctl)) return;
            ++o_phase;
            fence_after_sync();
        }
        // the end of the segment: join the streams (NQ == 1), then write
        float other = 0.f;                       // weight of stream 1's sums
        const bool joined = NQ == 1 && seg.tiles > 1;
        float scale = 1.f;
        if (joined) {
            if (w == 1) {
                ctl->row_max[row] = m;
                ctl->row_sum[row] = l;
            }
            if (!both_streams()) return;
            if (w == 0) {
                const float m1 = ctl->row_max[row], top = fmaxf(m, m1), ref = top == -INFINITY ? 0.f : top;
                scale = exp2_fast(m - ref);
                other = exp2_fast(m1 - ref);
                m = top;
                l = l * scale + ctl->row_sum[row] * other;
            }
        }
        const bool writes = active && live && (NQ == 2 || w == 0);
        float *dst = partial_of(p, blockIdx.x, seg.first > 0 ? 0 : 1);
        const float r = l == 0.f ? 0.f : 1.f / l;            // a row that saw nothing: zeros
        if (writes && !seg.whole) {
            *reinterpret_cast<float2 *>(dst + p.rt * D + ur * 2) = make_float2(m, l);
        }
        // stream 1 hands its output over through its queries' space, 64 columns at a time
        float *hand = reinterpret_cast<float *>(queries + Sh::kSlot);
        constexpr int kHandCols = D == 128 ? 64 : 32;
        for (int h = 0; h < D / kHandCols; ++h) {
            if (joined && w == 1) {
#pragma unroll
                for (int b = 0; b < kHandCols / 32; ++b) {
                    float o[32];
                    tmem_ld32(o_tmem + h * kHandCols + b * 32, o);
#pragma unroll
                    for (int x = 0; x < 32; ++x) hand[(b * 32 + x) * kTile + row] = o[x];
                }
            }
            if (joined && !both_streams()) return;
            if (active && warp_live && (NQ == 2 || w == 0)) {
#pragma unroll
                for (int b = 0; b < kHandCols / 32; ++b) {
                    float o[32];
                    tmem_ld32(o_tmem + h * kHandCols + b * 32, o);
                    if (joined) {
#pragma unroll
                        for (int x = 0; x < 32; ++x) o[x] = o[x] * scale + hand[(b * 32 + x) * kTile + row] * other;
                    }
                    const int col = h * kHandCols + b * 32;
                    if (seg.whole) {        // into the queries' place, as they lay
#pragma unroll
                        for (int x = 0; x < 32; ++x) o[x] *= r;
#pragma unroll
                        for (int x = 0; x < 32; x += 8)
                            store8(reinterpret_cast<__nv_bfloat16 *>(my_q + panel_off(kTile, row, (col + x) >> 3)), o + x);
                    } else if (writes) {
#pragma unroll
                        for (int x = 0; x < 32; x += 4)
                            *reinterpret_cast<float4 *>(dst + partial_at(p, ur, col + x)) = make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
                    }
                }
            }
            if (joined && !both_streams()) return;
        }
        if (seg.whole && active && warp_live && (NQ == 2 || w == 0)) {
            __syncwarp();
            uint4 u[D / 8];
#pragma unroll
            for (int x = 0; x < D / 8; ++x)
                u[x] = *reinterpret_cast<const uint4 *>(my_q + panel_off(kTile, (warp & 3) * 32 + x * (256 / D) + lane / (D / 8), lane % (D / 8)));
#pragma unroll
            for (int x = 0; x < D / 8; ++x) {
                const long long off = __shfl_sync(0xffffffffu, my_off, x * (256 / D) + lane / (D / 8));
                if (off >= 0) *(reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + off) + lane % (D / 8)) = u[x];
            }
            __syncwarp();
        }
        fence_before_sync();       // the reads of O come before the next unit's first product
        if (threadIdx.x == 0 && seg.first == 0 && !seg.whole) record_unit(p, cur, seg.tiles - 1, total);
        seq0 += 2 * seg.tiles;
        cur.advance(p, seg.tiles);
        if (cur.left > 0) load_queries<D, NQ>(p, cur, queries);
    }
}

template <int D, int NQ, bool TMA>
__global__ void __launch_bounds__(kThreadsTc, 1)
    attention_tc_kernel(const __grid_constant__ KvMaps maps, const AttnParams p) {
    using Sh = TcShape<D>;
    extern __shared__ uint8_t raw[];
    __shared__ ScanShared scan;
    uint8_t *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint8_t *queries = smem, *ring = smem + 2 * Sh::kSlot;
    Control *ctl = reinterpret_cast<Control *>(ring + Sh::kSlots * Sh::kSlot);
    const int warp = threadIdx.x >> 5;
    static_assert(sizeof(Control) <= Sh::kControl, "control block");

    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::kSlots; ++i) {
            mbar_init(&ctl->full[i], TMA ? 1 : 64);
            mbar_init(&ctl->empty[i], 1);
            ctl->bad[i] = 0;
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(&ctl->s_full[w], 1);
            mbar_init(&ctl->p_ready[w], 4);
            mbar_init(&ctl->o_full[w], 1);
            mbar_init(&ctl->q_ready[w], 4);
            ctl->accumulate[w] = 0;
        }
        mbar_init(&ctl->landed, 1);
        mbar_init(&ctl->pair, 8);
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        mbar_fence_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&ctl->tmem, kTmemCols);
        tmem_relinquish();
    }
    Cursor cur;
    const uint32_t total = start_block(p, scan, cur);
    // the first queries are requested before the ring's tiles, which would keep them waiting
    if (warp < kProducer0 && cur.left > 0) load_queries<D, NQ>(p, cur, queries);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (cur.left <= 0) {
        if (warp == kMmaWarp) tmem_dealloc(ctl->tmem, kTmemCols);
        return;
    }
    if (warp < kProducer0) {
        attend<D, NQ>(p, cur, total, queries, ctl);
        cp_wait_all();             // also where it gave up: no copy outlives the block
    } else if (warp < kMmaWarp) {
        produce<D, TMA>(p, maps, cur, ring, ctl);
        if (!TMA) cp_wait_all();
    } else {
        if (warp == kMmaWarp && elect_lane()) {
            issue<D, NQ, TMA>(p, cur, queries, ring, ctl);
            mma_commit(&ctl->drain);
            wait_phase(&ctl->drain, 0, nullptr);
        }
        __syncwarp();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (threadIdx.x == 0 && ctl->abort) flag_status(p.status, LORA_DEV_WAIT_TIMEOUT);
    if (warp == kMmaWarp) tmem_dealloc(ctl->tmem, kTmemCols);
}

template <int D, int NQ, bool TMA>
int launch(const KvMaps &maps, const AttnParams &p, cudaStream_t st) {
    if (smem_optin(reinterpret_cast<const void *>(attention_tc_kernel<D, NQ, TMA>), TcShape<D>::kSmem)) return LORA_ERR_CUDA;
    attention_tc_kernel<D, NQ, TMA><<<p.grid, kThreadsTc, TcShape<D>::kSmem, st>>>(maps, p);
    count_launch();
    return cuda_status(cudaGetLastError());
}

template <int D>
int launch(const KvMaps *maps, const AttnParams &p, cudaStream_t st) {
    const bool two = p.rt == 256;
    if (maps) return two ? launch<D, 2, true>(*maps, p, st) : launch<D, 1, true>(*maps, p, st);
    const KvMaps none = {};
    return two ? launch<D, 2, false>(none, p, st) : launch<D, 1, false>(none, p, st);
}

}  // namespace

namespace decode {

int launch_attention_tc(const KvMaps *maps, const AttnParams &p, cudaStream_t st) {
    return p.d == 128 ? launch<128>(maps, p, st) : launch<64>(maps, p, st);
}

}  // namespace decode
}  // namespace lora
