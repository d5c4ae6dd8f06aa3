/*
 * lora.h -- C ABI of the GB300 multi-LoRA mixed-batch adapter library.
 *
 * The operation ("Multi-LoRA Serving - S-LoRA/Punica Batching, Adapter
 * Hot-Swap & Memory", section "The kernel trick: gather, do not merge"): a
 * request i that names adapter a(i) needs
 *
 *     y_i = x_i W^T + scale_a * (x_i A_a^T) B_a^T
 *
 * The base product is one matmul shared by the whole batch; the adapter term
 * is a gather of small matmuls, "shrink" (x -> v, width r) then "expand"
 * (v -> y).  SGMV serves contiguous segments of tokens that share an adapter
 * (prefill), BGMV one adapter per token (decode).  Adapters of different
 * ranks live in one paged pool (S-LoRA slide 8: pages of H elements, R of them
 * for a rank-R adapter) and are gathered without padding to a common rank
 * (S-LoRA slide 10, MBGMM/MBGMV).
 *
 * Orientation used throughout.  For adapter a on one adapted matrix:
 *   A_T_a is rank x h_in; its row j is the j-th low-rank direction, so
 *         v[t][j] = sum_k x[t][k] * A_T_a[j][k];
 *   B_a   is rank x h_out, and y[t][n] += scale_a * sum_j v[t][j] * B_a[j][n].
 *   W     is h_out x h_in, row-major (row n = output feature n), like an
 *         nn.Linear weight; the base term is y[t][n] = sum_k x[t][k] W[n][k].
 *
 * Conventions shared by every call:
 *   - Element type: every x, y, W and page holds the pool's dtype (LORA_F32
 *     or LORA_BF16).  v is always fp32.  Arithmetic accumulates in fp32;
 *     bf16 results are rounded to nearest even on store.
 *   - Layout: x is T x h_in, y is T x h_out, v is T x ld_v, all row-major and
 *     dense (row stride = width).  Base pointers of x, y, v, W and the
 *     workspace must be 16-byte aligned (torch allocations are).
 *   - Pointers passed to compute calls are DEVICE pointers owned by the
 *     caller; the library keeps none of them after the call returns.
 *   - Streams: a lora_stream is a cudaStream_t (NULL = legacy default
 *     stream).  Compute calls only enqueue work on it and never synchronise.
 *   - Adapter ids: id < 0 means "no adapter" (the token keeps its base/y0
 *     value).  An id >= max_adapters, or of an adapter not loaded on that
 *     matrix, is a device-detected error: the token gets no adapter term and
 *     bit LORA_DEV_BAD_ADAPTER is set in the pool's device status word.
 *   - Segments: seg_starts has S+1 entries with seg_starts[0] == 0,
 *     non-decreasing, seg_starts[S] == T; segment s covers tokens
 *     seg_starts[s] .. seg_starts[s+1]-1 and uses adapter seg_adapter[s].
 *     Empty segments are legal.  The table lives on the device, so it is
 *     checked there: a violation sets LORA_DEV_BAD_SEGMENTS and the affected
 *     tokens are computed against a clamped segment index (no access leaves
 *     the arrays).
 *   - Host-detectable errors (NULL pointer, bad size, misalignment, unknown
 *     matrix, a pool of the wrong dtype) return a negative status before any
 *     work is enqueued.  No kernel traps, asserts or waits without a bound.
 *
 * Thread safety: a pool may be used from one host thread at a time.
 */
#ifndef LORA_GB300_H
#define LORA_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct lora_pool lora_pool;   /* opaque; owns pages, tables, status word */
typedef void *lora_stream;            /* a cudaStream_t */

/* Return codes. */
enum {
    LORA_OK = 0,
    LORA_ERR_ARG = -1,           /* bad argument (NULL, size, alignment, dtype) */
    LORA_ERR_POOL_FULL = -2,     /* not enough free pages for the load */
    LORA_ERR_RANK = -3,          /* rank < 0, rank > max_rank, or ld_v < max_rank */
    LORA_ERR_NOT_LOADED = -4,    /* unload of an entry that holds no adapter */
    LORA_ERR_CUDA = -5,          /* a CUDA runtime call failed (no device, OOM, ...) */
    LORA_ERR_DEVICE_INDEX = -6,  /* lora_get_error: the device status word was non-zero */
    LORA_ERR_SHAPE = -7          /* h_in/h_out disagree with the matrix or exceed the page */
};

/* Element types of the pool (and of x, y, W). */
enum { LORA_F32 = 0, LORA_BF16 = 1 };

/* Bits of the device status word (see lora_get_error). */
enum {
    LORA_DEV_BAD_ADAPTER = 1,    /* an id >= max_adapters, or an unloaded adapter */
    LORA_DEV_BAD_SEGMENTS = 2,   /* a segment table that breaks the rules above */
    LORA_DEV_WAIT_TIMEOUT = 4,   /* a pipeline wait inside a kernel gave up */
    /* decode-step operators (lora_kv_pages.status): */
    LORA_DEV_BAD_SLOT = 8,       /* an append slot beyond the cache (the token is not stored) */
    LORA_DEV_BAD_POSITION = 16,  /* a rotation position outside the table (clamped) */
    LORA_DEV_BAD_LENGTH = 32,    /* a cached length below the drafted count or beyond the page table (clamped;
                                    eviction: a length or budget beyond its table, the request stays) */
    LORA_DEV_BAD_PAGE = 64       /* a page id outside the cache (clamped; eviction: the request stays) */
};

/*
 * Create a paged adapter pool on the current CUDA device.
 *   dtype        LORA_F32 or LORA_BF16.
 *   page_elems   H, elements per page; a multiple of 8 and >= every h_in and
 *                h_out later loaded.  One page holds one row of A_T (h_in
 *                elements) or one row of B (h_out elements).
 *   n_pages      pages to allocate (device memory = n_pages*H*sizeof(dtype)).
 *   max_rank     largest rank any adapter may have (1..1024).
 *   n_matrices   number of adapted matrices (e.g. layers x projections).
 *   max_adapters adapter ids run 0 .. max_adapters-1.
 * A rank-r adapter on one matrix occupies exactly 2r pages (r for A_T, r for
 * B), wherever they are free: ranks are mixed without padding (S-LoRA
 * slides 8 and 10).  On success *out owns all device memory of the pool.
 * Errors: LORA_ERR_ARG, LORA_ERR_CUDA (nothing is left allocated).
 */
int lora_pool_create(lora_pool **out, int dtype, int page_elems, int n_pages,
                     int max_rank, int n_matrices, int max_adapters);

/* Free every device and host resource of the pool.  Synchronises the device
 * first.  NULL is accepted. */
int lora_pool_destroy(lora_pool *pool);

/*
 * Load adapter `adapter` on matrix `matrix`: rank, scale, and HOST arrays
 *   A_T  rank x h_in  (row-major, pool dtype),
 *   B    rank x h_out (row-major, pool dtype).
 * The first load on a matrix fixes that matrix's (h_in, h_out); later loads
 * must match (else LORA_ERR_SHAPE).  A previous adapter in the same entry is
 * replaced (the device is synchronised first).  The device copy and the table
 * update run on `stream` (after the work already queued there) and the call
 * returns once they are complete: the adapter is resident for every kernel
 * launched afterwards, on any stream, and the host arrays may be freed at once.
 * rank == 0 is legal (the adapter adds nothing).
 * Errors: LORA_ERR_ARG, LORA_ERR_RANK, LORA_ERR_SHAPE, LORA_ERR_POOL_FULL
 * (the pool is unchanged), LORA_ERR_CUDA.
 */
int lora_pool_load(lora_pool *pool, int adapter, int matrix, int rank, float scale,
                   int h_in, int h_out, const void *A_T, const void *B, lora_stream stream);

/* Return the entry's pages to the free list and mark it unloaded.
 * Synchronises the device first, so no queued kernel still reads the pages.
 * Errors: LORA_ERR_ARG, LORA_ERR_NOT_LOADED, LORA_ERR_CUDA. */
int lora_pool_unload(lora_pool *pool, int adapter, int matrix);

/*
 * Asynchronous upload (S-LoRA slide 9: the adapters that queued requests will
 * need are copied to the GPU while the current batch computes; "Multi-LoRA
 * Serving", section "Memory: slots, tiers and paging": a host-memory tier with
 * prefetch lets one GPU serve far more adapters than its slots hold).
 *
 * lora_pool_load_async takes the arguments of lora_pool_load and copies the
 * host arrays into a pinned staging slot of the pool (a CPU copy: A_T and B
 * may be freed when the call returns), then ENQUEUES on `stream` the copy to
 * the device, the scatter into the adapter's pages and the copy of its table
 * record, and returns without waiting for them.  The adapter is resident for
 * work enqueued on `stream` after the call, and for work on other streams
 * ordered after it (an event recorded on `stream` after the call).  Kernels
 * of this library launched on `stream` right after it read the new record
 * (the record copy is the last step and is not a kernel).
 * Replacing an adapter: every kernel that may still read the old one must be
 * ordered before the call (same stream, or an event); its pages return to the
 * free list only once `stream` has passed the table update.
 * The staging ring has a few slots; a call that finds its slot still in use
 * waits for that slot's earlier copies.  When the free list is short, pages
 * retired by earlier asynchronous calls are waited for (oldest first).
 * Errors: as lora_pool_load (the pool is unchanged on any error).
 */
int lora_pool_load_async(lora_pool *pool, int adapter, int matrix, int rank, float scale,
                         int h_in, int h_out, const void *A_T, const void *B, lora_stream stream);

/* Marks the entry unloaded by a copy enqueued on `stream` (no wait); its
 * pages return to the free list once `stream` has passed it.  Kernels that
 * may still read the entry must be ordered before the call.
 * Errors: LORA_ERR_ARG, LORA_ERR_NOT_LOADED, LORA_ERR_CUDA. */
int lora_pool_unload_async(lora_pool *pool, int adapter, int matrix, lora_stream stream);

/* One adapter of a prefetch list: lora_pool_load's arguments. */
typedef struct lora_adapter_src {
    int adapter, matrix, rank;
    float scale;
    int h_in, h_out;
    const void *A_T;   /* rank x h_in, host, pool dtype */
    const void *B;     /* rank x h_out, host, pool dtype */
} lora_adapter_src;

/* Prefetch: lora_pool_load_async for every entry of `list` whose (adapter,
 * matrix) is not resident yet (resident entries are left as they are), in
 * list order, on `stream`.  Returns the number of uploads enqueued (>= 0), or
 * the first error (entries before it stay enqueued). */
int lora_pool_prefetch(lora_pool *pool, const lora_adapter_src *list, int n, lora_stream stream);

/* Pages currently free (host bookkeeping; pages retired by asynchronous calls
 * count once the stream has passed them -- an event query, no wait). -1 on
 * NULL. */
int lora_pool_free_pages(const lora_pool *pool);

/*
 * SGMV shrink (prefill; MBGMM for mixed ranks):
 *   v[t][j] = sum_k x[t][k] * A_T_a[j][k],  j < rank_a,  a = adapter of t's segment.
 * x: T x h_in (pool dtype); v: T x ld_v fp32 with ld_v >= the pool's max_rank.
 * Only v[t][0..rank_a-1] of tokens with a valid adapter are written.
 * Errors: LORA_ERR_ARG, LORA_ERR_RANK (ld_v < max_rank), LORA_ERR_SHAPE.
 */
int lora_sgmv_shrink(lora_pool *pool, int matrix, const void *x, float *v, int ld_v,
                     const int *seg_starts, const int *seg_adapter, int S, int T,
                     lora_stream stream);

/*
 * SGMV expand:  y[t][n] += scale_a * sum_j v[t][j] * B_a[j][n]  (read-modify-write).
 * v as produced by lora_sgmv_shrink; y: T x h_out (pool dtype).
 * Errors as lora_sgmv_shrink.
 */
int lora_sgmv_expand(lora_pool *pool, int matrix, const float *v, int ld_v, void *y,
                     const int *seg_starts, const int *seg_adapter, int S, int T,
                     lora_stream stream);

/*
 * BGMV (decode; MBGMV for mixed ranks): shrink and expand fused, one adapter
 * id per token:  y[t][n] += scale_a * sum_j (sum_k x[t][k] A_T_a[j][k]) B_a[j][n].
 * x: T x h_in, y: T x h_out (read-modify-write), token_adapter: T device int32.
 * Errors: LORA_ERR_ARG, LORA_ERR_SHAPE.
 */
int lora_bgmv(lora_pool *pool, int matrix, const void *x, void *y,
              const int *token_adapter, int T, lora_stream stream);

/* Bytes of device workspace lora_layer_forward needs for T tokens on this
 * matrix (0 on a bad argument). */
size_t lora_layer_forward_workspace_size(const lora_pool *pool, int matrix, int S, int T);

/*
 * Adapted layer: the shared base product for the whole mixed batch plus each
 * token's own low-rank term (the base product is computed once for every
 * token, and each token then receives its own adapter's update, "Multi-LoRA
 * Serving", section "The kernel trick: gather, do not merge"):
 *   y[t][n] = sum_k x[t][k] * W[n][k] + scale_a * sum_j (sum_k x[t][k] A_T_a[j][k]) B_a[j][n]
 * y is OVERWRITTEN.  W: h_out x h_in (pool dtype).  Tokens without an
 * adapter (or with an invalid one) get the base term only.
 * workspace: device scratch of at least lora_layer_forward_workspace_size()
 * bytes, owned by the caller, contents undefined on entry and exit.
 * Streams: part of the call's work (planning the rows whose M-tile is not
 * fused into the GEMM, and their shrink) may run on an internal stream, one per host thread
 * and device, that the call forks from `stream` and joins back to it with
 * events; the call's work as a whole stays ordered after earlier work on
 * `stream` and before later work on it, and under stream capture the fork
 * and join become graph edges.  The internal stream and its events are
 * created by the first such call on a thread: make that call outside stream
 * capture.
 * Errors: LORA_ERR_ARG (includes ws_bytes too small), LORA_ERR_SHAPE.
 */
int lora_layer_forward(lora_pool *pool, int matrix, const void *x, const void *W, void *y,
                       const int *seg_starts, const int *seg_adapter, int S, int T,
                       void *workspace, size_t ws_bytes, lora_stream stream);

/*
 * lora_layer_forward without caller-provided workspace, for callers that
 * cannot allocate device memory: a serving runtime whose device memory is
 * carved into a fixed arena at start-up, a decode loop that must not call
 * cudaMalloc/cudaFree (they synchronise the whole device), or a C plugin with
 * no allocator of its own.  The pages describe no such variant; it exists
 * for these callers only.
 *
 * Same operation, arguments and errors as lora_layer_forward, minus the
 * workspace.  The scratch comes from one static device array of
 * LORA_NOALLOC_SCRATCH_BYTES inside the library, which every GPU that loads
 * the library keeps until the process exits.  Requires
 * lora_layer_forward_workspace_size(pool, matrix, S, T) <=
 * LORA_NOALLOC_SCRATCH_BYTES (about T * max_rank * 4 bytes plus a small
 * per-token plan; else LORA_ERR_ARG) and the pool's device to be current
 * (else LORA_ERR_ARG).  The first call on a
 * device looks up the array's device address (cudaGetSymbolAddress); make
 * that first call before any stream capture.  All calls share the array:
 * calls whose work overlaps on the GPU race and must be serialised by the
 * caller.  Allocates nothing (no cudaMalloc/cudaFree or allocating library
 * routine).
 */
#define LORA_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)
int lora_layer_forward_noalloc(lora_pool *pool, int matrix, const void *x, const void *W, void *y,
                               const int *seg_starts, const int *seg_adapter, int S, int T,
                               lora_stream stream);

/*
 * FP8 base ("Multi-LoRA Serving - S-LoRA/Punica Batching, Adapter Hot-Swap &
 * Memory", the failure assumptions and "Operating it": the base may run in
 * FP8 while adapters trained on a bf16 base keep working in bf16).
 *
 * lora_quantize_e4m3: per-row quantisation of x (T x h bf16, device, h a
 * multiple of 8) to e4m3 codes q (T x h bytes, device, 8-byte aligned) and
 * fp32 scales sx (T, device):
 *   a = max_k |x[t][k]|, sx[t] = a / 448 and r = 448 / a (two fp32
 *             divisions per row),
 *   q[t][k] = e4m3(x[t][k] * r)  (the product in fp32, then rounded to the
 *             nearest e4m3 value, ties to the even code, saturating at +-448;
 *             e4m3 = 1 sign, 4 exponent bits with bias 7, 3 mantissa bits, no
 *             infinities);
 *   a row with a < 2^-120 (a row of zeros included) gets sx[t] = 1 and +0 codes.
 * Errors: LORA_ERR_ARG.
 */
int lora_quantize_e4m3(const void *x, int T, int h, void *q, float *sx, lora_stream stream);

/* Workspace lora_layer_forward_fp8 needs: lora_layer_forward's plus the
 * codes and scales of x (0 on a bad argument). */
size_t lora_layer_forward_fp8_workspace_size(const lora_pool *pool, int matrix, int S, int T);

/*
 * lora_layer_forward with an FP8 base product:
 *   y[t][n] = sx[t] * w_scale * sum_k q[t][k] * W8[n][k]
 *           + scale_a * sum_j (sum_k x[t][k] A_T_a[j][k]) B_a[j][n]
 * W8: h_out x h_in e4m3 codes (device, the base weight quantised by the
 * caller with the per-tensor scale w_scale > 0); x: bf16 as for
 * lora_layer_forward -- quantised here per row (lora_quantize_e4m3) for the
 * base product, used unquantised for the low-rank term.  The base product
 * runs on the tensor cores (kind::f8f6f4), so the pool must be bf16, h_in a
 * multiple of 128 and h_out a multiple of 32 (else LORA_ERR_SHAPE).  y is
 * overwritten.  Workspace, streams and errors as lora_layer_forward.
 */
int lora_layer_forward_fp8(lora_pool *pool, int matrix, const void *x, const void *W8, float w_scale, void *y,
                           const int *seg_starts, const int *seg_adapter, int S, int T,
                           void *workspace, size_t ws_bytes, lora_stream stream);

/*
 * Decode step of an attention block: the operators around the adapted
 * projections when every request adds one token, or a few drafted ones.
 *
 *   lora_w4_matvec        base product of a projection from 4-bit weights
 *                         (lora_bgmv then adds each token's adapter term)
 *   lora_kv_append        norm and rotation of queries and keys, append of
 *                         keys and values to a paged cache
 *   lora_tree_attention   attention of the drafted tokens over that cache
 *
 * and, for long streams of text, images and video whose cache stays bounded,
 *
 *   lora_kv_append_axes          append with positions of several axes
 *   lora_tree_attention_weights  attention that sums up each cached token's weight
 *   lora_kv_evict                eviction of the tokens with the least
 *
 * They take no pool: element types are arguments (LORA_F32 or LORA_BF16) and
 * all memory is the caller's.  Arithmetic is fp32 (products of bf16 operands
 * are exact in it); outputs are rounded once on store.
 */

/*
 * Matrix products with 4-bit weights:
 *   y[t][n] = sum_k x[t][k] * scales[n][k / group] * (code(n, k) - zero(n, k / group))
 * y (T x h_out) is OVERWRITTEN; x is T x h_in; both of type dtype, row-major, dense.
 *   codes   h_out x h_in/2 bytes: element k of row n is the low half of byte
 *           k/2 when k is even, the high half when it is odd; 0..15.
 *   scales  h_out x h_in/group, bf16.
 *   zeros   h_out x h_in/group bytes (0..15), or NULL: 8 everywhere.
 *   group   32, 64 or 128; h_in is a multiple of it.  h_out is any size.  Both are
 *           at most 2^31 - 2^16.
 * Meant for the few tokens of a decode step: the weights are read once for
 * every 64 tokens.
 * Errors: LORA_ERR_ARG, LORA_ERR_SHAPE (group, or h_in no multiple of it, or a
 * size beyond the limit).  The call has no status word: a pipeline wait inside a
 * kernel that gives up (after 2 s) leaves NaN in the outputs that it concerns.
 */
int lora_w4_matvec(int dtype, const void *x, int T, int h_in, const void *codes, const void *scales,
                   const void *zeros, int group, int h_out, void *y, lora_stream stream);

/*
 * One layer's paged key/value cache, in caller-owned device memory.
 *   k, v    n_pages x n_kv_heads x page_size x head_dim elements of dtype, 16-byte
 *           aligned.  A cache slot is page * page_size + offset in the page.
 *           n_pages * n_kv_heads * page_size is below 2^31.
 *   page_size  a power of two, 1..1024.   head_dim  a multiple of 8, 8..256.
 *   status  one device int32 that collects LORA_DEV_* bits of the calls on
 *           this cache (never cleared by them), or NULL.
 * The struct is read during the call only.
 */
typedef struct lora_kv_pages {
    int dtype, n_pages, page_size, n_kv_heads, head_dim;
    void *k, *v;
    int *status;
} lora_kv_pages;

/*
 * Norm, rotation and append, for T new tokens of any requests:
 *   per query head and key head h of token t, r = 1 / sqrt(mean_i h[i]^2 + eps):
 *     h[i] <- h[i] * r * norm[i]                 (q_norm for queries, k_norm for keys; NULL: no norm)
 *     (a, b) <- (a c_i - b s_i, a s_i + b c_i)   over the rot_dim/2 pairs i,
 *   where (a, b) are elements i and i + rot_dim/2, or 2i and 2i+1 when
 *   interleaved is non-zero, and c_i, s_i are entries i and rot_dim/2 + i of
 *   row positions[t] of cos_sin; elements from rot_dim on are not rotated.
 *   q_out[t] gets the queries; slot slots[t] of the cache gets the keys (as
 *   above) and the values (as they are).  slots[t] < 0: not stored.
 *   q, k, v    T rows of n_q_heads (n_kv_heads) x head_dim elements, ld_* elements
 *              apart (a column range of one fused projection is fine); 16-byte
 *              aligned, ld_* a multiple of 16 bytes.  q may be NULL with
 *              n_q_heads 0 (nothing but the append).
 *   cos_sin    n_pos x rot_dim fp32; rot_dim even, 0..head_dim (0: no
 *              rotation; cos_sin and positions may then be NULL).
 *   q_out      T x n_q_heads x head_dim, dense; may be q itself when q is dense.
 *   q_norm, k_norm   head_dim elements, 16-byte aligned.
 * Two tokens with one slot in one call leave either's values in it.
 * Errors: LORA_ERR_ARG, LORA_ERR_SHAPE (head counts, head_dim, page_size, rot_dim, ld_*).
 * Device-detected: LORA_DEV_BAD_SLOT, LORA_DEV_BAD_POSITION.
 */
int lora_kv_append(const lora_kv_pages *kv, const void *q, int ld_q, const void *k, int ld_k, const void *v, int ld_v,
                   int T, int n_q_heads, const int *positions, const long long *slots, const float *cos_sin,
                   int n_pos, int rot_dim, int interleaved, const void *q_norm, const void *k_norm, float eps,
                   void *q_out, lora_stream stream);

/*
 * lora_kv_append for tokens whose positions have several axes (time, height and
 * width of images and video): pair i of a head turns by the row of cos_sin at
 * positions[t][pair_axis[i]],
 *   c_i = cos_sin[positions[t][pair_axis[i]]][i], s_i = .. [rot_dim/2 + i].
 *   positions  T x n_axes device int32.   n_axes  1..LORA_MAX_AXES.
 *   pair_axis  the axes of the rot_dim/2 pairs, below n_axes: sections of the head, axes
 *              taken in turn, or any other order.  A text token has the same position on
 *              every axis.
 * Everything else, errors included, as lora_kv_append; an axis that no pair names
 * is not looked at.  Device-detected also: LORA_DEV_WAIT_TIMEOUT.
 *
 * This call and the two others of a bounded cache take their arguments as a struct, which
 * is read during the call only: they have about twenty, which a struct names, and which a
 * binding can pass as one.
 */
enum { LORA_MAX_AXES = 4, LORA_MAX_PAIRS = 128 };
typedef struct lora_append_axes {
    const void *q, *k, *v;
    void *q_out;
    const int *positions;
    const long long *slots;
    const float *cos_sin;
    const void *q_norm, *k_norm;
    int ld_q, ld_k, ld_v, T, n_q_heads, n_axes, n_pos, rot_dim, interleaved;
    float eps;
    unsigned char pair_axis[LORA_MAX_PAIRS];
} lora_append_axes;
int lora_kv_append_axes(const lora_kv_pages *kv, const lora_append_axes *args, lora_stream stream);

/* Bytes of device workspace that lora_tree_attention needs at most for up to T
 * drafted tokens of up to S requests (0 on a bad argument): a workspace of the
 * largest batch serves every smaller one. */
size_t lora_tree_attention_workspace_size(const lora_kv_pages *kv, int n_q_heads, int S, int T);

/*
 * Attention of drafted tokens over the paged cache.  Request s has the tokens
 * seg_starts[s] .. seg_starts[s+1]-1 (n_s of them, n_s >= 0) and kv_lens[s]
 * cached tokens, the last n_s of which are its drafted ones, in order (append
 * them first).  Cached token c of request s is at offset c % page_size of page
 * page_table[s * max_pages + c / page_size].
 *   out[t][h] = sum_c p_c v_c,   p = softmax over the visible c of scale * q[t][h] . k_c,
 * k and v of kv head h / (n_q_heads / n_kv_heads).  Visible to drafted token i
 * of a request: every c < kv_lens[s] - n_s; and drafted token j (c = kv_lens[s]
 * - n_s + j) when bit j % 64 of word j / 64 of row t of tree_mask is set
 * (mask_words words a row; j beyond them is not visible), or, with tree_mask
 * NULL, when j <= i.  With n_s = 1 and no mask this is plain decoding.  A token
 * that sees nothing gets zeros.  What a masked or unused slot holds (NaN
 * included) reaches no output.
 *   q, out     T x n_q_heads x head_dim of the cache's dtype, dense, 16-byte aligned;
 *              out may be q.
 *   scale      greater than 0.
 *   workspace  lora_tree_attention_workspace_size() bytes, contents undefined
 *              on entry and exit.
 * Softmax statistics and sums are fp32; for a bf16 cache the probabilities
 * enter the second product as bf16.
 * Errors: LORA_ERR_ARG (includes ws_bytes too small), LORA_ERR_SHAPE (also for
 * tables so wide that the list of key tiles could pass 2^31).
 * Device-detected: LORA_DEV_BAD_SEGMENTS, LORA_DEV_BAD_LENGTH,
 * LORA_DEV_BAD_PAGE, LORA_DEV_WAIT_TIMEOUT; no access leaves the arrays.  Where
 * segments overlap until they name more work than T tokens can have, nothing is
 * computed and out stays as it was.
 */
int lora_tree_attention(const lora_kv_pages *kv, const void *q, int n_q_heads, const int *seg_starts, int S, int T,
                        const int *kv_lens, const int *page_table, int max_pages, const long long *tree_mask,
                        int mask_words, float scale, void *out, void *workspace, size_t ws_bytes, lora_stream stream);

/*
 * lora_tree_attention that also sums up the weight that each cached token gets: for
 * every request with drafted tokens, kv head and cached token c,
 *   weights <- decay * weights + sum p_c  for c in the prefix (c < kv_lens[s] - n_s),
 *   weights <-                   sum p_c  for a drafted token, whose slot may hold anything before,
 * the sums over the request's drafted tokens that see c and the query heads of the
 * kv head, p as normalised there.  With decay 0 no weight is read.  Weights of requests
 * without drafted tokens, and of slots past a request, are left as they were.  out is
 * lora_tree_attention's, bit for bit.
 *   weights  n_pages x n_kv_heads x page_size fp32, slots as the cache's, 16-byte
 *            aligned; a prefix token's is what earlier calls left there.
 *   decay    0..1.   out  apart from q.
 *   workspace  16-byte aligned.  lora_tree_attention_weights_workspace_size() bytes; one of
 *            the largest call serves every smaller one.  Most of them are for scores of up to
 *            16 rows a kv head and request (128 in an fp32 cache), which take 4 * T *
 *            n_q_heads * max_pages * page_size bytes, as wide as the table however short the
 *            requests are.  A smaller workspace, down to that size for max_pages 0, does as
 *            well: where it does not hold a call's scores they are computed once more, which
 *            takes longer (1.1 to 5 times), and weights may differ in their last bits.
 * Every drafted token counts: rows of tokens that are rejected afterwards stay in the sums.
 * A page that several requests of the call share ends up with either's weights.  A
 * page outside the cache has none.  Errors, device-detected ones and bad tables as
 * lora_tree_attention (where nothing is computed, weights stay as well).
 */
typedef struct lora_attention_weights {
    float *weights;
    const void *q;
    const int *seg_starts, *kv_lens, *page_table;
    const long long *tree_mask;
    void *out, *workspace;
    size_t ws_bytes;
    int n_q_heads, S, T, max_pages, mask_words;
    float scale, decay;
} lora_attention_weights;
size_t lora_tree_attention_weights_workspace_size(const lora_kv_pages *kv, int n_q_heads, int S, int T, int max_pages);
int lora_tree_attention_weights(const lora_kv_pages *kv, const lora_attention_weights *args, lora_stream stream);

/*
 * Eviction from the paged cache.  Request s has kv_lens[s] cached tokens, in the
 * pages of its row of page_table.  If that is more than keep[s], then every kv
 * head h on its own keeps keep[s] of them: the last `recent`, the `first` first
 * (less where keep[s] does not hold both: the recent ones go before), and of the
 * others those with the greatest scores, of equal ones the lower index.  The kept
 * tokens' keys, values and weights move, in their order, to cached places 0 ..
 * keep[s] - 1, and new_lens[s] = keep[s]; places from there on are left as they
 * are.  Other requests (and those with keep[s] < 0) stay as they are, and
 * new_lens[s] = kv_lens[s].
 *   scores    n_pages x n_kv_heads x page_size fp32, slots as the cache's, 16-byte
 *             aligned; -0 equals 0, a NaN is below everything.
 *   weights   the same layout, moved with the tokens; may be scores (else they do not
 *             overlap), or NULL.
 *   keep      S device int32.
 *   kept      S x n_kv_heads x ld_kept device int32: for a request that loses tokens
 *             entry j < keep[s] of a row gets the index that the token at place j had; the
 *             rest is not written.  ld_kept is at least every budget that is used.
 *   new_lens  S device int32; new_lens and kept are apart from each other and from what
 *             is read.
 * The pages of a request that loses tokens are its own, each named once: a page shared
 * with another request, or named twice, ends up with either's tokens.
 * Errors: LORA_ERR_ARG, LORA_ERR_SHAPE.
 * Device-detected: LORA_DEV_BAD_LENGTH (a length beyond the table or below 0, a budget
 * beyond ld_kept), LORA_DEV_BAD_PAGE; the request concerned stays as it is.
 */
typedef struct lora_eviction {
    const float *scores;
    float *weights;
    const int *kv_lens, *page_table, *keep;
    int *kept, *new_lens;
    int S, max_pages, first, recent, ld_kept;
} lora_eviction;
int lora_kv_evict(const lora_kv_pages *kv, const lora_eviction *args, lora_stream stream);

/*
 * Synchronise the device, read the pool's device status word into
 * *device_status (may be NULL), and clear it.  Returns LORA_OK when the word
 * was zero, LORA_ERR_DEVICE_INDEX when any LORA_DEV_* bit was set, or
 * LORA_ERR_CUDA when the device reported an error.
 */
int lora_get_error(lora_pool *pool, int *device_status);

/* Static English text for a return code. */
const char *lora_strerror(int status);

/* Kernels this library has launched since it was loaded (host-side count,
 * summed over all pools; launches replayed from a captured CUDA graph are
 * not counted again). */
unsigned long long lora_launch_count(void);

/*
 * Two-tier adapter residency cache (host code; no device access).
 *
 * "Multi-LoRA Serving - S-LoRA/Punica Batching, Adapter Hot-Swap & Memory",
 * section "Memory: slots, tiers and paging" and its adapter-cache simulation:
 * a few GPU slots (here: adapters resident in the paged pool), backed by a
 * larger host-RAM tier, backed by disk.  Each tier keeps its adapters in
 * least-recently-used order and evicts the least recently used one when a
 * new one would exceed its slot count.  A request first looks in the GPU
 * tier; only on a GPU miss is the host tier looked up (and reordered).  A
 * slot count of 0 keeps nothing.
 *
 * The cache decides residency only and moves no data: a caller maps a GPU
 * hit to "already in the pool", a host hit to an upload from pinned host
 * memory (lora_pool_load_async), a disk hit to a fetch plus that upload, and
 * the GPU tier's eviction to lora_pool_unload_async.
 */
typedef struct lora_tier_cache lora_tier_cache;
enum { LORA_TIER_GPU = 0, LORA_TIER_HOST = 1, LORA_TIER_DISK = 2 };

/* Adapter ids 0..n_keys-1; both tiers start empty.  Errors: LORA_ERR_ARG. */
int lora_tier_cache_create(lora_tier_cache **out, int n_keys, int gpu_slots, int host_slots);
int lora_tier_cache_destroy(lora_tier_cache *cache);   /* NULL accepted */

/* One request for `adapter`: returns the tier that served it (LORA_TIER_*),
 * or LORA_ERR_ARG for an id out of range.  *gpu_evicted (may be NULL) gets
 * the adapter the GPU tier dropped to make room, or -1. */
int lora_tier_cache_touch(lora_tier_cache *cache, int adapter, int *gpu_evicted);

/* Bit 0: the adapter is in the GPU tier; bit 1: in the host tier.
 * LORA_ERR_ARG for an id out of range. */
int lora_tier_cache_resident(const lora_tier_cache *cache, int adapter);

/* Replays a request trace (adapter ids in 0..n_keys-1) through a fresh
 * cache: counts[0] GPU hits, counts[1] host hits, counts[2] disk loads.
 * Errors: LORA_ERR_ARG (NULL, n < 0, an id out of range). */
int lora_tier_sim(const int *trace, long long n, int n_keys, int gpu_slots, int host_slots,
                  long long *counts);

#ifdef __cplusplus
}
#endif

#endif /* LORA_GB300_H */
