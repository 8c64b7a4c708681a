/*
 * rq.h - ResidualQuant KV cache and decode attention for NVIDIA GB300 (sm_103a).
 *
 * ResidualQuant (the learnaivisually explainer "ResidualQuant stores
 * looped-Transformer KV caches as 2-bit residuals", and the ai4snews summary
 * of the arXiv paper) compresses the KV cache of a looped Transformer.  The
 * last loop of each loop group is stored as an INT4 "anchor"; every earlier
 * loop l is stored as a 2-bit code of the rotated residual
 *     u_l = R (kv_l - c_l * anchor_hat),  c_l = <kv_l, anchor_hat> / <anchor_hat, anchor_hat>,
 * with c_l kept in BF16 and R a fixed orthogonal rotation.  Channels are
 * grouped (g = 32 or 16) with an FP8-E4M3 scale and offset per group.
 * Decode attention rebuilds c * anchor_hat + R^T dequant(u) on chip and never
 * writes the rebuilt K/V to memory.
 *
 * Conventions for every entry point
 *   - Device pointers are caller-owned device memory (e.g. from PyTorch);
 *     the library never allocates or frees device memory and never
 *     synchronizes the device.  Host pointers are marked "host".
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Work is enqueued asynchronously on it.  The decode calls
 *     launch their kernels as programmatic dependents of the work before
 *     them on the stream, and those kernels read their inputs (queries,
 *     current K/V, seq_lens, cache) before waiting for it.  A kernel that
 *     does not release its dependents early (no griddepcontrol.launch_
 *     dependents) has completed before a call starts, so any such kernel may
 *     write the inputs; a kernel that does release early must not be the one
 *     that writes them (its writes are visible only to a kernel that has
 *     waited for it).
 *   - Argument errors are found on the host before anything is enqueued and
 *     return a status; nothing is launched then.  A failed launch returns
 *     RQ_ERR_CUDA.  Faults inside a kernel surface on a later CUDA call.
 *   - Device pointers must be 16-byte aligned (RQ_ERR_ALIGNMENT).
 *   - A cache belongs to the device that was current when it was created;
 *     a call on it made with another device current returns
 *     RQ_ERR_INVALID_ARG (its memory is not addressable from there).
 *   - Supported shapes: head_dim in {96, 128}; group_size in {16, 32} dividing
 *     head_dim; loops_per_group in [1, 16]; num_query_heads a multiple of
 *     num_heads.  Others: RQ_ERR_UNSUPPORTED.
 *
 * Entry points: rq_cache_bytes / rq_cache_create (contiguous layout) or
 * rq_cache_paged_bytes / rq_cache_create_paged (block-table layout);
 * rq_append (compress new tokens: prefill, or one decode token);
 * rq_decode_workspace_bytes, rq_decode_attention (one loop's attention) and
 * rq_decode_attention_append (the anchor loop's attention plus the current
 * token's append); rq_decode_attention_noalloc (scratch inside the library);
 * rq_bf16_workspace_bytes / rq_decode_attention_bf16 (the uncompressed
 * comparator); rq_tree_workspace_bytes / rq_tree_attention (several drafted
 * tokens per row, each seeing its own ancestors); rq_pages_workspace_bytes and
 * rq_pages_copy / _fork / _reserve / _free / _compact (page bookkeeping of the
 * paged layout); rq_rope (rotary positions); rq_status_string.
 *
 * ---------------------------------------------------------------------------
 * Cache byte layout (this library's format; the pages fix the record
 * contents, not their placement)
 *   The cache is L x G x max_batch x H regions, index
 *   ((layer * G + group) * max_batch + b) * H + h, each `region` bytes.
 *   A region holds planes AK, AV, then RK_j, RV_j for j = 0 .. P-2.
 *   Each plane is ntiles = ceil(max_seq_len / 64) tiles of 64 token slots;
 *   tile t holds positions 64t .. 64t+63.
 *     anchor tile  (AK, AV)  : codes[64 * d/2] | meta[64 * ng * 2]
 *     residual tile (RK, RV) : codes[64 * d/4] | meta[64 * ng * 2] | c[64 * 2]
 *   K codes are token-major: row r = the token's d codes;
 *     INT4 byte i = ch 2i (bits 0-3) | ch 2i+1 (bits 4-7);
 *     INT2 byte i = ch 4i+m in bits 2m..2m+1.
 *   V codes are channel-major: row ch = that channel's 64 token codes in
 *     32-bit words; INT4 word w (tokens 8w..8w+7): byte i = token 8w+i
 *     (bits 0-3) | token 8w+4+i (bits 4-7); INT2 word j (tokens 16j..16j+15):
 *     byte i holds token 16j+4m+i in bits 2m..2m+1, m = 0..3.  Masking a word
 *     with 0x0F0F0F0F, 0xF0F0F0F0 or 0x03030303 << 2m leaves four consecutive
 *     tokens, one per byte.
 *   meta row r: for each channel group, the E4M3 scale byte then the E4M3
 *     offset byte.  c slot r: BF16, little-endian.
 *   Every tile and sub-block size is a multiple of 16 bytes.
 *
 * Quantizer (both code widths): per group, o = E4M3(min), s = E4M3((max-min)/(2^b-1)),
 * rounded to nearest even and saturating at +-448; code = the nearest grid
 * point o + k*s to the exact value, ties to even k, clamped to [0, 2^b-1];
 * s == 0 gives code 0.  Dequantized value: s * code + o.
 * ---------------------------------------------------------------------------
 */
#ifndef RQ_H_
#define RQ_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum rq_status {
  RQ_OK = 0,
  RQ_ERR_INVALID_ARG = 1,   /* null pointer, index out of range, bad count */
  RQ_ERR_ALIGNMENT = 2,     /* a device pointer is not 16-byte aligned */
  RQ_ERR_CAPACITY = 3,      /* batch > max_batch, or a write past max_seq_len */
  RQ_ERR_WORKSPACE = 4,     /* workspace smaller than the *_workspace_bytes value */
  RQ_ERR_CUDA = 5,          /* a CUDA runtime call or kernel launch failed */
  RQ_ERR_UNSUPPORTED = 6,   /* head_dim / group_size / loops outside the supported set */
  RQ_ERR_TIMEOUT = 7        /* a device-side wait gave up (reported via the status word) */
} rq_status;

typedef enum rq_mode {
  RQ_MODE_SHARED = 0,   /* every earlier loop coded against the anchor: 2 plane reads per loop */
  RQ_MODE_CHAINED = 1,  /* loop l coded against the rebuilt loop l+1: reads grow with distance */
  RQ_MODE_NORM_RATIO = 2, /* flag, OR'd with one of the above: the stored coefficient is the
                            norm ratio ||kv_l|| / ||ref|| (the scaling the arXiv summary lists
                            beside least squares among its appendix comparisons) instead of
                            the least-squares <kv_l, ref> / <ref, ref>; decode is unchanged */
  RQ_MODE_HADAMARD = 4  /* flag: the rotation is R = H_d / sqrt(d), H_d the Sylvester Hadamard
                           matrix (entry (i, k) = (-1)^popcount(i & k)), applied as a fast
                           Walsh-Hadamard transform (d log d adds) wherever R or R^T acts;
                           head_dim 128 only.  The explainer's related-explainers list points
                           to a 2-bit KV cache built on a Hadamard rotation; the summary's
                           ablation compares rotation methods.  R_dev may then be NULL. */
} rq_mode;

/* Shape of one cache.  The anchor is 4-bit and residuals 2-bit (fixed). */
typedef struct rq_config {
  int32_t num_layers;       /* L: layers of the shared block */
  int32_t loops_per_group;  /* P: loops per anchor group; the last one is the anchor */
  int32_t num_groups;       /* G: loop groups (Ouro-1.4B: 1 group of 4; Huginn-3.5B: 8 of 4) */
  int32_t num_heads;        /* H: KV heads (the cache stores these) */
  int32_t head_dim;         /* d: 96 or 128 */
  int32_t group_size;       /* g: 16 or 32 channels per quantization group */
  int32_t max_batch;        /* rows of the cache */
  int32_t max_seq_len;      /* token capacity per (layer, group, row, head) */
  int32_t mode;             /* rq_mode: SHARED or CHAINED, optionally | NORM_RATIO | HADAMARD */
  int32_t num_query_heads;  /* Hq: query heads; 0 (or H) = multi-head attention, else a multiple
                               of H (grouped-query: query head qh attends with KV head
                               qh / (Hq / H)).  Decode calls take q and out with Hq heads and
                               the current token's K/V with H heads. */
} rq_config;

typedef struct rq_cache rq_cache;   /* opaque host-side handle; holds no device memory */

/* Bytes of device memory a cache of this shape needs (0 if the shape is invalid).
 * Host only; no CUDA call. */
size_t rq_cache_bytes(const rq_config* cfg);

/* Bind a cache to caller memory.
 *   cfg    host; copied.  cfg->mode: RQ_MODE_SHARED or RQ_MODE_CHAINED, optionally
 *          OR'd with RQ_MODE_NORM_RATIO and RQ_MODE_HADAMARD.  In binary32 the
 *          Hadamard transform runs butterfly stages h = 1, 2, ..., d/2, each pair
 *          (j, j+h) becoming (a+b, a-b) rounded, then one product with the
 *          binary32 value of 1/sqrt(d); the stored codes follow that order.
 *   dev_buf device, >= rq_cache_bytes(cfg) bytes, 16-byte aligned.  Its
 *          contents are the cache; the caller zero-fills it before first use
 *          (only needed for byte-exact comparisons: unwritten slots are never read).
 *   R_dev  device float32 [d][d] row-major, the rotation (orthogonal); caller
 *          keeps it alive and unchanged while the cache is used.  Unused (may be
 *          NULL) with RQ_MODE_HADAMARD.
 *   out    host; receives the handle.  Free it with rq_cache_destroy.
 * Errors: INVALID_ARG (null), UNSUPPORTED (shape), CAPACITY (bytes too small),
 * ALIGNMENT. */
rq_status rq_cache_create(const rq_config* cfg, void* dev_buf, size_t bytes,
                          const float* R_dev, rq_cache** out);

/* Paged layout (block table, as a paged serving engine lays out its KV cache).
 * Instead of a contiguous capacity per (layer, group, row, head), each
 * (layer, group) owns a pool of num_pages pages; a page holds one 64-token tile
 * of every plane (anchor K/V, every residual K/V, with their metadata and
 * coefficients, laid out as in the contiguous tile) of every head:
 *   pool(layer, group) = base + (layer * G + group) * num_pages * page_bytes
 *   page p, head h:      pool + p * page_bytes + h * head_block
 *   head_block = 2 * anchor_tile + 2 * (P - 1) * residual_tile, page_bytes = H * head_block
 *   inside a head block: anchor K tile, anchor V tile, then residual plane j's
 *   K and V tiles for j = 0 .. P-2.
 * Tile t (token positions 64t .. 64t+63) of batch row b lives in page
 * block_table[b * max_tiles_per_row + t]; the same table serves every layer and
 * group.  The caller assigns pages (distinct for distinct (row, tile) pairs in
 * use) before a call touches the tile, and keeps the table unchanged while
 * calls that read it run.  An entry outside [0, num_pages) for a tile a call
 * touches is not followed: the call sets status word [2], reads page 0 for the
 * attention, and skips the append's write.  Everything else (appends, decode,
 * the fused call, all modes) is the same as for the contiguous layout. */
size_t rq_cache_paged_bytes(const rq_config* cfg, int32_t num_pages);   /* 0 if invalid */

/*   dev_pool     device, >= rq_cache_paged_bytes(cfg, num_pages), 16-byte aligned
 *   block_table  device int32 [max_batch][max_tiles_per_row], 16-byte aligned,
 *                max_tiles_per_row >= ceil(max_seq_len / 64); caller-owned
 *   R_dev, out   as rq_cache_create
 * Errors: INVALID_ARG (null, num_pages <= 0, table too narrow), UNSUPPORTED,
 * CAPACITY, ALIGNMENT, CUDA. */
rq_status rq_cache_create_paged(const rq_config* cfg, int32_t num_pages, void* dev_pool, size_t bytes,
                                const int32_t* block_table, int32_t max_tiles_per_row, const float* R_dev,
                                rq_cache** out);

/* Free the host handle (not the caller's device memory).  NULL is accepted. */
rq_status rq_cache_destroy(rq_cache* cache);

/* Compress n_tokens new tokens of one (layer, group) for rows 0..batch-1 and
 * write them at positions seq_lens[b] .. seq_lens[b] + n_tokens - 1.
 * Follows the explainer's stored-overlay paragraph: anchor = last loop, INT4;
 * every earlier loop: LS coefficient (BF16), rotated residual, INT2.
 *   kv        device bf16 [P][2][batch][H][n_tokens][d] (loop, K/V, row, head, token, channel);
 *             at decode time this is the BF16 temporary buffer with n_tokens = 1.
 *   seq_lens  device int32 [batch], tokens already cached per row (not modified;
 *             the caller advances it afterwards).  Every seq_lens[b] + n_tokens
 *             must be <= max_seq_len: the host cannot see device values, so the
 *             kernel skips a row that would overflow and sets status[1] = 1.
 *   status    device int32[4] or NULL; see the status word under
 *             rq_decode_workspace_bytes (the workspace's first 16 bytes serve).
 * Errors: INVALID_ARG, CAPACITY (batch > max_batch or n_tokens > max_seq_len),
 * ALIGNMENT, UNSUPPORTED (batch * num_heads > 65535), CUDA. */
rq_status rq_append(rq_cache* cache, int32_t layer, int32_t group, int32_t batch,
                    const void* kv, const int32_t* seq_lens, int32_t n_tokens,
                    int32_t* status, void* stream);

/* Workspace (device bytes) one rq_decode_attention call needs for `batch` rows
 * on the current device.  The workspace must be zero-filled once before its
 * first use (the status word must start at zero).  Its first 16 bytes
 * are the status word (int32[4]): [0] != 0 after a device-side wait timed out,
 * [1] != 0 after an append skipped a row that would overflow, [2] != 0 after a
 * call met a block-table entry outside the page pool (paged layout).  [3] is
 * written by rq_pages_reserve only. */
size_t rq_decode_workspace_bytes(const rq_config* cfg, int32_t batch);

/* One decode-attention call: query loop `loop` (0-based; loop == P-1 is the
 * anchor loop) of (layer, group), for rows 0..batch-1, all heads.
 * Keys/values are the seq_lens[b] cached tokens rebuilt for this loop, plus
 * the current token's BF16 K/V (the temporary buffer: the explainer's paragraph
 * on why the last-loop anchor forces the current token to stay in BF16).
 *   q              device bf16 [batch][H][d]
 *   k_cur, v_cur   device bf16 [batch][H][d], this loop's K/V of the current token
 *   seq_lens       device int32 [batch]
 *   softmax_scale  e.g. 1/sqrt(d)
 *   out            device float32 [batch][H][d]
 *   workspace      device, >= rq_decode_workspace_bytes(cfg, batch), zeroed once
 * Split-K over the sequence: each CTA of a balanced grid streams its range of
 * tiles into one partial softmax state per (CTA, row, head); a merge kernel
 * then combines the partial softmax
 * states, adds the current token and applies R^T once.
 * Chained mode reads the anchor and every residual plane from this loop to
 * the anchor; decode supports it for loops_per_group <= 8 (UNSUPPORTED beyond,
 * and for head_dim 128 with group_size 16 and 8 loops: one call's working set
 * would not fit one SM's shared memory).
 * Errors: INVALID_ARG, CAPACITY (batch > max_batch), WORKSPACE, ALIGNMENT,
 * UNSUPPORTED, CUDA. */
rq_status rq_decode_attention(rq_cache* cache, int32_t layer, int32_t group, int32_t loop,
                              int32_t batch, const void* q, const void* k_cur, const void* v_cur,
                              const int32_t* seq_lens, float softmax_scale, float* out,
                              void* workspace, size_t workspace_bytes, void* stream);

/* The group's last-loop (anchor-loop) call and the current token's append in
 * one call: the same output as rq_decode_attention(loop = P-1) and then the
 * same cache bytes as rq_append(n_tokens = 1) with the same kv_cur.  The
 * explainer's temporary-buffer paragraph: the current token of every loop
 * stays in BF16 until the anchor loop has produced its K/V; that is the moment
 * this call compresses it.  The merge kernel of the call does the append, one
 * CTA per (row, head); it computes while the attention kernel still streams
 * the cache and writes the new slot only after that kernel has finished.
 *   q          device bf16 [batch][H][d], query of loop P-1
 *   kv_cur     device bf16 [P][2][batch][H][d] (loop, K/V, row, head, channel):
 *              the current token of every loop (rq_append's kv with
 *              n_tokens = 1); its loop P-1 blocks are the attention's k_cur, v_cur
 *   seq_lens   device int32 [batch]: tokens already cached; the attention reads
 *              them and the token is written at position seq_lens[b] (not
 *              modified; the caller advances it afterwards).  A row with
 *              seq_lens[b] + 1 > max_seq_len is attended but not appended, and
 *              the workspace's status word gets [1] = 1.
 *   softmax_scale, out, workspace, workspace_bytes: as rq_decode_attention
 * Errors: as rq_decode_attention. */
rq_status rq_decode_attention_append(rq_cache* cache, int32_t layer, int32_t group, int32_t batch,
                                     const void* q, const void* kv_cur, const int32_t* seq_lens,
                                     float softmax_scale, float* out, void* workspace,
                                     size_t workspace_bytes, void* stream);

/* Rows one decode call (rq_decode_attention, _append, _noalloc, _bf16) may
 * cover; a larger batch returns RQ_ERR_UNSUPPORTED (split it into calls). */
#define RQ_MAX_DECODE_BATCH 256

/* Size of the workspace built into the library for rq_decode_attention_noalloc
 * (2 MiB of device memory, held on every device that loads the library until
 * the process exits).  With 152 SMs and head_dim 128 it covers batch *
 * num_query_heads up to about 740 (row, head) pairs (split-K partials of
 * 1040 B and a query pack of 1152 B per pair, plus 456 CTA partials). */
#define RQ_NOALLOC_WORKSPACE_BYTES (2u * 1024u * 1024u)

/* rq_decode_attention for callers that cannot allocate device memory.
 * The paper has no counterpart to this entry point.  Some callers are handed
 * their buffers and may not allocate more: a plugin whose host application
 * owns all device memory, a process under a memory budget fixed up front,
 * or a path on which an allocation could block or fail.  This call takes
 * the same arguments as rq_decode_attention, less the workspace, and
 * performs no device allocation: its scratch (status word, split-K
 * partials, query packs) lives in one array of RQ_NOALLOC_WORKSPACE_BYTES inside
 * the library.
 *   status   device int32[4] or NULL: receives the call's status word (as
 *            under rq_decode_workspace_bytes) on `stream` after the kernel.
 * The first call on a device looks up the array's device address (once per
 * device, with that device current); make that first call before any
 * stream capture.  Each call clears the part of the array it uses on
 * `stream` before its kernel, then runs the same kernel as
 * rq_decode_attention.  All calls share the one array: calls that overlap
 * on the GPU (other streams, other host threads) race and give wrong
 * results, so serialize them.  On one stream the clear is an ordinary
 * stream operation: it starts after the previous call's kernels have
 * finished, so consecutive noalloc calls do not overlap their start with
 * the previous call's tail the way rq_decode_attention calls with
 * workspaces do.  The status copied to `status` is the current call's only
 * (the clear zeroes the word first); a caller that wants to know whether
 * any of several calls failed ORs the words it receives.
 * Errors: as rq_decode_attention; WORKSPACE when the call needs more than
 * RQ_NOALLOC_WORKSPACE_BYTES (too many rows x heads for the built-in array;
 * use rq_decode_attention with a workspace of rq_decode_workspace_bytes). */
rq_status rq_decode_attention_noalloc(rq_cache* cache, int32_t layer, int32_t group,
                                      int32_t loop, int32_t batch, const void* q,
                                      const void* k_cur, const void* v_cur,
                                      const int32_t* seq_lens, float softmax_scale, float* out,
                                      int32_t* status, void* stream);

/* Workspace (device bytes) for rq_decode_attention_bf16; same zero-once rule. */
size_t rq_bf16_workspace_bytes(int32_t batch, int32_t num_heads, int32_t head_dim);

/* Uncompressed comparator: the same split-K decode attention over plain BF16
 * K/V (the role the pages give vLLM's BF16 FlashAttention baseline).
 *   k_cache, v_cache  device bf16 [batch][H][max_seq][d]
 *   k_cur, v_cur, q   device bf16 [batch][H][d]
 *   seq_lens          device int32 [batch] (each <= max_seq)
 *   out               device float32 [batch][H][d]
 * Errors: INVALID_ARG, UNSUPPORTED (head_dim), WORKSPACE, ALIGNMENT, CUDA. */
rq_status rq_decode_attention_bf16(const void* k_cache, const void* v_cache,
                                   const void* k_cur, const void* v_cur, const void* q,
                                   const int32_t* seq_lens, int32_t batch, int32_t num_heads,
                                   int32_t head_dim, int32_t max_seq, float softmax_scale,
                                   float* out, void* workspace, size_t workspace_bytes,
                                   void* stream);

/* ---------------------------------------------------------------------------
 * Attention of a tree of drafted tokens
 * --------------------------------------------------------------------------- */

/* Drafted tokens per row that one rq_tree_attention call may cover. */
#define RQ_MAX_TREE_NODES 256

/* Workspace (device bytes) of one rq_tree_attention call for `batch` rows of
 * n_nodes drafted tokens on the current device (0 if the shape is invalid).
 * Zero-filled once before its first use; the first 16 bytes are the status
 * word, as under rq_decode_workspace_bytes.  Calls that may run at the same
 * time need a workspace each. */
size_t rq_tree_workspace_bytes(const rq_config* cfg, int32_t batch, int32_t n_nodes);

/* Attention of the drafted tokens of a speculative step: node t of row b
 * attends, for query loop `loop` of (layer, group), the row's seq_lens[b]
 * cached tokens (rebuilt for this loop, as rq_decode_attention does) and those
 * drafted tokens of its row that its mask names, whose K/V of this loop are
 * still in BF16.  A node sees itself only if its own bit is set.  The
 * cache is only read; append the accepted path with rq_append afterwards.
 *   n_nodes      T, drafted tokens per row: 1 .. RQ_MAX_TREE_NODES
 *   q            device bf16 [batch][Hq][T][d]
 *   k_new, v_new device bf16 [batch][H][T][d]: this loop's block of a
 *                [P][2][batch][H][T][d] buffer, the layout that rq_append takes
 *   mask         device uint64 [batch][T][ceil(T / 64)], or NULL: bit j % 64 of
 *                word j / 64 of node t set = node t sees drafted token j.  Bits
 *                at or behind the row's node count are ignored.  NULL: node t
 *                sees drafted tokens 0 .. t (a single drafted sequence).
 *   node_counts  device int32 [batch] or NULL: nodes in use per row (taken into
 *                0 .. T); the output rows of nodes behind the count are not
 *                written, their inputs do not enter any result (they may hold
 *                anything).  NULL: T for every row.
 *   seq_lens     device int32 [batch]
 *   out          device bf16 [batch][Hq][T][d]; zero for a node that sees no key
 * A K or V that a node's mask hides does not enter that node's result, not even
 * when it is infinite or NaN.  q (finite: up to 2^120 in magnitude) is scaled per
 * node by a power of two and kept in 16-bit floating point (11 significant bits),
 * as are the rebuilt K/V and the softmax weights; scores, softmax sums and
 * accumulators are float32.  The rebuilt V may be up to 65504 in magnitude.  (Beyond
 * what rq_append makes of such V: in a residual loop of a shared-anchor cache |c| times
 * a V group's scale has to stay below 2^18.)  A V below 1/2 with a coefficient below
 * 1/4 is met to within 1.25 * 2^-10; there a coefficient below 2^-126 counts as zero.
 * With T = 1 and a mask that names the token itself this is
 * rq_decode_attention with a BF16 result.
 * Chained caches (RQ_MODE_CHAINED) are read as rq_decode_attention reads them, but
 * node by node: a call takes about a hundred times what it takes on a shared-anchor
 * cache, so a single token there is better served by rq_decode_attention.
 * Errors: as rq_decode_attention; INVALID_ARG (n_nodes < 1), UNSUPPORTED
 * (n_nodes > RQ_MAX_TREE_NODES, batch > RQ_MAX_DECODE_BATCH, more than 2^30
 * queries, batch * H * ceil(Hq / H * T / 64) * ceil(max_seq_len / 128) > 2^31 - 1). */
rq_status rq_tree_attention(rq_cache* cache, int32_t layer, int32_t group, int32_t loop,
                            int32_t batch, int32_t n_nodes, const void* q, const void* k_new,
                            const void* v_new, const uint64_t* mask, const int32_t* node_counts,
                            const int32_t* seq_lens, float softmax_scale, void* out,
                            void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Pages of a paged cache
 *
 * Bookkeeping on the device, in stream order, for callers that branch rows
 * (beams, parallel samples, drafted paths).  It uses the cache's block table
 * (these calls write the table that rq_cache_create_paged was given) and one
 * array the caller owns:
 *   refs   device int32 [num_pages]: how many table entries name the page;
 *          0 = free.  A caller that lets these calls do all its paging starts
 *          with refs zero and every table entry -1 (no page).
 * Rows that share a page (refs > 1) may all read it; before a row writes to it
 * (rq_append, rq_decode_attention_append), rq_pages_reserve gives the row a page
 * of its own.  Table entries outside [0, num_pages) name no page; none of these
 * calls follows one.
 *   status device int32[4] or NULL: [1] = 1 after a row was skipped, [2] = 1
 *          after a page pair was skipped, [3] = 1 when the free pages ran out.
 * A call on a cache of the contiguous layout returns RQ_ERR_INVALID_ARG.  All
 * other errors: INVALID_ARG (null, negative count), CAPACITY (more rows than
 * max_batch, n_tokens > max_seq_len), ALIGNMENT, WORKSPACE, CUDA.
 * --------------------------------------------------------------------------- */

/* Workspace (device bytes) of rq_pages_reserve and rq_pages_compact for caches
 * of this shape with num_pages pages; needs no initial value.  0 if invalid. */
size_t rq_pages_workspace_bytes(const rq_config* cfg, int32_t num_pages);

/* Copy page src[i] to page dst[i], in every layer and group, i < n.  Table and
 * counts are not touched.  A pair is skipped (status [2]) when a page is outside
 * the pool, when dst[i] is the source of another pair, or when an earlier pair
 * has the same dst; src[i] == dst[i] does nothing.
 *   src, dst   device int32 [n], 16-byte aligned; n <= num_pages (CAPACITY) */
rq_status rq_pages_copy(rq_cache* cache, int32_t n, const int32_t* src, const int32_t* dst,
                        int32_t* status, void* stream);

/* Row dst_rows[i] takes the pages of row src_rows[i] (shared, no bytes are
 * copied) and gives up its own, i < n: all sources are read before any row is
 * changed, so a permutation of beams is one call.  A dst row named twice takes
 * the last pair's source.  A row index outside [0, max_batch) skips its pair
 * (status [1]).  The caller moves the rows' lengths.
 *   src_rows, dst_rows  device int32 [n], n <= max_batch; more than 6144 pairs:
 *                       UNSUPPORTED */
rq_status rq_pages_fork(rq_cache* cache, int32_t n, const int32_t* src_rows, const int32_t* dst_rows,
                        int32_t* refs, int32_t* status, void* stream);

/* Make the tiles of positions seq_lens[b] .. seq_lens[b] + n_tokens - 1 of rows
 * 0 .. batch-1 writable: an entry that names no page gets a free page; a page
 * that other entries share is replaced by a free page, which receives a copy of
 * its bytes when the tile already holds tokens of the row (copy on write).  When
 * every holder of a page asks in one call, the last of them keeps it.  Requests are
 * served in row, then tile order, from the lowest free page up.  Where the free
 * pages run out an entry stays as it is (status [3]): pages may then still be shared
 * by rows that asked, and no row may be written to before a reserve has succeeded.  A row with a negative
 * length or seq_lens[b] + n_tokens > max_seq_len is skipped (status [1]).  n_tokens = 0 does
 * nothing. */
rq_status rq_pages_reserve(rq_cache* cache, int32_t batch, const int32_t* seq_lens, int32_t n_tokens,
                           int32_t* refs, int32_t* status, void* workspace, size_t workspace_bytes,
                           void* stream);

/* Give up the tiles of rows[i] at or behind token keep[i] (tiles that hold none
 * of the first keep[i] tokens), i < n: their entries become -1 and their pages
 * lose one holder.  keep NULL: the whole row.  A row named twice loses what any
 * of its pairs gives up.  A row index outside [0, max_batch) is skipped (status [1]).
 *   rows, keep   device int32 [n] */
rq_status rq_pages_free(rq_cache* cache, int32_t n, const int32_t* rows, const int32_t* keep,
                        int32_t* refs, int32_t* status, void* stream);

/* Move pages so that the used ones are 0 .. used-1: the i-th free page below
 * `used` takes the bytes, the count and the table entries of the i-th used page at or above it.
 *   used   device int32, receives the number of pages with refs > 0 */
rq_status rq_pages_compact(rq_cache* cache, int32_t* refs, int32_t* used, int32_t* status,
                           void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Rotary positions
 * --------------------------------------------------------------------------- */

typedef enum rq_dtype { RQ_BF16 = 0, RQ_F16 = 1, RQ_F32 = 2 } rq_dtype;

typedef enum rq_rope_scaling {
  RQ_ROPE_PLAIN = 0,    /* f_i = theta^(-2i / rotary_dim) */
  RQ_ROPE_LINEAR = 1,   /* f_i / factor: positions squeezed by `factor` */
  RQ_ROPE_BASE = 2,     /* theta replaced by theta * factor^(r / (r - 2)): the slowest frequency
                           is divided by `factor`, the fastest stays */
  RQ_ROPE_PARTS = 3     /* f_i (k_i + (1 - k_i) / factor), k_i = clamp((u_i - low_turns) /
                           (high_turns - low_turns), 0, 1), u_i = original_len f_i / 2pi: the turns
                           that pair i makes over the original length.  The ramp is linear in the
                           turns; models trained with one that is linear in the pair's index i,
                           between two bounds rounded to indices, have other frequencies */
} rq_rope_scaling;

/* How rq_rope turns a head. */
typedef struct rq_rope_config {
  int32_t head_dim;      /* channels per head, 2 .. 512 */
  int32_t rotary_dim;    /* r: the first r channels are rotated (even, 2 .. min(head_dim, 256)); the
                            others are copied */
  int32_t interleaved;   /* 0: channel i pairs with i + r/2; 1: channel 2i pairs with 2i + 1 */
  int32_t inverse;       /* 1: rotate by the negative angle.  The map is linear and this is its
                            transpose: out = gradient of in for in = gradient of out */
  int32_t scaling;       /* rq_rope_scaling */
  int32_t original_len;  /* RQ_ROPE_PARTS: context the model was trained for */
  double theta;          /* > 1, e.g. 10000 */
  double factor;         /* > 0; not used by RQ_ROPE_PLAIN */
  double low_turns, high_turns;   /* RQ_ROPE_PARTS: low < high */
  double magnitude;      /* the rotated channels are multiplied by it (0 counts as 1) */
} rq_rope_config;

/* One tensor [batch][heads][n][d] read and written by rq_rope: the element
 * strides of row, head and token; channels are contiguous.  Any strides do;
 * pointers and strides that are multiples of 16 bytes are faster.  out's elements
 * are distinct (strides that put two results of it in one place are refused).
 * out may be in (with the same strides); otherwise the two must not overlap, nor
 * q's out and k's, nor either's out and the other's in: these are not checked. */
typedef struct rq_rope_tensor {
  const void* in;
  void* out;
  int32_t heads;
  int64_t in_row, in_head, in_token;
  int64_t out_row, out_head, out_token;
} rq_rope_tensor;

/* Rotate queries and keys by their positions: pair (a, b) of frequency i becomes
 * magnitude * (a cos - b sin, b cos + a sin) at angle position * f_i.  Positions
 * are start[b] + offsets[b][t], offsets NULL: start[b] + t, so with start =
 * seq_lens a prompt, a decoded token (n = 1) or the nodes of a drafted tree
 * (offsets = their depths) sit where they belong.  Angles are taken modulo a
 * turn in 64-bit fixed point from float64 frequencies: off by less than 2^-51 of
 * a turn a position for theta >= 10000, 2^-20 at the farthest.  Arithmetic is
 * float32, rounded once to the tensors' type.
 *   dtype    rq_dtype of every tensor
 *   q, k     host; k (or q) may be NULL
 *   start    device int32 [batch], or NULL: zeros
 *   offsets  device int32 [batch][n] or NULL
 * The tensors need only be aligned to their element.
 * Errors: INVALID_ARG (null, bad count or config, a stretched base or frequencies not
 * finite in float64, results of one tensor that overlap), ALIGNMENT, UNSUPPORTED
 * (head_dim or rotary_dim outside the ranges, heads x batch > 2^30), CUDA. */
rq_status rq_rope(const rq_rope_config* cfg, int32_t dtype, int32_t batch, int32_t n,
                  const rq_rope_tensor* q, const rq_rope_tensor* k, const int32_t* start,
                  const int32_t* offsets, void* stream);

/* Static description of a status code (never NULL). */
const char* rq_status_string(rq_status status);

#ifdef __cplusplus
}
#endif
#endif /* RQ_H_ */
