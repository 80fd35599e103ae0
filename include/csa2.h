/*
 * csa2.h -- C ABI of libcsa2.so: CSA2 sparse decode attention on one GB300.
 *
 * The method (DeepSeek V4.1 Flash, as described on the architecture page
 * k-a.in "DeepSeek V4.1 Flash"):
 *   - section "CSA2 with cross-layer reuse", mode table: a Full layer computes
 *     its own main KV / indexer keys and a fresh Top-K; a Reindex layer reuses
 *     them but runs its own indexer query and a fresh Top-K; a Reuse layer
 *     reuses KV, indexer keys and the Top-K indices.  Every mode computes its
 *     own main query and SWA KV.
 *   - bullet "Sparse attention": each query reads its Top-512 main-KV entries
 *     plus a 128-token sliding window (SWA).
 *   - bullet "Hierarchical indexer": later decoder indexers score at most
 *     16,384 candidates whatever the context length (blocks of 8 entries, a
 *     pool of at most 2,048 blocks); page "DeepSeek V4.1 Flash made encoders
 *     cool" (artofsm.art): the hierarchical sparse indexer narrows candidates
 *     to blocks.
 * The pages do not give the indexer formula (they point to "section 4.2.1" of
 * a report that is not among them).  This library computes, for a query with
 * indexer heads q_h and weights w_h, the score of a key k as
 *     s(k) = sum_h w_h * ReLU(q_h . k)          (ReLU optional, see relu)
 * and selects Top-K under the total order (score descending, index ascending).
 *
 * Conventions shared by every entry point
 *   - Every pointer argument is DEVICE memory owned by the caller, row-major
 *     and contiguous, unless stated otherwise.  Arrays read by bulk copies
 *     (keys, main KV, SWA KV, queries) must be 16-byte aligned.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *     stream).  No entry point allocates or frees memory, and none
 *     synchronises except csa2_read_device_error and
 *     csa2_read_static_device_error.
 *   - Arguments are validated on the host before anything is enqueued; a
 *     negative csa2_status is returned and nothing is launched.  A failed
 *     launch returns CSA2_ERR_CUDA.
 *   - Conditions only the device can see (an index outside the cache, a count
 *     outside its range, a pooled block id outside the valid blocks) are
 *     clamped or skipped by the kernels and recorded in a sticky error word in
 *     the workspace header; kernels never trap.  Read it with
 *     csa2_read_device_error.
 *   - Kernels are launched with programmatic dependent launch.  Some read
 *     the call's own inputs (q, SWA rows, n_swa, k_swa, v_swa) before waiting
 *     for the preceding kernel of the stream, which is safe under ordinary
 *     stream order.  If the kernel enqueued just before a call lets its
 *     dependents start early (griddepcontrol.launch_dependents), it must not
 *     write those inputs after doing so.  The library's own kernels never
 *     write them; csa2_kv_append and csa2_swa_append, which do, never start
 *     their dependents early.
 *   - `ws` is a caller-owned device workspace of at least
 *     csa2_workspace_bytes(shape) bytes, 256-byte aligned, zeroed once with
 *     csa2_workspace_init before first use.  Calls that share a workspace
 *     must be ordered on one stream.  The cache-maintenance calls
 *     (csa2_block_keys, csa2_kv_append, csa2_swa_append) use only the
 *     workspace's error word; they also accept ws = NULL with ws_bytes = 0,
 *     and then record device errors in the header of the library's static
 *     scratch array (see csa2_layer_group_static), where
 *     csa2_read_static_device_error reads them.
 *   - Element type (csa2_shape.dtype): bf16 or fp32, for queries, keys,
 *     values and indexer tensors alike.  Scores, weights, outputs and lse are
 *     fp32; indices and counts are int32.
 */
#ifndef CSA2_H_
#define CSA2_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* csa2_stream_t; /* identical to cudaStream_t */

typedef enum {
  CSA2_OK = 0,
  CSA2_ERR_INVALID_ARG = -1,  /* null pointer, bad size, misaligned pointer, illegal mode sequence */
  CSA2_ERR_UNSUPPORTED = -2,  /* valid but not implemented (e.g. dims beyond the generic limits) */
  CSA2_ERR_WORKSPACE = -3,    /* ws too small or misaligned */
  CSA2_ERR_CUDA = -4,         /* a CUDA launch or runtime call failed */
  CSA2_ERR_DEVICE_CHECK = -5, /* returned by csa2_read_device_error: a kernel recorded a bad input */
  CSA2_ERR_TIMEOUT = -6       /* returned by csa2_read_device_error: a bounded device wait gave up */
} csa2_status;

/* CSA2_SWA: a pure sliding-window layer (the first two encoder layers of the
 * architecture figure caption): it attends only its own SWA rows and neither
 * needs nor produces indices. */
typedef enum { CSA2_FULL = 0, CSA2_REINDEX = 1, CSA2_REUSE = 2, CSA2_SWA = 3 } csa2_mode;
typedef enum { CSA2_BF16 = 0, CSA2_F32 = 1 } csa2_dtype;

/* Problem shape shared by a layer group.  Symbols: B batch (one decode query
 * per sequence), N compressed main-KV entries per sequence (cache capacity),
 * HI x dI indexer heads x dim, P pool blocks, K Top-K, H query heads sharing
 * one KV head with key dim dk and value dim dv, W SWA rows. */
typedef struct {
  int32_t batch;       /* B >= 1 */
  int32_t n_entries;   /* N >= 1; a multiple of `block` when a hierarchical stage is used */
  int32_t idx_heads;   /* HI, 1..64 */
  int32_t idx_dim;     /* dI, 1..1024 */
  int32_t block;       /* entries per block, >= 1 (8 in the architecture) */
  int32_t pool_blocks; /* P: blocks kept by the hierarchical stage; 0 = no hierarchical stage */
  int32_t topk;        /* K, 1..1024 (512 in the architecture) */
  int32_t q_heads;     /* H, 1..1024 */
  int32_t k_dim;       /* dk, 1..1024 */
  int32_t v_dim;       /* dv, 1..1024 */
  int32_t swa;         /* W, 0..1024 (128 in the architecture); K + W <= 1024 */
  float scale;         /* softmax scale; <= 0 selects 1/sqrt(dk) */
  int32_t relu;        /* 1: ReLU on each indexer head's dot product (default reading); 0: none */
  int32_t dtype;       /* csa2_dtype */
  int32_t tokens;      /* T: query tokens per sequence (0 or 1: one).  With T > 1 (architecture
                          page, "Asymmetric encoder-decoder": prompt tokens run a 128-token decoder
                          replay), B is a multiple of T and queries b = s*T .. s*T + T-1 share the
                          caches of sequence s: k_main, v_main and k_idx are then [B / T, N, ...].
                          Everything else stays per query, including n_valid (each token's own
                          causal count), the SWA rows and kb (block summary keys of the query's own
                          valid prefix, so a token's partial last block averages only entries it
                          may see).  csa2_kv_append and csa2_swa_append take T <= 1. */
} csa2_shape;

/* One layer of a group (csa2_layer_group). */
typedef struct {
  int32_t mode;        /* csa2_mode */
  int32_t hier;        /* 1: hierarchical (block pool) indexing; needs kb and pool_blocks > 0 */
  const void* q;       /* [B, H, dk] the layer's own query */
  const void* q_idx;   /* [B, HI, dI] indexer query (Full / Reindex; ignored for Reuse and SWA) */
  const float* w_idx;  /* [B, HI] indexer head weights (Full / Reindex; ignored for Reuse and SWA) */
  const void* k_swa;   /* [B, W, dk] the layer's own SWA keys: rows 0..n_swa-1 in any order
                          (oldest first, or the ring csa2_swa_append keeps) */
  const void* v_swa;   /* [B, W, dv] the layer's own SWA values */
  float* out;          /* [B, H, dv] attention output */
  float* lse;          /* [B, H] natural-log sum of exp of the scaled logits, or NULL */
  int32_t* idx_out;    /* [B, K] fresh indices of an indexing layer, or NULL; untouched for Reuse / SWA */
} csa2_layer;

/* Workspace bytes needed by any entry point for this shape (host only). */
size_t csa2_workspace_bytes(const csa2_shape* shape);

/* Zero the workspace header (device error word).  Call once before first use. */
int csa2_workspace_init(void* ws, size_t ws_bytes, csa2_stream_t stream);

/* Block summary keys (cache-side maintenance, architecture page bullet
 * "Hierarchical indexer"; the 128K Reindex workload defines the summary as
 * the mean of the block's 8 keys rounded to integers).
 * kb[b, j, :] = mean of k_idx[b, j*block + t, :] over the valid entries
 * t < block with j*block + t < n_valid[b] (a partial last block averages its
 * valid entries), rounded half-to-even to an integer if round_to_int, then
 * stored in the element type.  Blocks j >= ceil(n_valid[b] / block) are
 * written as 0.
 *   k_idx   [B, N, dI]     n_valid [B] (0..N)
 *   kb      [B, ceil(N / block), dI]  (output) */
int csa2_block_keys(const csa2_shape* shape, const void* k_idx, const int32_t* n_valid,
                    int32_t round_to_int, void* kb, void* ws, size_t ws_bytes, csa2_stream_t stream);

/* Decode-step cache maintenance, main caches (architecture page: the
 * compressed main KV grows by one entry per compressed span of tokens, and
 * bullet "Hierarchical indexer" keeps one summary key per block of 8 entries;
 * producing the compressed entries themselves is a learned operator the pages
 * do not describe, so they are inputs here).
 * For each query b, the first n_new[b] rows (0..max_new) of k_new[b],
 * v_new[b] and kidx_new[b] are written at entry positions n_valid[b],
 * n_valid[b] + 1, ... of k_main, v_main and k_idx; then, when kb is not NULL,
 * the summary key of every block those positions fall in is recomputed over
 * the block's valid entries exactly as csa2_block_keys computes it (other
 * blocks are left as they are); finally n_valid[b] grows by n_new[b].
 * Entries that would land at N or beyond are dropped and recorded in the
 * device error word (bad count).
 *   k_new [B, max_new, dk]  v_new [B, max_new, dv]  kidx_new [B, max_new, dI]  n_new [B]
 *   k_main [B, N, dk]  v_main [B, N, dv]  k_idx [B, N, dI]  kb [B, ceil(N / block), dI] or NULL
 *   n_valid [B] (read and updated)
 * The caches, kb and n_valid are updated in place; ws holds only the error word. */
int csa2_kv_append(const csa2_shape* shape, int32_t max_new, const int32_t* n_new, const void* k_new,
                   const void* v_new, const void* kidx_new, void* k_main, void* v_main, void* k_idx, void* kb,
                   int32_t* n_valid, int32_t round_to_int, void* ws, size_t ws_bytes, csa2_stream_t stream);

/* One layer's part of csa2_swa_append. */
typedef struct {
  const void* k_tok;   /* [B, dk] the layer's key of the new token */
  const void* v_tok;   /* [B, dv] the layer's value of the new token */
  void* k_swa;         /* [B, W, dk] the layer's SWA ring (updated in place) */
  void* v_swa;         /* [B, W, dv] */
} csa2_swa_slot;

/* Decode-step cache maintenance, SWA windows (architecture page, bullet
 * "Sparse attention": every query also attends its last W tokens
 * uncompressed; mode table: every layer has its own SWA KV).
 * The layers of a group keep their windows as rings that share one head and
 * one fill count per query: for every layer l and query b, row swa_head[b] of
 * layers[l].k_swa[b] / v_swa[b] takes layers[l].k_tok[b] / v_tok[b]; then
 * swa_head[b] advances by one modulo W and n_swa[b] grows by one up to W.
 * Attention uses rows 0..n_swa[b]-1 as a set, so a ring needs no reordering.
 * A swa_head or n_swa outside 0..W-1 / 0..W is clamped and recorded in the
 * device error word (bad count).  1 <= n_layers <= 64; shape.swa >= 1.
 *   swa_head [B], n_swa [B] (read and updated) */
int csa2_swa_append(const csa2_shape* shape, const csa2_swa_slot* layers, int32_t n_layers, int32_t* swa_head,
                    int32_t* n_swa, void* ws, size_t ws_bytes, csa2_stream_t stream);

/* Hierarchical first stage: score every valid block summary key with the
 * indexer formula and keep the top min(P, NB_b) blocks, NB_b = ceil(n_valid[b] / block),
 * under (block score descending, block id ascending).
 *   q_idx [B, HI, dI]   w [B, HI]   kb [B, ceil(N / block), dI]   n_valid [B]
 *   pool_out   [B, P]  (output) pooled block ids in ascending order, padded with -1
 *   n_pool_out [B]     (output) min(P, NB_b) */
int csa2_index_blocks(const csa2_shape* shape, const void* q_idx, const float* w, const void* kb,
                      const int32_t* n_valid, int32_t* pool_out, int32_t* n_pool_out, void* ws,
                      size_t ws_bytes, csa2_stream_t stream);

/* Token-level indexer scores.
 * Flat (pool == NULL): scores_out[b, j] = s(k_idx[b, j]) for j < n_valid[b];
 *   cand_out (nullable) receives j; n_cand_out (nullable) receives n_valid[b].
 *   scores_out / cand_out have row stride N.
 * Pooled (pool != NULL, from csa2_index_blocks): the candidates are the
 *   entries of the pooled blocks in pool order (ascending entry id);
 *   position p*block + t holds entry pool[b, p]*block + t, its score, or
 *   cand -1 / score -inf when that entry is >= n_valid[b].
 *   scores_out / cand_out have row stride P*block; n_cand_out[b] = n_pool[b]*block.
 *   cand_out and n_cand_out are required. */
int csa2_index_tokens(const csa2_shape* shape, const void* q_idx, const float* w, const void* k_idx,
                      const int32_t* n_valid, const int32_t* pool, const int32_t* n_pool,
                      float* scores_out, int32_t* cand_out, int32_t* n_cand_out, void* ws,
                      size_t ws_bytes, csa2_stream_t stream);

/* Token scoring and exact Top-k in one call: the candidates of
 * csa2_index_tokens (flat when pool == NULL, else the pooled blocks' entries)
 * are scored and the top k (1 <= k <= shape.topk) selected under (score
 * descending, entry index ascending), as csa2_index_tokens followed by
 * csa2_topk would -- bullet "Sparse attention" (Top-512) and bullet
 * "Hierarchical indexer" (at most 16,384 pooled candidates).  On the fast
 * path (bf16, 8 x 64 indexer, blocks of 8) one thread-block cluster per query
 * scores its candidates and selects in shared memory without writing scores
 * to HBM.
 *   q_idx [B, HI, dI]  w [B, HI]  k_idx [B, N, dI]  n_valid [B]
 *   pool [B, P], n_pool [B] (from csa2_index_blocks) or NULL
 *   idx_out [B, k] (output) selected entry ids ascending, padded with -1
 *   n_out   [B]    (output, nullable) number selected */
int csa2_index_topk(const csa2_shape* shape, const void* q_idx, const float* w, const void* k_idx,
                    const int32_t* n_valid, const int32_t* pool, const int32_t* n_pool, int32_t k,
                    int32_t* idx_out, int32_t* n_out, void* ws, size_t ws_bytes, csa2_stream_t stream);

/* Exact Top-k of each row: scores [B, ld] (row stride ld), optional candidate
 * ids cand [B, ld] (NULL: the id is the position; ids < 0 are skipped; ids
 * must ascend with position), n_cand [B] positions to consider (NULL: ld).
 * Order: score descending, id ascending; -0 equals +0 and NaN ranks as -inf.
 *   idx_out   [B, k] (output) selected ids in ascending order, padded with -1
 *   score_out [B, k] (output, nullable) their scores (-inf for padding)
 * 1 <= k <= 16384, ld <= 2^28. */
int csa2_topk(const csa2_shape* shape, const float* scores, int32_t ld, const int32_t* cand,
              const int32_t* n_cand, int32_t k, int32_t* idx_out, float* score_out, void* ws,
              size_t ws_bytes, csa2_stream_t stream);

/* Sparse attention of one decode query per sequence (all H heads share one
 * KV head): one softmax over the main-KV rows idx[b, :] (entries < 0 are
 * skipped) and the SWA rows 0..n_swa[b]-1.
 *   q [B, H, dk]  k_main [B, N, dk]  v_main [B, N, dv]  idx [B, K]
 *   k_swa [B, W, dk]  v_swa [B, W, dv]  n_swa [B] (0..W)
 *   out [B, H, dv] (output)  lse [B, H] (output, nullable; -inf and out = 0
 *   when a query attends no row at all). */
int csa2_sparse_attn(const csa2_shape* shape, const void* q, const void* k_main, const void* v_main,
                     const int32_t* idx, const void* k_swa, const void* v_swa, const int32_t* n_swa,
                     float* out, float* lse, void* ws, size_t ws_bytes, csa2_stream_t stream);

/* A whole layer group over one shared main KV and indexer-key cache (the
 * group's Full layer's): layers run in order; Full and Reindex compute fresh
 * indices (flat, or hierarchical when layer.hier), Reuse attends with the
 * latest indices; every layer attends with its own q and SWA KV; an SWA
 * layer attends its SWA rows only.
 * Rules: a Reuse layer needs an earlier Full or Reindex layer in the group;
 * hier needs kb (from csa2_block_keys) and pool_blocks > 0.
 *   k_main [B, N, dk]  v_main [B, N, dv]  k_idx [B, N, dI]
 *   kb [B, ceil(N / block), dI] (nullable when no layer is hierarchical)
 *   n_valid [B] (0..N)  n_swa [B] (0..W) */
int csa2_layer_group(const csa2_shape* shape, const csa2_layer* layers, int32_t n_layers,
                     const void* k_main, const void* v_main, const void* k_idx, const void* kb,
                     const int32_t* n_valid, const int32_t* n_swa, void* ws, size_t ws_bytes,
                     csa2_stream_t stream);

/* csa2_layer_group for callers that cannot allocate device memory -- the
 * paper has no counterpart; this is a convenience of this library.  Some
 * callers have no way to provide a workspace: a plugin inside a host framework
 * that owns all device memory and exposes no allocator, or a latency-critical
 * decode loop that must not call cudaMalloc (it can synchronise the device).
 * This entry point takes the same arguments as csa2_layer_group minus the
 * workspace, and runs the same layer group on a 32 MiB scratch array that the
 * library holds in device memory (a file-scope __device__ array: every GPU
 * that loads the library keeps it until the process exits; it starts zeroed).
 *   - Shapes whose layer groups need more than 32 MiB of workspace return
 *     CSA2_ERR_WORKSPACE and enqueue nothing.
 *   - The first call made while a device is current looks up the array's
 *     device address (once per device, safe against host threads making
 *     their first calls at the same time); make that first call before any
 *     stream capture.
 *   - Every call shares the one array: calls that may overlap on the GPU (on
 *     different streams, or from different host threads without ordering)
 *     race on it and must be serialised by the caller.
 *   - No memory is allocated or freed.  Device-side range problems are
 *     skipped by the kernels as in csa2_layer_group and recorded in the
 *     array's header; read them with csa2_read_static_device_error.
 *   - kb can be prepared without a workspace too: csa2_block_keys and
 *     csa2_kv_append accept ws = NULL, ws_bytes = 0. */
int csa2_layer_group_static(const csa2_shape* shape, const csa2_layer* layers, int32_t n_layers,
                            const void* k_main, const void* v_main, const void* k_idx, const void* kb,
                            const int32_t* n_valid, const int32_t* n_swa, csa2_stream_t stream);

/* csa2_read_device_error for the static scratch array of the current device
 * (the error word of csa2_layer_group_static and of cache-maintenance calls
 * made with ws = NULL): synchronises `stream`, returns and clears the word.
 * The paper has no counterpart. */
int csa2_read_static_device_error(csa2_stream_t stream, int32_t* detail);

/* ---------------------------------------------------------------- context parallelism
 * One long sequence per query split over G ranks by block-aligned entry
 * ranges: rank g holds entries [e0_g, e0_g + n_loc_g) of every sequence.  The
 * pages describe no multi-GPU scheme; the split keeps the method's results
 * because its selection order (score descending, id ascending) is a strict
 * total order -- the Top-k of a union is the Top-k of the union of the parts'
 * Top-k lists -- and softmax partials over disjoint key sets combine exactly by
 * their log-sum-exp.  It serves contexts beyond one GPU, which the
 * architecture page's bullet "Hierarchical indexer" (at most 16,384
 * candidates whatever the context length) makes cheap to select over.  The
 * ranks exchange (score, id) lists and (out, lse) partials with their own
 * collectives; these calls are the per-rank steps around the exchanges. */

/* Keep the ids of each row that fall in [lo, hi), in their order, add delta,
 * and write them compacted to out[b, 0 .. n) with -1 after (n_out[b] = n).
 * Used both ways: a rank's local ids to global (lo = 0, hi = n_loc,
 * delta = e0) and a global list to a rank's local ids (lo = e0,
 * hi = e0 + n_loc, delta = -e0).  ids < 0 are dropped.  When a row keeps more
 * than ld_out ids the rest are dropped and the device error word records a
 * bad count.
 *   ids [batch, ld]   out [batch, ld_out]   n_out [batch] (nullable)
 *   ws: only its 256-byte header (error word) is used. */
int csa2_shard_slice(const int32_t* ids, int32_t batch, int32_t ld, int32_t lo, int32_t hi, int32_t delta,
                     int32_t* out, int32_t ld_out, int32_t* n_out, void* ws, size_t ws_bytes, csa2_stream_t stream);

/* A rank's valid entries (div = 1) or valid blocks (div = block) per query:
 * out[b] = ceil(clamp(n_valid[b] - e0, 0, n_loc) / div).
 *   n_valid [batch] (global counts)   out [batch] */
int csa2_shard_counts(const int32_t* n_valid, int32_t batch, int32_t e0, int32_t n_loc, int32_t div, int32_t* out,
                      csa2_stream_t stream);

/* The G parts' (id, score) lists of every row side by side, in part order:
 * ids_out[b, g*k + p] = ids[g, b, p] and likewise for the scores (nullable),
 * turning the [parts, batch, k] result of an all-gather into the [batch,
 * parts*k] candidate rows of csa2_topk. */
int csa2_concat_parts(int32_t parts, int32_t batch, int32_t k, const int32_t* ids, const float* scores,
                      int32_t* ids_out, float* scores_out, csa2_stream_t stream);

/* Combine the softmax attention of `parts` disjoint key sets, in part order:
 * with M = max_g lse_g and w_g = exp(lse_g - M),
 *   out = sum_g w_g out_g / sum_g w_g,   lse = M + log(sum_g w_g);
 * parts with lse = -inf (no key) contribute nothing; all -inf gives out = 0
 * and lse = -inf.  Rows are (query, head) pairs.
 *   out_parts [parts, rows, v_dim]  lse_parts [parts, rows] (natural log)
 *   out [rows, v_dim]  lse [rows] (nullable) */
int csa2_merge_attn(int32_t parts, int32_t rows, int32_t v_dim, const float* out_parts, const float* lse_parts,
                    float* out, float* lse, csa2_stream_t stream);

/* ---------------------------------------------------------------- drafted tokens and bounded caches
 * A decode step that verifies several drafted tokens per sequence at once, and
 * caches that are held at a fixed size.  In the order of a step: csa2_rope
 * turns the drafted queries and keys to their positions, csa2_index_topk
 * (shape.tokens = T) selects each drafted token's entries, csa2_tree_attn
 * attends them along the tree; once the caller has chosen the accepted path,
 * csa2_attn_weights gives the accepted queries' attention weights,
 * csa2_tree_commit pushes the path into the windows and adds the weights up,
 * and csa2_kv_evict shrinks the caches that have filled.  The pages describe
 * neither drafting nor eviction; these calls keep the method's own definitions
 * (bullet "Sparse attention": selected entries plus the last W tokens) and
 * bookkeeping.  Their kernels read nothing before the preceding kernel of the
 * stream has completed.  No array of theirs may lie in the ws_bytes of the call's
 * ws, and each begins at a multiple of its elements' size (refused). */

/* Frequencies of rotary positions, in radians per position, for rot_dim / 2
 * pairs (host only; the caller copies them to the device once).  With
 * f_i = base^(-2i / rot_dim):
 *   CSA2_ROPE_PLAIN   f_i
 *   CSA2_ROPE_LINEAR  f_i / factor
 *   CSA2_ROPE_NTK     as PLAIN with base * factor^(rot_dim / (rot_dim - 2)), rot_dim > 2; refused where that is not finite
 *   CSA2_ROPE_YARN    pairs that turn more than beta_fast times over orig_ctx positions keep f_i, pairs that turn less than
 *                     beta_slow times get f_i / factor, a linear ramp over the pairs between them; the magnitude is
 *                     0.1 ln(factor) + 1
 * *mag (nullable) receives the magnitude (1 but for YARN).  rot_dim even,
 * 2..1024; base > 1; factor >= 1; YARN: orig_ctx >= 1, beta_fast > beta_slow > 0. */
typedef enum { CSA2_ROPE_PLAIN = 0, CSA2_ROPE_LINEAR = 1, CSA2_ROPE_NTK = 2, CSA2_ROPE_YARN = 3 } csa2_rope_scaling;
int csa2_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor, int32_t orig_ctx, double beta_fast,
                    double beta_slow, double* freqs, float* mag);

/* One tensor of csa2_rope: x and out [rows, heads, dim] in dtype (csa2_dtype).
 * Dims rot_off .. rot_off + rot_dim - 1 of every head are turned, the others
 * copied.  out == x works in place (only the turned dims are touched); any
 * other overlap is refused. */
typedef struct {
  const void* x;
  void* out;
  int32_t heads, dim, rot_off, dtype;
} csa2_rope_slot;

/* Rotary positions, partial and in either layout, for several tensors of the
 * same rows (queries, keys, indexer queries, ...) in one launch:
 * the pair (a, b) of row r, pair i becomes
 *   mag * (a cos t - b sin t, b cos t + a sin t),  t = pos[r] * freqs[i];
 * inverse = 1 turns back: the angle is -t and the magnitude 1 / mag.
 * Pairs are dims (i, i + rot_dim / 2) of the turned range, or (2i, 2i + 1)
 * when interleaved = 1.  The angle is reduced in fixed-point turns, off by at
 * most |t| 2^-52 + |pos| 2 pi 2^-65 + 2 pi 2^-26 for any int32 position; the
 * arithmetic is fp32, rounded once.
 *   pos [rows] int32   freqs [rot_dim / 2] double (device)
 * rows >= 1; 1 <= n_slots <= 16; mag finite and > 0. */
int csa2_rope(const csa2_rope_slot* slots, int32_t n_slots, int32_t rows, int32_t rot_dim, int32_t interleaved,
              const int32_t* pos, const double* freqs, float mag, int32_t inverse, csa2_stream_t stream);

/* Sparse attention of a tree of drafted tokens (shape.tokens = T <= 128,
 * B = S * T queries, query b = s*T + t is drafted token t of sequence s).
 * One softmax per query and head over
 *   - the main-KV rows idx[b, :] (entries < 0 are skipped, as in csa2_sparse_attn);
 *   - token t itself and its ancestors in the tree, rows of k_draft / v_draft;
 *   - the sequence's committed window rows,
 * the last two limited to the W = shape.swa tokens that end at token t along
 * its path: a token of depth d (0 for a root) sees the nearest min(d + 1, W)
 * drafted tokens of its path and the newest W - (d + 1) committed ones.
 * parent[s, t] is the token's parent, an earlier token (0 <= parent < t), or
 * -1 for a root; anything else is recorded (bad index) and taken as -1.
 * parent == NULL is a chain (parent = t - 1).  Tokens t >= n_draft[s] are not
 * live: out = 0, lse = -inf (n_draft == NULL: all T are).  A live token must
 * not have a parent that is not live; parent < t ensures that.
 * The window is what csa2_swa_append and csa2_tree_commit keep: a full ring
 * (n_swa[s] == W) has its oldest row at swa_head[s] (swa_head == NULL: row 0),
 * one that is not full holds its rows oldest first from row 0.
 *   q [B, H, dk]  k_main [S, N, dk]  v_main [S, N, dv]  idx [B, K]
 *   k_swa [S, W, dk]  v_swa [S, W, dv]  swa_head, n_swa [S]
 *   k_draft [S, T, dk]  v_draft [S, T, dv]  parent [S, T]  n_draft [S] (0..T)
 *   out [B, H, dv] in the element type (it feeds the output projection)
 *   lse [B, H] fp32 (nullable); NaN where a key that is attended scores NaN or +inf, as out is
 * shape.swa >= 1; batch <= 65,535; out and lse overlap nothing else (refused).
 * A chain of T gives what T steps of csa2_swa_append and csa2_sparse_attn
 * give.  Weights are rounded to bf16 (half a step, 2^-8 of a weight) before they
 * meet bf16 values on tensor cores, as csa2_sparse_attn rounds them; bf16 rows that
 * are not whole 8-byte pieces are multiplied in fp32.  The weights' sums and lse are never rounded.
 * csa2_merge_attn takes fp32 parts, so that out cannot be one of them.  ws also holds lists of the sequences' keys, where the indexing calls
 * keep scores, lists and the group's indices (caches much shorter than topk need
 * the most for them). */
int csa2_tree_attn(const csa2_shape* shape, const void* q, const void* k_main, const void* v_main, const int32_t* idx,
                   const void* k_swa, const void* v_swa, const int32_t* swa_head, const int32_t* n_swa,
                   const void* k_draft, const void* v_draft, const int32_t* parent, const int32_t* n_draft, void* out,
                   float* lse, void* ws, size_t ws_bytes, csa2_stream_t stream);

/* The attention weight of every selected entry, summed over the heads:
 *   weights[b, j] = sum_h exp(scale * q[b, h] . k_main[idx[b, j]] - lse[b, h])
 * with the lse of csa2_tree_attn, csa2_sparse_attn or a layer of
 * csa2_layer_group; 0 where idx[b, j] < 0, and heads with lse = -inf add
 * nothing.  live[b] = 0 leaves the query out: its weights are written as 0
 * and nothing of it is read (NULL: all are wanted).
 *   q [B, H, dk]  k_main [B / T, N, dk]  idx [B, K]  lse [B, H]  live [B]
 *   weights [B, K] fp32 (overlaps nothing else: refused)
 * batch <= 65,535. */
int csa2_attn_weights(const csa2_shape* shape, const void* q, const void* k_main, const int32_t* idx, const float* lse,
                      const int32_t* live, float* weights, void* ws, size_t ws_bytes, csa2_stream_t stream);

/* One layer's part of csa2_tree_commit (B = S * T as in csa2_tree_attn). */
typedef struct {
  const void* k_draft;    /* [S, T, dk] */
  const void* v_draft;    /* [S, T, dv] */
  void* k_swa;            /* [S, W, dk] the layer's window (updated in place) */
  void* v_swa;            /* [S, W, dv] */
  const int32_t* idx;     /* [B, K] the layer's selected entries, or NULL */
  const float* weights;   /* [B, K] their weights (csa2_attn_weights), or NULL: the layer adds nothing */
} csa2_tree_slot;

/* Commit the accepted path of every sequence: path[s, 0 .. n_path[s]) are its
 * drafted tokens, root first (n_path[s] in 0..T; the rest of path is not
 * read).  Every layer's rows k_draft / v_draft of these tokens go into its
 * window ring at swa_head[s], swa_head[s] + 1, ... modulo W, as as many
 * csa2_swa_append calls would put them (one head and one fill count per
 * sequence, shared by the layers); then swa_head and n_swa are advanced.
 * mass (nullable) accumulates attention weights per cache entry, for
 * csa2_kv_evict: for every accepted token b = s*T + path[s, i] and layer with
 * weights,
 *   mass[s, idx[b, j]] += rint(weights[b, j] * 2^32)
 * in integers, so that the sums depend on no order and lose nothing over long
 * runs.  A mass stops at 2^63 - 1, a weight of 2^31 in all, and does not wrap
 * (64 heads of 20 layers that give one entry all their weight reach it in 1.7
 * million tokens); entries that stand there tie in csa2_kv_evict, so a caller
 * whose runs are longer scales its masses down in time.  Entries with idx < 0 add nothing; a weight that is not in
 * [0, 2^20] is recorded (bad weight, bit 4 of the error word) and adds
 * nothing, an idx >= N is recorded and skipped.  A path id outside 0..T-1 is
 * recorded (bad index) and ends the path before it.
 *   path [S, T]  n_path [S]  swa_head [S], n_swa [S] (read and updated)
 *   mass [S, N] int64 (read and updated)
 * 1 <= n_layers <= 64; shape.swa >= 1; shape.tokens = T <= 128; S <= 65,535.
 * ws holds only the error word (NULL with ws_bytes = 0: the static scratch's,
 * as for csa2_swa_append).  Windows, heads and mass overlap neither each other
 * nor anything else of the call (refused). */
int csa2_tree_commit(const csa2_shape* shape, const csa2_tree_slot* layers, int32_t n_layers, const int32_t* path,
                     const int32_t* n_path, int32_t* swa_head, int32_t* n_swa, int64_t* mass, void* ws, size_t ws_bytes,
                     csa2_stream_t stream);

/* Evict from every sequence that holds more than `trigger` entries, down to
 * `keep`: the first `sink` and the last `recent` entries stay, and of the
 * others the keep - sink - recent with the greatest mass (ties: the lowest
 * index).  What stays moves together in its order; sequences at or below the
 * trigger keep all.  0 <= sink, recent; 1 <= keep <= trigger <= N;
 * sink + recent <= keep; shape.tokens <= 1.
 *   k_main [S, N, dk]  v_main [S, N, dv]  k_idx [S, N, dI]  mass [S, N] int64  n_valid [S]
 *   k_main_out, v_main_out, k_idx_out, mass_out, n_valid_out: the same shapes
 *   kept [S, N] int32 (output): the entry that each row held before, -1 behind the last
 *   kb_out [S, ceil(N / block), dI] (nullable): block keys of the result, as csa2_block_keys gives them
 * Rows behind the last entry stay as they were, but for mass_out, which is 0
 * there.  Either every _out is its input (in place: a sequence that is not
 * evicted from is not written, its row of kept apart), or the
 * outputs overlap no input (then every sequence is copied).  kept and kb_out
 * overlap nothing.  ws as for csa2_tree_commit; batch <= 65,535. */
int csa2_kv_evict(const csa2_shape* shape, int32_t trigger, int32_t keep, int32_t sink, int32_t recent,
                  const void* k_main, const void* v_main, const void* k_idx, const int64_t* mass, const int32_t* n_valid,
                  void* k_main_out, void* v_main_out, void* k_idx_out, int64_t* mass_out, int32_t* n_valid_out,
                  int32_t* kept, void* kb_out, int32_t round_to_int, void* ws, size_t ws_bytes, csa2_stream_t stream);

/* Static description of a status code. */
const char* csa2_status_str(int status);

/* Synchronise `stream`, read and clear the sticky device error word of `ws`.
 * Returns CSA2_OK, CSA2_ERR_DEVICE_CHECK or CSA2_ERR_TIMEOUT (a bounded wait
 * gave up); *detail (nullable) receives the error bits (bit 0 bad index,
 * bit 1 bad count, bit 2 timeout, bit 3 bad pooled block, bit 4 bad weight) in
 * its low byte. */
int csa2_read_device_error(void* ws, csa2_stream_t stream, int32_t* detail);

/* 1 when the fast (tensor-core) kernels serve this shape, 0 when the generic
 * kernels do (host only; for diagnostics and tests). */
int csa2_fast_path(const csa2_shape* shape, int32_t* indexer_fast, int32_t* attention_fast);

/* Number of kernel launches this library has enqueued since it was loaded
 * (all threads and devices; launches recorded into a CUDA graph count once,
 * at capture).  For diagnostics and launch accounting. */
unsigned long long csa2_launch_count(void);

/* Test hook of the device-side failure detection (diagnostics; the paper has
 * no counterpart).  Runs the fused flat scoring + Top-k of csa2_index_topk
 * (pool == NULL; fast path only, else CSA2_ERR_UNSUPPORTED) with the copy of
 * every CTA's first key tile left out, so that the tile's stage barrier can
 * never complete, and with every bounded wait limited to wait_limit_ns
 * (1,000 .. 100,000,000) instead of 2 s.  The waits give up, the kernel
 * records CSA2_ERR_TIMEOUT (bit 2) in the workspace's error word, the CTAs
 * that gave up offer no candidate, and the kernel returns: no copy is in
 * flight when a wait gives up and every write stays inside idx_out [B, k].
 * csa2_read_device_error then returns CSA2_ERR_TIMEOUT, and the stream and
 * context stay usable. */
int csa2_debug_wait_timeout(const csa2_shape* shape, const void* q_idx, const float* w, const void* k_idx,
                            const int32_t* n_valid, int32_t k, int32_t* idx_out, uint32_t wait_limit_ns,
                            void* ws, size_t ws_bytes, csa2_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CSA2_H_ */
