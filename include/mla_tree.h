/*
 * mla_tree.h - C ABI of a speculative decode step over trees of drafted
 * tokens: ragged queries, ragged cache append, tree attention, and the move
 * of the accepted path's cache rows.
 *
 * The multi-token decode of "Huawei Ascend servers: DeepSeek V3/R1 inference
 * best practice" (sections 5.3 and 7.1: one speculative token per step) is a
 * chain of s_q = 2 tokens, which mla_decode covers.  A draft that branches is
 * a tree: request b brings n_b <= 64 nodes, which stand in its cache at slots
 * L_b - n_b .. L_b - 1 (L_b = seq_lens[b], the nodes included) in the order of
 * the token arrays.  The slots before them are its context.  Node i sees the
 * whole context and those nodes j < n_b whose bit j is set in its mask (its
 * ancestors and itself, for a tree; any mask is accepted):
 *
 *   q_latent[t][h] = q_nope[t][h] . W_UK[h],  q_rope[t][h] = RoPE(q_pe[t][h], pos_t)   (mla_query)
 *   cache row of slot L_b - n_b + i = RMSNorm(kv_latent[t]) || RoPE(k_pe[t], pos_t)    (mla_cache_append)
 *   s_j  = scale * (q_latent . r_j[0:512] + q_rope . r_j[512:576])                     (mla_tree_decode)
 *   o    = sum_j softmax(s)_j r_j[0:512],  lse = ln sum_j exp(s_j),  j over the visible keys
 *   row of slot L_b - n_b + i <- row of slot L_b - n_b + path_b[i]                     (mla_cache_commit)
 *
 * with t = token_offsets[b] + i.  A node that sees no key at all (an empty
 * context and an empty mask) gives o = 0 and lse = -infinity.  Masked rows may
 * hold anything, NaN and infinities included.
 *
 * Ragged token arrays: the tokens of all requests one after another,
 * request b's being token_offsets[b] .. token_offsets[b + 1] - 1, with
 * token_offsets[0] = 0, non-decreasing, token_offsets[batch] <= tokens.  Rows
 * at or past token_offsets[batch] are neither read nor written (arrays padded
 * to a fixed size, e.g. for a captured graph); a request without tokens is
 * left out whatever its seq_len.
 *
 * Conventions as in mla_decode.h: device pointers, caller-owned buffers, work
 * enqueued on `stream`, nothing synchronises and nothing is allocated; host
 * argument errors return a status and enqueue nothing.  Arrays are dense and
 * row-major unless strides are given; base pointers 16-byte aligned except the
 * int32 and int64 arrays' (natural alignment).
 *
 * Errors found on the device are OR-ed into a status word (MLA_DEV_* bits of
 * mla_decode.h and the two below): mla_tree_decode's in its workspace
 * (mla_decode_check reads it), the others' in *device_status, which the caller
 * clears.
 */
#ifndef MLA_TREE_H
#define MLA_TREE_H

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_TREE_MAX_NODES 64

#define MLA_DEV_BAD_OFFSETS 0x10 /* token_offsets not as above, or a tree of more than 64 nodes */
#define MLA_DEV_BAD_PATH 0x20    /* an accepted path not strictly increasing within its tree */

/*
 * A ragged problem.  batch >= 1, tokens >= 1 (rows of the token arrays),
 * num_heads == 128, page_size == 64, max_pages_per_seq >= 1; flags 0, or
 * MLA_FLAG_POW2_MAX for the tree entry points.  batch up to 2^24;
 * batch * max_pages_per_seq, max_pages_per_seq * 64 and tokens * 128 below 2^31.
 */
typedef struct mla_ragged {
    int32_t batch;
    int32_t tokens;
    int32_t num_heads;
    int32_t page_size;
    int32_t max_pages_per_seq; /* row stride of block_table; bounds every seq_len */
    int32_t flags;
} mla_ragged;

/*
 * Absorbed and rotated queries of `tokens` tokens at explicit positions.
 *   q_nope    bf16, element (t, h, k) at t * nope_token_stride + h * nope_head_stride + k, k < 128
 *   q_pe      bf16, element (t, h, k) at t * pe_token_stride + h * pe_head_stride + k, k < 64
 *             (strides in elements, positive multiples of 8, below 2^31: both may be views of one
 *             projection's output)
 *   w_uk      [128][128][512] bf16, rope_table: of mla_prolog_rope_table
 *   positions [tokens] int32; a negative one marks a token to leave out (its outputs are not written)
 *   q_latent  [tokens][128][512] bf16, q_rope [tokens][128][64] bf16
 * The outputs are those of mla_prolog for the same tokens and positions.
 */
mla_status mla_query(int32_t tokens, const void *q_nope, int64_t nope_token_stride, int64_t nope_head_stride,
                     const void *q_pe, int64_t pe_token_stride, int64_t pe_head_stride, const void *w_uk,
                     const float *rope_table, const int32_t *positions, void *q_latent, void *q_rope,
                     int32_t *device_status, mla_stream_t stream);

/*
 * Append the tokens' rows to the paged cache: any number of tokens per
 * request (a tree, a prefill chunk), at slots seq_lens[b] - n_b .. seq_lens[b] - 1.
 *   kv_latent bf16, element (t, k) at t * latent_stride + k, k < 512
 *   k_pe      bf16, element (t, k) at t * k_pe_stride + k, k < 64
 *             (strides in elements, positive multiples of 8)
 *   kv_norm_weight [512] bf16, rms_eps finite and >= 0
 *   positions [tokens] int32 or NULL (each token's slot): the RoPE position (a tree node's is its
 *             depth past the context, whatever its slot); a negative one marks a token to leave out
 *   kv_cache  [num_pages][64][576] bf16, or for mla_cache_append_fp8 [num_pages][64][656] bytes
 *             (mla_fp8.h); only the tokens' rows are written.  Distinct tokens must have distinct rows.
 * The fp8 row is quantised from the unrounded values, s = max |c_kv| / 448 of them (1 for a zero row).
 * A latent that is not finite (NaN or infinities in kv_latent or the weight; a zero one with rms_eps = 0)
 * gives a row that is not: NaN where the arithmetic makes it in bf16, NaN codes and a NaN scale in fp8.
 * A token whose slot is out of range (MLA_DEV_BAD_SEQ_LEN) or whose page is (MLA_DEV_BAD_PAGE) is
 * not written.  With bad offsets (MLA_DEV_BAD_OFFSETS) which tokens are written is unspecified, but
 * nothing outside the pool is.  MLA_TREE_MAX_NODES does not bound n_b here.
 */
mla_status mla_cache_append(const mla_ragged *prob, const void *kv_latent, int64_t latent_stride, const void *k_pe,
                            int64_t k_pe_stride, const void *kv_norm_weight, float rms_eps, const float *rope_table,
                            const int32_t *positions, void *kv_cache, int64_t num_pages, const int32_t *block_table,
                            const int32_t *seq_lens, const int32_t *token_offsets, int32_t *device_status,
                            mla_stream_t stream);
mla_status mla_cache_append_fp8(const mla_ragged *prob, const void *kv_latent, int64_t latent_stride,
                                const void *k_pe, int64_t k_pe_stride, const void *kv_norm_weight, float rms_eps,
                                const float *rope_table, const int32_t *positions, void *kv_cache_fp8,
                                int64_t num_pages, const int32_t *block_table, const int32_t *seq_lens,
                                const int32_t *token_offsets, int32_t *device_status, mla_stream_t stream);

/*
 * Workspace bytes of mla_tree_plan / mla_tree_decode on the current device
 * (the schedule, every node's mask, fp32 partial outputs of split rows).
 */
mla_status mla_tree_workspace_size(const mla_ragged *prob, size_t *bytes);

/*
 * Build the split-KV schedule of a batch of trees: one row per node, cut over
 * the work units as mla_decode_plan cuts its rows.  masks: [tokens] uint64,
 * copied into the workspace; bits at or past the tree's size are ignored.  The
 * schedule stays valid for every later mla_tree_decode with the same problem,
 * lengths, offsets and masks (every layer of a step).  Also clears the status
 * word.  Up to 10,000 tokens (MLA_ERR_UNSUPPORTED beyond: the planner's
 * working set is held on one SM).
 * Rows of a request whose seq_len is below its node count or beyond
 * max_pages_per_seq pages: MLA_DEV_BAD_SEQ_LEN, and NaN outputs.  Bad offsets:
 * MLA_DEV_BAD_OFFSETS, and NaN outputs for every row.
 */
mla_status mla_tree_plan(const mla_ragged *prob, const int32_t *seq_lens, const int32_t *token_offsets,
                         const uint64_t *masks, void *workspace, size_t workspace_bytes, mla_stream_t stream);

/*
 * Attention of every node over its visible keys, for the schedule in
 * `workspace`: q_latent [tokens][128][512], q_rope [tokens][128][64],
 * o_latent [tokens][128][512] bf16, lse [tokens][128] fp32; cache, block table,
 * scale, flags and error contract as in mla_decode / mla_decode_fp8.  Calls
 * that share a workspace must be ordered (one stream, or events).
 */
mla_status mla_tree_decode(const mla_ragged *prob, const void *q_latent, const void *q_rope, const void *kv_cache,
                           int64_t num_pages, const int32_t *block_table, float scale, void *o_latent, float *lse,
                           void *workspace, size_t workspace_bytes, mla_stream_t stream);
mla_status mla_tree_decode_fp8(const mla_ragged *prob, const void *q_latent, const void *q_rope,
                               const void *kv_cache_fp8, int64_t num_pages, const int32_t *block_table, float scale,
                               void *o_latent, float *lse, void *workspace, size_t workspace_bytes, void *scratch,
                               size_t scratch_bytes, mla_stream_t stream);

/*
 * Bytes of the optional scratch of mla_tree_decode_fp8: room for every table
 * entry's page as bf16 rows (batch * max_pages_per_seq * 73,984).  With scratch
 * (16-byte aligned, at least this size) each page that the trees read is
 * expanded once per call and the nodes share it; without (NULL) each node expands
 * the pages again as it reads them: 64 requests of 4096 keys take 0.8 times as long
 * with 1 node each, and 1.1, 1.4 and 1.6 times with 2, 4 and 8.  The results are equal
 * bit for bit.  Concurrent calls need a scratch each.  Batches of more than 65,535
 * cannot use one (MLA_ERR_UNSUPPORTED).
 */
mla_status mla_tree_scratch_size(const mla_ragged *prob, size_t *bytes);

/*
 * The planner's algorithm on the host, for tests and tooling: the schedule
 * bytes that mla_tree_plan writes at the start of the workspace, for
 * `num_units` units.  All arrays in host memory.
 */
size_t mla_tree_plan_bytes(const mla_ragged *prob, int32_t num_units);
mla_status mla_tree_plan_host(const mla_ragged *prob, const int32_t *seq_lens_host, const int32_t *token_offsets_host,
                              const uint64_t *masks_host, int32_t num_units, void *plan_host, size_t plan_bytes);

/*
 * After verification: move the rows of each request's accepted nodes to the
 * front of its tree's slots, in every layer's cache.
 *   kv_cache    [num_layers] caches of [num_pages][64][row_bytes] bytes, layer_stride_bytes apart (a
 *               multiple of 16); row_bytes 1152 (bf16 rows) or 656 (fp8 rows).  One block table for all.
 *   paths       [batch][max_path] int32: path_lens[b] node indices, strictly increasing, below n_b
 *   path_lens   [batch] int32, 0 <= path_lens[b] <= min(max_path, n_b); max_path in [1, 64]
 *   new_seq_lens [batch] int32 out: seq_lens[b] - n_b + path_lens[b] (another array than seq_lens)
 * Only slots L_b - n_b .. + path_lens[b] - 1 are written; a request's tree slots must lie in no other
 * request's.  A bad path (MLA_DEV_BAD_PATH), seq_len, page or tree size leaves the request's rows as they
 * were, and new_seq_lens[b] = seq_lens[b].
 */
mla_status mla_cache_commit(const mla_ragged *prob, void *kv_cache, int32_t num_layers, int64_t layer_stride_bytes,
                            int32_t row_bytes, int64_t num_pages, const int32_t *block_table,
                            const int32_t *seq_lens, const int32_t *token_offsets, const int32_t *paths,
                            int32_t max_path, const int32_t *path_lens, int32_t *new_seq_lens,
                            int32_t *device_status, mla_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_TREE_H */
