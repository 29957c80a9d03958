/*
 * mla_chunk.h - C ABI of a layer step over chunks of prompts: rotary positions
 * of the chunk's queries, attention of its tokens over their requests' paged
 * caches, and the layer's boundary (residual addition and RMSNorm).
 *
 * A prompt is prefilled in chunks.  The tokens of a step's chunks are a ragged
 * array as in mla_tree.h (request b's n_b tokens are rows token_offsets[b] ..
 * token_offsets[b + 1] - 1), and mla_cache_append has put their rows into the
 * cache, at slots L_b - n_b .. L_b - 1 (L_b = seq_lens[b], the chunk included).
 * Each token sees its request's slots up to its own:
 *
 *   k[j][h] = [ W_UK[h] r_j[0:512] | r_j[512:576] ],  v[j][h] = W_UV[h] r_j[0:512]     r_j: the cache row
 *   s_j     = scale * [ q_nope[t][h] | q_rope[t][h] ] . k[j][h]      0 <= j <= slot of t
 *   o[t][h] = sum_j softmax(s)_j v[j][h],  lse = ln sum_j exp(s_j)                     (mla_chunk_attend)
 *
 * which is the attention of mla_decode and mla_epilog_uv without absorbed
 * weights: 2 * 320 flops a head for each (token, key) pair instead of 2 * 1088,
 * and 2 * 131072 a head for each key, once.  The pages followed describe decode
 * only ("Huawei Ascend servers: DeepSeek V3/R1 inference best practice" section
 * 3.2.1 names the unabsorbed form as the one of prefill); rotary scaling for
 * long contexts is YaRN (Peng et al., 2023).
 *
 * Conventions as in mla_decode.h and mla_tree.h: device pointers, caller-owned
 * buffers, work enqueued on `stream`, nothing synchronises and nothing is
 * allocated; host argument errors return a status and enqueue nothing.
 */
#ifndef MLA_CHUNK_H
#define MLA_CHUNK_H

#include "mla_decode.h"
#include "mla_tree.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_DEV_BAD_KV_TOKENS 0x40 /* the requests hold more pages than kv_tokens says */

/* ------------------------------------------------------------------ rotary positions */

#define MLA_LAYOUT_INTERLEAVED 0 /* pairs (2i, 2i + 1) */
#define MLA_LAYOUT_HALF 1        /* pairs (i, i + dims / 2) */

/*
 * The rotary table of a model whose positions are scaled for long contexts:
 * table[i] + table[dims / 2 + i] = turns per position of pair i, in the form of
 * mla_prolog_rope_table (for dims = 64 the entry points that take that table
 * take this one).  With r_i = rope_base^(-2i / dims) a pair's rate is
 *   r_i (1 - w_i) + r_i / factor w_i,   w_i = clamp((i - low) / (high - low), 0, 1)
 *   low = max(0, floor(p(beta_fast))),  high = min(dims - 1, ceil(p(beta_slow))),
 *   p(n) = dims ln(original_positions / (2 pi n)) / (2 ln rope_base)
 * (high - low at least 0.001): pairs that turn more than beta_fast times within
 * the original length keep their rate, those that turn less than beta_slow
 * times are slowed by the factor.  factor = 1 gives mla_prolog_rope_table's values.
 * dims 16, 32, 64, 128 or 256; rope_base finite and > 1; factor finite and >= 1;
 * original_positions >= 1; beta_fast >= beta_slow > 0, finite.
 */
mla_status mla_rope_table_scaled(double rope_base, int32_t dims, double factor, int32_t original_positions,
                                 double beta_fast, double beta_slow, float *table, mla_stream_t stream);

/*
 * Rotate x by the tokens' positions: out[t][h] = magnitude * R(positions[t]) x[t][h].
 *   x, out     bf16, element (t, h, k) at t * token_stride + h * head_stride + k, k < dims (strides in
 *              elements, positive multiples of 8, below 2^31): a view of part of each head.  out may be x
 *              with the same strides; otherwise they do not overlap.  16-byte aligned.
 *   positions  [tokens] int32; a negative one marks a token to leave out (its rows are not written)
 *   table      [dims] floats, of mla_rope_table_scaled or, for dims = 64, mla_prolog_rope_table
 *   layout     MLA_LAYOUT_*;  inverse: 0, or 1 to rotate back (the transpose, and so the gradient)
 *   magnitude  finite: a factor on the result (1; YaRN's attention factor where a model has one)
 * Angles as in mla_prolog; the result is rounded once.  dims as above, tokens and heads >= 1,
 * tokens * heads below 2^31.
 */
mla_status mla_rotate(int32_t tokens, int32_t heads, int32_t dims, const void *x, int64_t x_token_stride,
                      int64_t x_head_stride, const int32_t *positions, const float *table, int32_t layout,
                      int32_t inverse, float magnitude, void *out, int64_t out_token_stride,
                      int64_t out_head_stride, mla_stream_t stream);

/* ------------------------------------------------------------------ residual and norm */

/*
 * z = x + residual (x alone where residual is NULL), y = z / sqrt(mean z^2 + rms_eps) * weight over each
 * row of `hidden` values, in fp32 and rounded once.
 *   x, residual   bf16, element (t, k) at t * stride + k (strides in elements, multiples of 8)
 *   weight        [hidden] bf16
 *   out           [tokens][hidden] bf16: y
 *   residual_out  [tokens][hidden] bf16, or NULL: z; may be residual itself, if that is dense
 * hidden: a multiple of 8 from 8 to 16384.  Base pointers 16-byte aligned.
 */
mla_status mla_residual_norm(int32_t tokens, int32_t hidden, const void *x, int64_t x_stride, const void *residual,
                             int64_t residual_stride, const void *weight, float rms_eps, void *out,
                             void *residual_out, mla_stream_t stream);

/*
 * The same with y in 8 bits: codes [tokens][hidden] e4m3 bytes and scales [tokens][ceil(hidden / group)] fp32,
 * y ~ code * scale.  scale = max |y| / 448 over the group's values (1 where they are all zero); the codes are
 * rounded from the unrounded values.  group 128, or 0 for one scale per row.  A group whose values are not all
 * finite has NaN codes and a NaN scale.  codes: 8-byte aligned.
 */
mla_status mla_residual_norm_fp8(int32_t tokens, int32_t hidden, const void *x, int64_t x_stride,
                                 const void *residual, int64_t residual_stride, const void *weight, float rms_eps,
                                 int32_t group, void *codes, float *scales, void *residual_out,
                                 mla_stream_t stream);

/* ------------------------------------------------------------------ attention of chunks */

/*
 * A chunk problem.  batch, tokens, num_heads, page_size and max_pages_per_seq as in mla_ragged (flags 0);
 * kv_tokens: at least the sum over the requests with tokens of their seq_lens, each rounded up to whole
 * pages; it sizes the workspace and the scratch.  A multiple of 64, below 2^30.
 */
typedef struct mla_chunk {
    int32_t batch;
    int32_t tokens;
    int32_t num_heads;
    int32_t page_size;
    int32_t max_pages_per_seq;
    int32_t flags;
    int64_t kv_tokens;
} mla_chunk;

/*
 * Two forms compute a request: every head's keys and values worked out once from its cached rows (the whole form), or,
 * for few tokens over a long context, the absorbed form of mla_decode with its roundings (absorbed queries and latent
 * outputs in bf16).  By both forms' measured times the absorbed one is taken where it saves a quarter at least (up to some
 * 100 tokens).  A step of one request, of up to 80 tokens or of few keys (below some 9000, unless the absorbed form suits
 * them spread evenly) has one form, chosen from the problem alone; any other step is mixed, and mla_chunk_plan takes a form
 * for each request, whatever the others hold.
 *
 * Workspace bytes of mla_chunk_plan / mla_chunk_attend on the current device.
 */
mla_status mla_chunk_workspace_size(const mla_chunk *prob, size_t *bytes);

/*
 * Scratch bytes of mla_chunk_attend (fp8 = 1: mla_chunk_attend_fp8) with the keys and values of `heads` heads at
 * once (1 .. 128): 128 bytes a key and 512 a key and head, rounded up to 256 keys.  In the absorbed form instead 279 KB a token
 * whatever `heads`, and over an fp8 cache room to expand each page once for all tokens (mla_tree_scratch_size) if
 * they average two a request and it takes no more than 8 GiB; less than that runs without.  A mixed step: both.
 */
mla_status mla_chunk_scratch_size(const mla_chunk *prob, int32_t heads, int32_t fp8, size_t *bytes);

/*
 * Lay out a step's chunks: tiles of up to 256 tokens, longest first, and the pages that they read.  Valid for
 * every later mla_chunk_attend with the same problem, lengths and offsets (every layer of a step).  Clears
 * the status word (mla_decode_check reads it).
 * A request whose seq_len is below its token count or beyond max_pages_per_seq pages: MLA_DEV_BAD_SEQ_LEN and
 * NaN outputs for its tokens.  Bad offsets (MLA_DEV_BAD_OFFSETS) or more pages than kv_tokens
 * (MLA_DEV_BAD_KV_TOKENS): NaN outputs for every row.  (The absorbed form does not depend on kv_tokens and
 * does not check it: of a mixed step the requests in that form are not counted and keep their outputs.)
 */
mla_status mla_chunk_plan(const mla_chunk *prob, const int32_t *seq_lens, const int32_t *token_offsets,
                          void *workspace, size_t workspace_bytes, mla_stream_t stream);

/*
 * Attention of every token over its request's slots up to its own.
 *   q_nope, q_rope  bf16, element (t, h, k) at t * token_stride + h * head_stride + k (k < 128, k < 64; strides
 *                   in elements, positive multiples of 8, below 2^31); q_rope is rotated (mla_rotate)
 *   w_uk, w_uv      [128][128][512] bf16
 *   kv_cache        [num_pages][64][576] bf16, or for mla_chunk_attend_fp8 [num_pages][64][656] bytes
 *   out             [tokens][128][128] bf16 (what mla_epilog_oproj takes); rows behind the last request are
 *                   not written
 *   lse             [tokens][128] fp32 or NULL
 *   scratch         at least mla_chunk_scratch_size for one head; with room for fewer than 128 heads the call
 *                   runs in passes of as many heads as fit (128-byte aligned)
 * Keys are rounded to bf16, values and the softmax's weights to fp16: a score is off by the rounding of its key, and
 * lse with it; a value beyond 65504 gives NaN to the tokens that see it, and one below 2^-14 is off by up to 2^-25 (the
 * absorbed form has neither border).  A page index outside the pool: MLA_DEV_BAD_PAGE, and NaN for
 * the tokens that see it.  Slots that a token does not see may hold anything.  Calls that share a workspace
 * or a scratch must be ordered.  scale finite and > 0.
 */
mla_status mla_chunk_attend(const mla_chunk *prob, const void *q_nope, int64_t nope_token_stride,
                            int64_t nope_head_stride, const void *q_rope, int64_t rope_token_stride,
                            int64_t rope_head_stride, const void *w_uk, const void *w_uv, const void *kv_cache,
                            int64_t num_pages, const int32_t *block_table, float scale, void *out, float *lse,
                            void *workspace, size_t workspace_bytes, void *scratch, size_t scratch_bytes,
                            mla_stream_t stream);
mla_status mla_chunk_attend_fp8(const mla_chunk *prob, const void *q_nope, int64_t nope_token_stride,
                                int64_t nope_head_stride, const void *q_rope, int64_t rope_token_stride,
                                int64_t rope_head_stride, const void *w_uk, const void *w_uv,
                                const void *kv_cache_fp8, int64_t num_pages, const int32_t *block_table, float scale,
                                void *out, float *lse, void *workspace, size_t workspace_bytes, void *scratch,
                                size_t scratch_bytes, mla_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_CHUNK_H */
