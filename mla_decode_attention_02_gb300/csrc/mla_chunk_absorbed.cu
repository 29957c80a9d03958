// Chunks of few tokens over long contexts (include/mla_chunk.h), in the absorbed form:
//
//   q_latent = q_nope W_UK[h],  o_latent = attention over the cached rows themselves,  o = W_UV[h] o_latent
//
// Every (token, key) pair costs 2 x 1088 flops a head instead of 2 x 320, but no
// key is brought into the heads' space (2 x 131072 flops a head and key), which is what
// a few tokens over a long context spend their time on otherwise.  The kernels are those of the
// decode step: the queries (their rotary parts turned by nothing, which only packs
// them), the tree variants of the main kernel with a row per token that sees its request's slots
// up to its own, and the value projection.  Of a mixed step they run over the rows of the requests in this form and
// return at once where there is none.
#include <cuda_runtime.h>

#include <cstdint>

#include "mla_chunk.cuh"
#include "mla_internal.h"
#include "mla_prolog.h"

namespace mla {
cudaError_t main_units(int32_t *units);
bool tree_plan_fits(int32_t rows, int32_t units);
mla_status launch_query(int32_t tokens, const void *q_nope, int64_t nope_token_stride, int64_t nope_head_stride,
                        const void *q_pe, int64_t pe_token_stride, int64_t pe_head_stride, const void *w_uk,
                        const float *rope_table, const int32_t *positions, void *q_latent, void *q_rope,
                        int32_t *device_status, const TreePlanRef &plan, mla_stream_t stream);
cudaError_t launch_tree_plan(const int32_t *seq_lens, const int32_t *offsets, const uint64_t *masks, const uint8_t *forms,
                             int32_t *zeros, void *ws, int32_t batch, int32_t tokens, int32_t max_pages,
                             int32_t num_units, cudaStream_t stream);
cudaError_t launch_main(const void *q_latent, const void *q_rope, const void *kv, int64_t num_pages,
                        const int32_t *block_table, float scale, void *ws, void *o_latent, float *lse, int32_t batch,
                        int32_t s_q, int32_t max_pages, int32_t num_units, uint64_t wait_limit_ns, uint32_t test_flags,
                        uint32_t flags, bool fp8, bool tree, const void *expanded, cudaStream_t stream);
cudaError_t launch_expand(const void *ws, const void *kv_cache_fp8, int64_t num_pages, const int32_t *block_table,
                          void *expanded, int32_t batch, int32_t tokens, int32_t max_pages, int32_t num_units,
                          cudaStream_t stream);
cudaError_t launch_combine(const void *ws, void *o_latent, float *lse, int32_t batch, int32_t s_q, int32_t max_pages,
                           int32_t num_units, bool tree, bool sparse, cudaStream_t stream);
mla_status launch_epilog_uv(int64_t tokens, const void *o_latent, const void *w_uv, void *o_v, const TreePlanRef &plan,
                            int32_t *device_status, mla_stream_t stream);
namespace {

constexpr uint64_t kWaitNs = 2000000000ull;

// Scratch: absorbed queries, packed rotary parts, latent outputs, lse.
struct AbsorbedScratch {
    size_t q_latent, q_rope, o_latent, lse, total;
};

AbsorbedScratch absorbed_scratch(int32_t tokens) {
    const size_t rows = (size_t)tokens * kHeads;
    AbsorbedScratch S;
    S.q_latent = 0;
    S.q_rope = S.q_latent + rows * kDl * 2;
    S.o_latent = S.q_rope + rows * kDr * 2;
    S.lse = S.o_latent + rows * kDl * 2;
    S.total = align_up(S.lse + rows * 4, 256);
    return S;
}

// Workspace: the schedule, then positions and a rotary table of zeros (launch_tree_plan's).
size_t zeros_at(const mla_chunk *p, int32_t units) { return make_layout(p->tokens, units, p->batch).total; }
size_t zeros_bytes(const mla_chunk *p) { return align_up(4 * ((size_t)p->tokens + MLA_ROPE_TABLE_FLOATS), 256); }

}  // namespace

// How a step is computed.  Times in microseconds, plan and attention in a graph, from which absorbed_ns and whole_ns are
// fitted (requests x keys: tokens a request: absorbed / whole):
//   1 x 512: 8: 40 / 39, 64: 46 / 40           4 x 512: 8: 43 / 94, 32: 63 / 96, 64: 107 / 99
//   1 x 2048: 64: 69 / 92, 128: 109 / 93       4 x 2048: 32: 110 / 278, 64: 202 / 281, 128: 326 / 286
//   1 x 8192: 64: 167 / 270, 128: 286 / 271    4 x 8192: 64: 515 / 1023, 128: 970 / 1027, 192: 1428 / 1158
//   1 x 32768: 1: 63 / 971, 64: 496 / 989, 128: 933 / 994, 192: 1367 / 1169
// (an fp8 cache adds some 12 us to both).  The absorbed form rounds its queries and latent outputs to bf16 as well (3.1e-3
// of the output's norm instead of 2.1e-3), so it is taken where it saves a quarter at least.
// The host knows neither which requests have tokens nor how tokens and keys are spread over them, and one form is many times
// slower than the other for some spreads (2048 tokens over 32768 keys beside 31 idle slots: 4.0 ms by keys and values,
// 14.0 absorbed; 2048 tokens beside 15 single ones over 32768 keys each: 15.4 and, a form for each request, 0.43).  So a step
// is mixed, the plan takes a form for each request, but where one is sound for the whole step whatever the spread:
//  - one request;
//  - up to kQuerySmall tokens: absorbed if an even spread saves a quarter and no spread is slower, not with all tokens at the
//    longest context that kv_tokens and the table allow;
//  - up to a tile of tokens: absorbed if it saves a quarter even so;
//  - few keys: the absorbed form could save no more than twice its fixed part.
// The launches of a form that no request takes cost some 10 us (15 over an fp8 cache), so steps of less than kMixedLeast are
// mixed only if an even spread would be absorbed.
constexpr int64_t kMixedLeast = 300000;
ChunkForm chunk_form(const mla_chunk *p, int32_t units) {
    if (!tree_plan_fits(p->tokens, units)) return ChunkForm::kWhole;
    const int64_t tokens = p->tokens, keys = p->kv_tokens, batch = p->batch, some = batch < tokens ? batch : tokens;
    const int64_t pays = kAbsorbedFixed - kWholeFixed * 3 / 4;
    if (batch == 1) return absorbed_gain(tokens, keys, units) > pays ? ChunkForm::kAbsorbed : ChunkForm::kWhole;
    const int64_t width = (int64_t)p->max_pages_per_seq * kPage, longest = keys < width ? keys : width;
    const int64_t most = kAbsorbedFixed + absorbed_ns(tokens, longest, units);
    const int64_t least = whole_ns(1, keys, units), slots = (some - 1) * whole_ns(1, 0, units);
    if (tokens <= kQuerySmall)
        return most < kWholeFixed + least && some * absorbed_gain((tokens + some - 1) / some, keys / some, units) > pays
                   ? ChunkForm::kAbsorbed
                   : ChunkForm::kWhole;
    if (tokens <= kChunkTile && most < (kWholeFixed + least) * 3 / 4) return ChunkForm::kAbsorbed;
    if ((least + slots) * 3 / 4 < 2 * kAbsorbedFixed) return ChunkForm::kWhole;
    const int64_t even = batch * absorbed_gain((tokens + batch - 1) / batch, keys / batch, units);
    return kWholeFixed + least < kMixedLeast && even <= kAbsorbedFixed ? ChunkForm::kWhole : ChunkForm::kMixed;
}

size_t absorbed_workspace_bytes(const mla_chunk *p, int32_t units) { return zeros_at(p, units) + zeros_bytes(p); }

size_t absorbed_scratch_bytes(const mla_chunk *p) { return absorbed_scratch(p->tokens).total; }

// As a tree step takes it: from two tokens a request on, up to 8 GiB.
size_t absorbed_expanded_bytes(const mla_chunk *p) {
    const size_t bytes = expanded_bytes(p->batch, p->max_pages_per_seq);
    return p->tokens >= 2 * (int64_t)p->batch && p->batch <= 65535 && bytes <= (size_t)8 << 30 ? bytes : 0;
}

mla_status absorbed_plan(const mla_chunk *p, const int32_t *seq_lens, const int32_t *offsets, const uint8_t *forms, void *ws,
                         int32_t units, cudaStream_t stream) {
    int32_t *zeros = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) + zeros_at(p, units));
    return launch_tree_plan(seq_lens, offsets, nullptr, forms, zeros, ws, p->batch, p->tokens, p->max_pages_per_seq, units,
                            stream) == cudaSuccess
               ? MLA_OK
               : MLA_ERR_CUDA;
}

mla_status absorbed_attend(const mla_chunk *p, const void *q_nope, int64_t nope_token, int64_t nope_head,
                           const void *q_rope, int64_t rope_token, int64_t rope_head, const void *w_uk, const void *w_uv,
                           const void *cache, bool fp8, int64_t num_pages, const int32_t *block_table, float scale,
                           void *out, float *lse, void *ws, bool mixed, int32_t *status, uint8_t *scratch,
                           void *expanded, int32_t units, mla_stream_t stream) {
    const AbsorbedScratch S = absorbed_scratch(p->tokens);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t *w = static_cast<uint8_t *>(ws);
    const TreePlanRef plan = {w, p->batch, p->tokens, p->max_pages_per_seq, units, mixed};
    const int32_t *zeros = reinterpret_cast<const int32_t *>(w + zeros_at(p, units));
    void *ql = scratch + S.q_latent, *qr = scratch + S.q_rope, *ol = scratch + S.o_latent;
    float *l = lse ? lse : reinterpret_cast<float *>(scratch + S.lse);
    const mla_status st = launch_query(p->tokens, q_nope, nope_token, nope_head, q_rope, rope_token, rope_head, w_uk,
                                       reinterpret_cast<const float *>(zeros + p->tokens), zeros, ql, qr, status, plan,
                                       stream);
    if (st != MLA_OK) return st;
    if (expanded && launch_expand(ws, cache, num_pages, block_table, expanded, p->batch, p->tokens, p->max_pages_per_seq,
                                  units, s) != cudaSuccess)
        return MLA_ERR_CUDA;
    // (over an fp8 cache power-of-two maxima round a weight once: see tree_decode_fp8's binding)
    const uint32_t flags = (fp8 ? MLA_FLAG_POW2_MAX : 0) | (mixed ? kMainSparse : 0);
    if (launch_main(ql, qr, cache, num_pages, block_table, scale, ws, ol, l, p->batch, p->tokens, p->max_pages_per_seq, units,
                    kWaitNs, 0, flags, fp8, true, expanded, s) != cudaSuccess ||
        launch_combine(ws, ol, l, p->batch, p->tokens, p->max_pages_per_seq, units, true, mixed, s) != cudaSuccess)
        return MLA_ERR_CUDA;
    return launch_epilog_uv(p->tokens, ol, w_uv, out, plan, status, stream);
}

}  // namespace mla
