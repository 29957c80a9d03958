// What the kernels of chunk attention share (include/mla_chunk.h): the layout of
// a step's plan and of the scratch that holds the heads' keys and values.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime_api.h>

#include "mla_chunk.h"
#include "mla_internal.h"

namespace mla {

constexpr uint32_t kChunkMagic = 0x43414c4du;   // "MLAC"
constexpr int kChunkTile = 256;                 // tokens of a tile: two MMA tiles of 128
constexpr int kDn = 128, kDv = 128;             // no-position and value dims of a head
constexpr int kPairRows = 256;                  // scratch rows that an SM pair fills at a time: four pages

// The tokens of a tile: rows t0 .. t0 + count - 1 of the token arrays, the first at slot slot0 of its
// request (-1: the request is in error, its rows become NaN), whose keys begin at scratch row base; the
// request's tiles are first .. end - 1.
struct ChunkTile {
    int32_t t0, count, slot0, base, first, end, pad[2];
};
static_assert(sizeof(ChunkTile) == 32, "tile layout");
// A page that the chunks read, in the order of the scratch: its block table entry and the tokens in it.
struct ChunkPage {
    int32_t entry, valid;
};

// The workspace: a PlanHeader (s_q = tokens, num_items = tiles, num_parts = pages, total_cost = kv_tokens),
// the tiles, the pages.
struct ChunkLayout {
    size_t tiles, pages, total;
    int32_t max_tiles, max_pages;
};

MLA_HD ChunkLayout chunk_layout(int32_t batch, int32_t tokens, int64_t kv_tokens) {
    ChunkLayout L;
    L.max_tiles = tokens / kChunkTile + (batch < tokens ? batch : tokens) + 1;
    L.max_pages = (int32_t)(kv_tokens / kPage);
    L.tiles = sizeof(PlanHeader);
    L.pages = L.tiles + sizeof(ChunkTile) * (size_t)L.max_tiles;
    L.total = align_up(L.pages + sizeof(ChunkPage) * (size_t)L.max_pages, 256);
    return L;
}

// Scratch rows: every page, and one page of zeros behind them (a key tile of 128 rows may begin at the last
// page), in whole pairs of tiles.
MLA_HD int64_t chunk_rows(int64_t kv_tokens) {
    return (kv_tokens + kPage + kPairRows - 1) / kPairRows * kPairRows;
}
// The scratch: k_rope of every row [rows][64], then [heads][rows][256]: keys (128) and values (128).
MLA_HD size_t chunk_rope_bytes(int64_t kv_tokens) { return (size_t)chunk_rows(kv_tokens) * kDr * 2; }
MLA_HD size_t chunk_head_bytes(int64_t kv_tokens) { return (size_t)chunk_rows(kv_tokens) * (kDn + kDv) * 2; }

// Checks of a chunk problem that make no CUDA call.
mla_status check_chunk(const mla_chunk *p);

// How a step is computed.  kMixed: the plan takes one of the two forms for each request, and both run over theirs.
enum class ChunkForm { kWhole, kAbsorbed, kMixed };
ChunkForm chunk_form(const mla_chunk *p, int32_t units);
size_t chunk_workspace_bytes(const mla_chunk *p, ChunkForm form, int32_t units);

// The two forms' times for a request of n tokens at the end of `keys` keys, in nanoseconds and without the steps' fixed
// parts (mla_chunk_absorbed.cu: from a sweep of both).  n below 2^20, keys below 2^31.
constexpr int64_t kWholeFixed = 19000, kAbsorbedFixed = 36000;
MLA_HD int64_t absorbed_ns(int64_t n, int64_t keys, int32_t units) {
    return 34 * n + 1044 * n * (keys + kItemCost * kPage) / (kPage * units);
}
MLA_HD int64_t whole_ns(int64_t n, int64_t keys, int32_t units) {
    return keys * (248 + 50 * ((n + 127) / 128)) / 10 + 4550 * ((n + kChunkTile - 1) / kChunkTile) * kHeads / (2 * units);
}
// What the absorbed form saves (it is taken where it saves a quarter at least: its roundings are more).
MLA_HD int64_t absorbed_gain(int64_t n, int64_t keys, int32_t units) {
    return whole_ns(n, keys, units) * 3 / 4 - absorbed_ns(n, keys, units);
}

// The absorbed form (mla_chunk_absorbed.cu): its workspace (of a mixed step: behind the whole form's, from
// mixed_forms on a byte per request, whether it is computed so, and from mixed_tree on its schedule) and scratch, its calls.
MLA_HD size_t mixed_forms(const mla_chunk *p) { return chunk_layout(p->batch, p->tokens, p->kv_tokens).total; }
MLA_HD size_t mixed_tree(const mla_chunk *p) { return align_up(mixed_forms(p) + (size_t)p->batch, 256); }
size_t absorbed_workspace_bytes(const mla_chunk *p, int32_t units);
size_t absorbed_scratch_bytes(const mla_chunk *p);    // without room for expanded pages, for which
size_t absorbed_expanded_bytes(const mla_chunk *p);   // 0: pages are not expanded
// forms: the requests that are computed so (null: all).
mla_status absorbed_plan(const mla_chunk *p, const int32_t *seq_lens, const int32_t *offsets, const uint8_t *forms, void *ws,
                         int32_t units, cudaStream_t stream);
mla_status absorbed_attend(const mla_chunk *p, const void *q_nope, int64_t nope_token, int64_t nope_head,
                           const void *q_rope, int64_t rope_token, int64_t rope_head, const void *w_uk, const void *w_uv,
                           const void *cache, bool fp8, int64_t num_pages, const int32_t *block_table, float scale,
                           void *out, float *lse, void *ws, bool mixed, int32_t *status, uint8_t *scratch,
                           void *expanded, int32_t units, mla_stream_t stream);

}  // namespace mla
