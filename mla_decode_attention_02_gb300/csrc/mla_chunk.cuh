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
// A page that the chunks read, in the order of the scratch: its block table entry (-1: none, a page of
// zeros) and the tokens in it.
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

// The absorbed form (mla_chunk_absorbed.cu): whether a problem takes it, its workspace and scratch, its calls.
bool chunk_absorbed(const mla_chunk *p, int32_t units);
size_t absorbed_workspace_bytes(const mla_chunk *p, int32_t units);
size_t absorbed_scratch_bytes(const mla_chunk *p, bool fp8);
mla_status absorbed_plan(const mla_chunk *p, const int32_t *seq_lens, const int32_t *offsets, void *ws, int32_t units,
                         cudaStream_t stream);
mla_status absorbed_attend(const mla_chunk *p, const void *q_nope, int64_t nope_token, int64_t nope_head,
                           const void *q_rope, int64_t rope_token, int64_t rope_head, const void *w_uk, const void *w_uv,
                           const void *cache, bool fp8, int64_t num_pages, const int32_t *block_table, float scale,
                           void *out, float *lse, void *ws, uint8_t *scratch, size_t scratch_bytes, int32_t units,
                           mla_stream_t stream);

}  // namespace mla
