// The plan of a step's chunks (include/mla_chunk.h, mla_chunk_plan): tiles of up
// to 256 tokens, those that read the most keys first, and the list of the pages
// that the requests read, in the order of the scratch.
//
// One CTA: a scan over the requests (their pages and tiles), the tiles ranked by
// counting, then the pages written by whole warps.
#include <cuda_runtime.h>

#include <cstdint>

#include "mla_chunk.cuh"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

constexpr int kPlanThreads = 1024;
// Tiles are put in order of their keys up to this many (every tile is compared with every other); more
// run in token order, where so many even out by themselves.
constexpr int kRankTiles = 2048;

// Inclusive scan of a and b over the block.
__device__ __forceinline__ void block_scan(int64_t &a, int64_t &b, int64_t (*sums)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
    __syncthreads();
    if (lane == 31) {
        sums[warp][0] = a;
        sums[warp][1] = b;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        a += sums[w][0];
        b += sums[w][1];
    }
}

__global__ void __launch_bounds__(kPlanThreads)
mla_chunk_plan_kernel(const int32_t *__restrict__ seq_lens, const int32_t *__restrict__ off, uint8_t *ws, int32_t batch,
                      int32_t tokens, int32_t max_pages, int64_t kv_tokens) {
    __shared__ int64_t sums[kPlanThreads / 32][2];
    __shared__ int64_t carry[2];
    __shared__ ChunkTile s_tile[kRankTiles];
    const ChunkLayout L = chunk_layout(batch, tokens, kv_tokens);
    PlanHeader *hdr = reinterpret_cast<PlanHeader *>(ws);
    ChunkTile *tiles = reinterpret_cast<ChunkTile *>(ws + L.tiles);
    ChunkPage *pages = reinterpret_cast<ChunkPage *>(ws + L.pages);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    ptx::pdl_wait_prior();
    ptx::pdl_launch_dependents();
    // The offsets as a whole, and the pages of all requests.
    bool bad_off = false, bad_len = false;
    if (t == 0) bad_off = off[0] != 0 || off[batch] > tokens;
    int64_t total_pages = 0, total_tiles = 0;
    // a request's pages and tiles (none if it has no tokens); false: its seq_len is in error
    auto request = [&](int32_t b, int64_t &np, int64_t &nt) {
        const int32_t n = off[b + 1] - off[b], len = seq_lens[b];
        np = nt = 0;
        if (n <= 0) return true;
        nt = (n + kChunkTile - 1) / kChunkTile;
        const bool ok = len >= n && len <= (int64_t)max_pages * kPage;
        if (ok) np = (len + kPage - 1) / kPage;
        return ok;
    };
    for (int32_t b = t; b < batch; b += kPlanThreads) {
        if (off[b] > off[b + 1] || off[b] < 0) {
            bad_off = true;
            continue;
        }
        int64_t np, nt;
        bad_len |= !request(b, np, nt);
        total_pages += np;
        total_tiles += nt;
    }
    bad_off = __syncthreads_or(bad_off);
    bad_len = __syncthreads_or(bad_len);
    block_scan(total_pages, total_tiles, sums);
    if (t == kPlanThreads - 1) {
        carry[0] = total_pages;
        carry[1] = total_tiles;
    }
    __syncthreads();
    total_pages = carry[0];
    total_tiles = carry[1];
    __syncthreads();
    const bool over = !bad_off && total_pages * kPage > kv_tokens;
    if (t == 0) {
        PlanHeader h = {};
        h.magic = kChunkMagic;
        h.batch = batch;
        h.s_q = tokens;
        h.max_pages = max_pages;
        h.num_items = bad_off ? (tokens + kChunkTile - 1) / kChunkTile : (int32_t)total_tiles;
        h.num_parts = bad_off || over ? 0 : (int32_t)total_pages;
        h.status = bad_off ? MLA_DEV_BAD_OFFSETS
                           : (over ? MLA_DEV_BAD_KV_TOKENS : 0) | (bad_len ? MLA_DEV_BAD_SEQ_LEN : 0);
        h.total_cost = kv_tokens;
        *hdr = h;
        carry[0] = carry[1] = 0;
    }
    __syncthreads();
    if (bad_off) {   // every row becomes NaN
        for (int32_t i = t; i < (tokens + kChunkTile - 1) / kChunkTile; i += kPlanThreads) {
            const int32_t left = tokens - i * kChunkTile;
            tiles[i] = {i * kChunkTile, left < kChunkTile ? left : kChunkTile, -1, 0};
        }
        return;
    }
    const bool rank = total_tiles <= kRankTiles;
    ChunkTile *to = rank ? s_tile : tiles;
    for (int32_t b0 = 0; b0 < batch; b0 += kPlanThreads) {
        const int32_t b = b0 + t;
        int64_t np = 0, nt = 0;
        const bool ok = b >= batch || request(b, np, nt);
        if (over) np = 0;
        int64_t p = np, i = nt;
        block_scan(p, i, sums);
        const int64_t first_page = carry[0] + p - np, first_tile = carry[1] + i - nt;
        __syncthreads();
        if (t == kPlanThreads - 1) {
            carry[0] += p;
            carry[1] += i;
        }
        __syncthreads();
        // each warp writes its requests' tiles and pages one request after another
        for (int l = 0; l < 32; ++l) {
            const int64_t n_tiles = __shfl_sync(0xffffffffu, nt, l);
            if (n_tiles == 0) continue;
            const int64_t at = __shfl_sync(0xffffffffu, first_tile, l), page0 = __shfl_sync(0xffffffffu, first_page, l);
            const int64_t n_pages = __shfl_sync(0xffffffffu, np, l);
            const bool good = __shfl_sync(0xffffffffu, (int)(ok && !over), l);
            const int32_t r = b0 + warp * 32 + l, begin = off[r], n = off[r + 1] - begin, len = seq_lens[r];
            for (int64_t k = lane; k < n_tiles; k += 32) {
                const int32_t skip = (int32_t)k * kChunkTile, left = n - skip;
                to[at + k] = {begin + skip, left < kChunkTile ? left : kChunkTile, good ? len - n + skip : -1,
                              (int32_t)(page0 * kPage)};
            }
            for (int64_t k = lane; k < n_pages; k += 32) {
                const int32_t left = len - (int32_t)k * kPage;
                pages[page0 + k] = {(int32_t)((int64_t)r * max_pages + k), left < kPage ? left : kPage};
            }
        }
    }
    if (!rank) return;
    __syncthreads();
    // longest first (ties: in token order); a tile in error reads no key
    const int32_t n = (int32_t)total_tiles;
    auto keys = [&](int32_t i) { return s_tile[i].slot0 < 0 ? 0 : s_tile[i].slot0 + s_tile[i].count; };
    for (int32_t i = t; i < n; i += kPlanThreads) {
        const int32_t mine = keys(i);
        int32_t at = 0;
        for (int32_t j = 0; j < n; ++j) {
            const int32_t other = keys(j);
            at += other > mine || (other == mine && j < i);
        }
        tiles[at] = s_tile[i];
    }
}

bool aligned(const void *p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

// Checks of a chunk problem that make no CUDA call.
mla_status check_chunk(const mla_chunk *p) {
    if (!p) return MLA_ERR_INVALID_ARG;
    const mla_ragged r = {p->batch, p->tokens, p->num_heads, p->page_size, p->max_pages_per_seq, p->flags};
    const mla_status st = check_ragged(&r, 0);
    if (st != MLA_OK) return st;
    if (p->kv_tokens < kPage || p->kv_tokens % kPage) return MLA_ERR_INVALID_ARG;
    return p->kv_tokens >= (int64_t)1 << 30 ? MLA_ERR_UNSUPPORTED : MLA_OK;
}

}  // namespace mla

extern "C" mla_status mla_chunk_workspace_size(const mla_chunk *prob, size_t *bytes) {
    const mla_status st = mla::check_chunk(prob);
    if (st != MLA_OK) return st;
    if (!bytes) return MLA_ERR_INVALID_ARG;
    *bytes = mla::chunk_layout(prob->batch, prob->tokens, prob->kv_tokens).total;
    return MLA_OK;
}

extern "C" mla_status mla_chunk_plan(const mla_chunk *prob, const int32_t *seq_lens, const int32_t *token_offsets,
                                     void *workspace, size_t workspace_bytes, mla_stream_t stream) {
    mla::NvtxRange nvtx_range("mla_chunk_plan");
    using namespace mla;
    const mla_status st = check_chunk(prob);
    if (st != MLA_OK) return st;
    if (!aligned(seq_lens, 4) || !aligned(token_offsets, 4) || !aligned(workspace, 16)) return MLA_ERR_INVALID_ARG;
    if (workspace_bytes < chunk_layout(prob->batch, prob->tokens, prob->kv_tokens).total) return MLA_ERR_WORKSPACE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mla_chunk_plan_kernel, seq_lens, token_offsets, static_cast<uint8_t *>(workspace),
                              prob->batch, prob->tokens, prob->max_pages_per_seq, prob->kv_tokens) == cudaSuccess
               ? MLA_OK
               : MLA_ERR_CUDA;
}
