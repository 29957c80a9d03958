// The plan of a step's chunks (include/mla_chunk.h, mla_chunk_plan): tiles of up
// to 256 tokens, and the list of the pages that the requests read, in the order of
// the scratch.
//
// A request's tiles stand together, its last (which reads the most keys) first, the
// requests with the longest tiles first: what runs at the same time then shares keys, and
// what runs last is short.
// Of a mixed step the plan first decides which requests the absorbed form takes (mla_chunk_absorbed.cu): those where it
// saves a quarter at least, if that pays for its launches; they have no tiles and pages here.
// One CTA: a scan over the requests (their pages and tiles), then tiles and pages
// by all threads, each finding its request in the scan; the tiles are ranked by
// counting.
#include <cuda_runtime.h>

#include <cstdint>

#include "mla_chunk.cuh"
#include "sm103_ptx.cuh"

namespace mla {
cudaError_t main_units(int32_t *units);
namespace {

constexpr int kPlanThreads = 1024;
// Tiles are put in order up to this many (every tile is compared with every other); more run in token order,
// where so many even out by themselves.
constexpr int kRankTiles = 1024;

struct RankKey {
    int32_t longest;      // key tiles of the request's longest tile
    int32_t first, tiles; // the request's first tile in token order, and how many it has
};

// Inclusive scan of a and b over the block.
__device__ __forceinline__ void block_scan(int32_t &a, int32_t &b, int32_t (*sums)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
    if (lane == 31) {
        sums[warp][0] = a;
        sums[warp][1] = b;
    }
    __syncthreads();
    int32_t x = sums[lane][0], y = sums[lane][1];   // 32 warps: a sum a lane
    x = lane < warp ? x : 0;
    y = lane < warp ? y : 0;
    a += __reduce_add_sync(0xffffffffu, x);
    b += __reduce_add_sync(0xffffffffu, y);
    __syncthreads();
}
static_assert(kPlanThreads == 1024, "a warp's lanes hold the warps' sums");

// The entry e of the prefix sums with sum[e] <= i < sum[e + 1].
__device__ __forceinline__ int find(const int32_t *sum, int n, int32_t i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (sum[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// kMixed: of a mixed step (with forms).
template <bool kMixed>
__global__ void __launch_bounds__(kPlanThreads)
mla_chunk_plan_kernel(const int32_t *__restrict__ seq_lens, const int32_t *__restrict__ off, uint8_t *ws, int32_t batch,
                      int32_t tokens, int32_t max_pages, int64_t kv_tokens, uint8_t *forms, int32_t units) {
    __shared__ int32_t sums[kPlanThreads / 32][2];
    __shared__ unsigned long long all_pages, all_gain;
    __shared__ int32_t s_page[kPlanThreads + 1], s_first[kPlanThreads + 1];   // pages and tiles before each request
    __shared__ int4 s_tile[kRankTiles];   // t0, count, slot0, base
    __shared__ RankKey s_key[kRankTiles];
    const ChunkLayout L = chunk_layout(batch, tokens, kv_tokens);
    PlanHeader *hdr = reinterpret_cast<PlanHeader *>(ws);
    ChunkTile *tiles = reinterpret_cast<ChunkTile *>(ws + L.tiles);
    ChunkPage *pages = reinterpret_cast<ChunkPage *>(ws + L.pages);
    const int t = threadIdx.x;
    if (t == 0) all_pages = all_gain = 0;
    ptx::pdl_wait_prior();
    ptx::pdl_launch_dependents();
    // A request's tokens, length, pages and tiles (none without tokens, or in the absorbed form); ok: its seq_len is sound.
    struct Request {
        int32_t begin, n, len, np, nt;
        bool ok, absorbed;
        __device__ int64_t gain(int32_t units) const { return nt > 0 && ok ? absorbed_gain(n, len, units) : 0; }
    };
    bool take = false;   // whether any request is in the absorbed form
    auto leave = [&](Request &r) {
        r.absorbed = kMixed && take && r.gain(units) > 0;
        if (r.absorbed) r.np = r.nt = 0;
    };
    auto request = [&](int32_t b) {
        Request r = {};
        r.ok = true;
        if (b >= batch) return r;
        r.begin = off[b];
        r.n = off[b + 1] - r.begin;
        r.len = seq_lens[b];
        if (r.n <= 0) return r;
        r.nt = (r.n - 1) / kChunkTile + 1;
        r.ok = r.len >= r.n && r.len <= (int64_t)max_pages * kPage;
        if (r.ok) r.np = (r.len - 1) / kPage + 1;
        leave(r);
        return r;
    };
    // The offsets as a whole, and the pages of all requests.
    bool bad_off = t == 0 && (off[0] != 0 || off[batch] > tokens), bad_len = false, keeps = false;
    int64_t mine = 0, gain = 0;
    Request own;
    for (int32_t b = t; b < batch || b == t; b += kPlanThreads) {
        own = request(b);
        bad_off |= b < batch && (own.begin < 0 || own.n < 0);
        bad_len |= !own.ok;
        mine += own.np;
        if constexpr (kMixed) {
            const int64_t g = own.gain(units);
            if (g > 0) gain += g;
            keeps |= own.nt > 0 && g <= 0;
        }
    }
    bad_off = __syncthreads_or(bad_off);
    bad_len = __syncthreads_or(bad_len);
    if constexpr (kMixed) {
        // (in whole nanoseconds, so that the sum does not depend on its order)
        if (gain) atomicAdd(&all_gain, (unsigned long long)gain);
        keeps = __syncthreads_or(keeps);
        // a step all in the absorbed form saves the other's launches; its kernels look through all tokens (9431: some 80 us)
        const int64_t fixed = kAbsorbedFixed + 10 * (int64_t)tokens - (keeps ? 0 : kWholeFixed * 3 / 4);
        take = !bad_off && (int64_t)all_gain > fixed;
        mine = 0;
        for (int32_t b = t; b < batch; b += kPlanThreads) {
            if (batch > kPlanThreads) own = request(b);
            else leave(own);
            forms[b] = own.absorbed;
            mine += own.np;
        }
    }
    if (mine) atomicAdd(&all_pages, (unsigned long long)mine);
    __syncthreads();
    const bool over = !bad_off && (int64_t)all_pages * kPage > kv_tokens;
    const int32_t num_pages = bad_off || over ? 0 : (int32_t)all_pages;
    int32_t num_tiles = 0, done_pages = 0;
    if (bad_off) {   // every row becomes NaN
        num_tiles = (tokens - 1) / kChunkTile + 1;
        for (int32_t i = t; i < num_tiles; i += kPlanThreads) {
            const int32_t left = tokens - i * kChunkTile;
            tiles[i] = {i * kChunkTile, left < kChunkTile ? left : kChunkTile, -1, 0, i, i + 1, {0, 0}};
        }
    } else {
        for (int32_t b0 = 0; b0 < batch; b0 += kPlanThreads) {
            const int32_t left = batch - b0 < kPlanThreads ? batch - b0 : kPlanThreads;
            if (batch > kPlanThreads) own = request(b0 + t);
            int32_t p = over ? 0 : own.np, i = own.nt;
            block_scan(p, i, sums);
            s_page[t + 1] = p;
            s_first[t + 1] = i;
            if (t == 0) s_page[0] = s_first[0] = 0;
            __syncthreads();
            const int32_t n_pages = s_page[kPlanThreads], n_tiles = s_first[kPlanThreads];
            for (int32_t k = t; k < n_tiles; k += kPlanThreads) {
                const int e = find(s_first, left, k);
                const Request r = request(b0 + e);
                const int32_t skip = (k - s_first[e]) * kChunkTile, rest = r.n - skip;
                const ChunkTile tile = {r.begin + skip, rest < kChunkTile ? rest : kChunkTile,
                                        r.ok && !over ? r.len - r.n + skip : -1, (done_pages + s_page[e]) * kPage,
                                        num_tiles + s_first[e], num_tiles + s_first[e + 1], {0, 0}};
                const int32_t at = num_tiles + k;
                if (at < kRankTiles) {
                    s_tile[at] = make_int4(tile.t0, tile.count, tile.slot0, tile.base);
                    // the last tile reads the most keys, but takes half the time with up to 128 tokens
                    const int32_t last = r.n - (r.nt - 1) * kChunkTile <= 128 ? r.len / 2 : r.len;
                    const int32_t before = r.nt > 1 ? r.len - (r.n - (r.nt - 1) * kChunkTile) : 0;
                    s_key[at] = {tile.slot0 < 0 ? 0 : last > before ? last : before, tile.first, r.nt};
                }
                tiles[at] = tile;
            }
            for (int32_t k = t; k < n_pages; k += kPlanThreads) {
                const int e = find(s_page, left, k);
                const int32_t j = k - s_page[e], rest = seq_lens[b0 + e] - j * kPage;
                pages[done_pages + k] = {(int32_t)((int64_t)(b0 + e) * max_pages + j), rest < kPage ? rest : kPage};
            }
            num_tiles += n_tiles;
            done_pages += n_pages;
            __syncthreads();
        }
        if (num_tiles <= kRankTiles)
            for (int32_t i = t; i < num_tiles; i += kPlanThreads) {
                const RankKey k = s_key[i];
                int32_t at = 0;
                for (int32_t j = 0; j < num_tiles; ++j) {
                    const RankKey o = s_key[j];
                    at += o.longest > k.longest ||
                          (o.longest == k.longest && (o.first < k.first || (o.first == k.first && j > i)));
                }
                const int4 v = s_tile[i];
                const int32_t first = at - (k.first + k.tiles - 1 - i);
                tiles[at] = {v.x, v.y, v.z, v.w, first, first + k.tiles, {0, 0}};
            }
    }
    if (t == 0) {
        PlanHeader h = {};
        h.magic = kChunkMagic;
        h.batch = batch;
        h.s_q = tokens;
        h.max_pages = max_pages;
        h.num_items = num_tiles;
        h.num_parts = num_pages;
        h.status = bad_off ? MLA_DEV_BAD_OFFSETS
                           : (over ? MLA_DEV_BAD_KV_TOKENS : 0) | (bad_len ? MLA_DEV_BAD_SEQ_LEN : 0);
        h.total_cost = kv_tokens;
        *hdr = h;
    }
}

bool aligned(const void *p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

size_t chunk_workspace_bytes(const mla_chunk *p, ChunkForm form, int32_t units) {
    return form == ChunkForm::kAbsorbed ? absorbed_workspace_bytes(p, units)
           : form == ChunkForm::kMixed  ? mixed_tree(p) + absorbed_workspace_bytes(p, units)
                                        : chunk_layout(p->batch, p->tokens, p->kv_tokens).total;
}

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
    int32_t units = 0;
    if (mla::main_units(&units) != cudaSuccess) return MLA_ERR_CUDA;
    *bytes = mla::chunk_workspace_bytes(prob, mla::chunk_form(prob, units), units);
    return MLA_OK;
}

extern "C" mla_status mla_chunk_plan(const mla_chunk *prob, const int32_t *seq_lens, const int32_t *token_offsets,
                                     void *workspace, size_t workspace_bytes, mla_stream_t stream) {
    mla::NvtxRange nvtx_range("mla_chunk_plan");
    using namespace mla;
    const mla_status st = check_chunk(prob);
    if (st != MLA_OK) return st;
    if (!aligned(seq_lens, 4) || !aligned(token_offsets, 4) || !aligned(workspace, 16)) return MLA_ERR_INVALID_ARG;
    int32_t units = 0;
    if (main_units(&units) != cudaSuccess) return MLA_ERR_CUDA;
    const ChunkForm form = chunk_form(prob, units);
    if (workspace_bytes < chunk_workspace_bytes(prob, form, units)) return MLA_ERR_WORKSPACE;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (form == ChunkForm::kAbsorbed) return absorbed_plan(prob, seq_lens, token_offsets, nullptr, workspace, units, s);
    uint8_t *ws = static_cast<uint8_t *>(workspace), *forms = form == ChunkForm::kMixed ? ws + mixed_forms(prob) : nullptr;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    auto *kernel = forms ? mla_chunk_plan_kernel<true> : mla_chunk_plan_kernel<false>;
    if (cudaLaunchKernelEx(&cfg, kernel, seq_lens, token_offsets, ws, prob->batch, prob->tokens,
                           prob->max_pages_per_seq, prob->kv_tokens, forms, units) != cudaSuccess)
        return MLA_ERR_CUDA;
    return forms ? absorbed_plan(prob, seq_lens, token_offsets, forms, ws + mixed_tree(prob), units, s) : MLA_OK;
}
