// The accepted path's cache rows move together (include/mla_tree.h,
// mla_cache_commit): for request b and i < path_lens[b],
//
//   row of slot p + i  <-  row of slot p + path_b[i],    p = seq_lens[b] - n_b
//
// in place, in every layer.  A path is strictly increasing, so path[i] >= i: a
// destination p + i is never the source of a later row (path[j] >= j > i), only
// of an earlier one or of itself.  One thread owns one 16-byte column of a
// request's rows in one layer and walks the path in order, eight rows at a time
// (all eight loaded before the first is stored), so no thread depends on
// another.  Bound by memory: every moved row is read and written once; nodes
// that stay in place are skipped.  One CTA per request and layer: 64 requests in 61
// layers' fp8 caches, at most five moved rows each, 5.1 us (5.0 TB/s); three requests
// in four layers 1.7 us, the launch.
#include <cuda_runtime.h>

#include <cstdint>

#include "mla_fp8.h"
#include "mla_internal.h"
#include "mla_tree.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

constexpr int kRowsAhead = 8;

struct CommitParams {
    uint8_t *cache;
    const int32_t *block_table, *seq_lens, *offsets, *paths, *path_lens;
    int32_t *new_seq_lens, *status;
    int64_t layer_stride, num_pages;
    int32_t row_bytes, batch, tokens, max_pages, max_path, layers;
};

// One CTA per (request, stride of layers); thread c owns the 16-byte column c of the rows.
__global__ void __launch_bounds__(96) mla_cache_commit_kernel(const CommitParams P) {
    __shared__ int32_t path[MLA_TREE_MAX_NODES];
    const int32_t b = blockIdx.x;
    const int tid = threadIdx.x;
    ptx::pdl_wait_prior();
    ptx::pdl_launch_dependents();
    const int32_t o0 = P.offsets[b], o1 = P.offsets[b + 1], len = P.seq_lens[b], n = P.path_lens[b];
    const int64_t nodes = (int64_t)o1 - o0;
    if (nodes == 0) {   // no request in this slot of the batch
        if (blockIdx.y == 0 && tid == 0) P.new_seq_lens[b] = len;
        return;
    }
    int32_t bad = 0;
    if (o0 < 0 || nodes < 0 || nodes > MLA_TREE_MAX_NODES || o1 > P.tokens) bad |= MLA_DEV_BAD_OFFSETS;
    else if (len < nodes || len > (int64_t)P.max_pages * kPage) bad |= MLA_DEV_BAD_SEQ_LEN;
    else if (n < 0 || n > nodes || n > P.max_path) bad |= MLA_DEV_BAD_PATH;
    const int32_t p0 = bad ? 0 : len - (int32_t)nodes;
    // the tree's slots lie in two pages at most
    int32_t page0 = 0, page1 = 0;
    if (!bad) {
        if (tid < n) {
            const int32_t at = P.paths[(size_t)b * P.max_path + tid];
            const int32_t before = tid > 0 ? P.paths[(size_t)b * P.max_path + tid - 1] : -1;
            if (at <= before || at >= nodes) bad |= MLA_DEV_BAD_PATH;
            path[tid] = at;
        }
        const int32_t *row = P.block_table + (size_t)b * P.max_pages;
        page0 = row[p0 / kPage];
        page1 = row[(len - 1) / kPage];
        if (page0 < 0 || page0 >= P.num_pages || page1 < 0 || page1 >= P.num_pages) bad |= MLA_DEV_BAD_PAGE;
    }
    const bool none = __syncthreads_or(bad) != 0;
    if (bad && blockIdx.y == 0) atomicOr(P.status, bad);
    if (blockIdx.y == 0 && tid == 0) P.new_seq_lens[b] = none ? len : p0 + n;
    if (none || tid * 16 >= P.row_bytes) return;
    const int32_t edge = (p0 / kPage + 1) * kPage;   // first slot of the second page
    for (int32_t layer = blockIdx.y; layer < P.layers; layer += gridDim.y) {
        uint8_t *base = P.cache + layer * P.layer_stride + tid * 16;
        auto at = [&](int32_t i) {
            const int32_t slot = p0 + i;
            return reinterpret_cast<uint4 *>(base + ((size_t)(slot < edge ? page0 : page1) * kPage + slot % kPage) *
                                                        P.row_bytes);
        };
        for (int32_t i0 = 0; i0 < n; i0 += kRowsAhead) {
            uint4 v[kRowsAhead];
#pragma unroll
            for (int j = 0; j < kRowsAhead; ++j)
                if (i0 + j < n && path[i0 + j] != i0 + j) v[j] = *at(path[i0 + j]);
#pragma unroll
            for (int j = 0; j < kRowsAhead; ++j)
                if (i0 + j < n && path[i0 + j] != i0 + j) *at(i0 + j) = v[j];
        }
    }
}

bool aligned(const void *p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace mla

extern "C" mla_status mla_cache_commit(const mla_ragged *prob, void *kv_cache, int32_t num_layers,
                                       int64_t layer_stride_bytes, int32_t row_bytes, int64_t num_pages,
                                       const int32_t *block_table, const int32_t *seq_lens,
                                       const int32_t *token_offsets, const int32_t *paths, int32_t max_path,
                                       const int32_t *path_lens, int32_t *new_seq_lens, int32_t *device_status,
                                       mla_stream_t stream) {
    mla::NvtxRange nvtx_range("mla_cache_commit");
    using namespace mla;
    const mla_status st = check_ragged(prob, 0);
    if (st != MLA_OK) return st;
    if (!aligned(kv_cache, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(token_offsets, 4) ||
        !aligned(paths, 4) || !aligned(path_lens, 4) || !aligned(new_seq_lens, 4) || !aligned(device_status, 4) ||
        new_seq_lens == seq_lens)
        return MLA_ERR_INVALID_ARG;
    if (row_bytes != 2 * kDrow && row_bytes != MLA_FP8_ROW_BYTES) return MLA_ERR_INVALID_ARG;
    if (num_layers < 1 || num_pages < 1 || num_pages >= (int64_t)1 << 31 || max_path < 1 ||
        max_path > MLA_TREE_MAX_NODES || layer_stride_bytes % 16 ||
        (num_layers > 1 && layer_stride_bytes < num_pages * kPage * row_bytes))
        return MLA_ERR_INVALID_ARG;
    CommitParams p;
    p.cache = static_cast<uint8_t *>(kv_cache);
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.offsets = token_offsets;
    p.paths = paths;
    p.path_lens = path_lens;
    p.new_seq_lens = new_seq_lens;
    p.status = device_status;
    p.layer_stride = layer_stride_bytes;
    p.num_pages = num_pages;
    p.row_bytes = row_bytes;
    p.batch = prob->batch;
    p.tokens = prob->tokens;
    p.max_pages = prob->max_pages_per_seq;
    p.max_path = max_path;
    p.layers = num_layers;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)prob->batch, (unsigned)(num_layers < 65535 ? num_layers : 65535));
    cfg.blockDim = dim3(96);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mla_cache_commit_kernel, p) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
