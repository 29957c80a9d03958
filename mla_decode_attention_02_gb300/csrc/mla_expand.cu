// The fp8 cache pages of a batch of trees as bf16 rows, ahead of their attention.
//
// All nodes of a tree read the same pages, and the attention kernel's own
// expansion of e4m3 codes (once per node and page, mla_main_tc.cu) sets the rate
// of its page loop.  Expanding each page once, here, leaves the loop with the
// loads of a bf16 cache: row j of request b's page becomes
//
//   [ value(code_i), i < 512 | k_rope / s ]  (576 bf16 values, exact: every e4m3 value is a bf16 value)
//
// and its scale s goes to an array beside, for the softmax.  Values and roundings of
// the result are those of the in-kernel expansion.  One warp per row: lane l turns
// 16 codes into two 16-byte stores.  Bound by memory: 656 bytes in, 1156 out per row
// (17 requests, 43,600 rows: about 12 us, most of it the first touch of the cache).
// With it a page of tree attention costs a bf16 page (1.0 us a unit instead of 1.9):
// 64 requests of 4096 keys with 1, 2, 4, 8 nodes each took 143, 273, 509, 989 us with the
// in-kernel expansion and 174, 246, 368, 612 with this one.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "mla_fp8.h"
#include "mla_internal.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

constexpr int kExpandWarps = 8;

// Two e4m3 codes -> two bf16 values (exact).
__device__ __forceinline__ uint32_t expand2(uint32_t codes) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xFFFFu), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// CTA (x, b): pages x, x + gridDim.x, ... of request b.
__global__ void __launch_bounds__(32 * kExpandWarps)
mla_tree_expand_kernel(const uint8_t *__restrict__ ws, const uint8_t *__restrict__ cache, int64_t num_pages,
                       const int32_t *__restrict__ block_table, uint8_t *__restrict__ out, int32_t batch,
                       int32_t tokens, int32_t max_pages, int32_t num_units) {
    ptx::pdl_wait_prior();
    ptx::pdl_launch_dependents();
    const PlanHeader *hdr = reinterpret_cast<const PlanHeader *>(ws);
    // (a workspace that holds another schedule is flagged by the main kernel)
    if (hdr->magic != kTreeMagic || hdr->batch != batch || hdr->s_q != tokens || hdr->num_units != num_units ||
        hdr->max_pages != max_pages)
        return;
    const int32_t b = blockIdx.y;
    const int32_t pages = reinterpret_cast<const int32_t *>(ws + make_layout(tokens, num_units, batch).tree_pages)[b];
    float *scales = reinterpret_cast<float *>(out + expanded_scales(batch, max_pages));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int32_t j = blockIdx.x; j < pages; j += gridDim.x) {
        const size_t entry = (size_t)b * max_pages + j;
        const int32_t page = block_table[entry];
        if (page < 0 || page >= num_pages) continue;   // its rows come out as NaN, flagged
        const uint8_t *src = cache + (size_t)page * kPage * MLA_FP8_ROW_BYTES;
        uint8_t *dst = out + entry * kExpandedPage;
#pragma unroll 4
        for (int r = warp; r < kPage; r += kExpandWarps) {
            const uint8_t *row = src + r * MLA_FP8_ROW_BYTES;
            const uint4 c = reinterpret_cast<const uint4 *>(row)[lane];
            uint4 *to = reinterpret_cast<uint4 *>(dst + (size_t)r * kDrow * 2);
            // lane 0: the scale; lanes 0-7: k_rope / s
            if (lane < kDr * 2 / 16) to[2 * kDl / 16 + lane] = reinterpret_cast<const uint4 *>(row + kDl)[lane];
            if (lane == 0) scales[entry * kPage + r] = *reinterpret_cast<const float *>(row + kDl + 2 * kDr);
            to[2 * lane] = make_uint4(expand2(c.x), expand2(c.x >> 16), expand2(c.y), expand2(c.y >> 16));
            to[2 * lane + 1] = make_uint4(expand2(c.z), expand2(c.z >> 16), expand2(c.w), expand2(c.w >> 16));
        }
    }
}

}  // namespace

cudaError_t launch_expand(const void *ws, const void *kv_cache_fp8, int64_t num_pages, const int32_t *block_table,
                          void *expanded, int32_t batch, int32_t tokens, int32_t max_pages, int32_t num_units,
                          cudaStream_t stream) {
    // about eight CTAs per SM over the requests (65535 at most: the caller checks)
    int32_t x = 8 * 2 * num_units / batch;
    x = x < 1 ? 1 : x > max_pages ? max_pages : x;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)x, (unsigned)batch);
    cfg.blockDim = dim3(32 * kExpandWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mla_tree_expand_kernel, static_cast<const uint8_t *>(ws),
                              static_cast<const uint8_t *>(kv_cache_fp8), num_pages, block_table,
                              static_cast<uint8_t *>(expanded), batch, tokens, max_pages, num_units);
}

}  // namespace mla
