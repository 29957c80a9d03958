// Ragged append to the paged latent cache, bf16 or fp8 rows.
//
// For token t, the i-th of request b's n_b new tokens (include/mla_tree.h):
//
//   row of slot seq_lens[b] - n_b + i  <-  [ x / sqrt(mean x^2 + eps) * gamma | RoPE(k_pe, pos) ]
//
// with x the 512 latent values, in fp32 and rounded once: to bf16, or to the
// fp8 row's codes c / s (e4m3), k / s (bf16) and s = max |c| / 448.
//
// One warp per token, warps striding over the tokens: lane l holds latent
// chunks l and l + 32 (8 values each, 16-byte loads that are contiguous over the
// warp) and the rotary pair l, so the norm, the row's maximum and the rotation
// need no shared memory.  The token's request is found by a 32-way search of
// token_offsets (two or three rounds of one load per lane) while the token's
// values are already on their way.  Bound by memory: 1152 bytes in and 1152 or
// 656 out per token (8780 tokens of six prompts in 4.5 us, 4.5 TB/s); small batches
// by the chain of dependent loads (offsets, length and table, page) and the launch
// (8 tokens 1.9 us, 1300 tokens into fp8 rows 3.1 us).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "mla_fp8.h"
#include "mla_internal.h"
#include "mla_rope.cuh"
#include "mla_tree.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

constexpr int kAppendWarps = 8;
constexpr int kAppendGrid = 152 * 8;   // CTAs at most: eight of 256 threads fill an SM

struct AppendParams {
    const __nv_bfloat16 *kv_latent;
    const __nv_bfloat16 *k_pe;
    const __nv_bfloat16 *gamma;
    const float *rope_table;
    const int32_t *positions;   // or null: the slots
    const int32_t *block_table;
    const int32_t *seq_lens;
    const int32_t *offsets;
    uint8_t *cache;
    int32_t *status;
    int64_t latent_stride, k_pe_stride, num_pages;
    float eps;
    int32_t batch, tokens, max_pages;
};

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[j]));
        f[2 * j] = x.x;
        f[2 * j + 1] = x.y;
    }
}

// Codes of 448 f / amax.
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float amax) {
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        c[j / 4] |= (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(f[j] * 448.f, amax), __NV_SATFINITE, __NV_E4M3)
                    << (8 * (j % 4));
    return make_uint2(c[0], c[1]);
}

// The request b with off[b] <= tok < off[b + 1], or -1 (a padding row, or offsets out of
// order): every lane probes one of 32 evenly spaced entries a round.  The indexes stay in
// [0, batch] whatever the array holds.
__device__ __forceinline__ int32_t find_request(const int32_t *off, int32_t batch, int32_t tok, int lane,
                                                int32_t &first, int32_t &end) {
    int32_t lo = 0, hi = batch;   // the answer lies in [lo, hi)
    while (hi - lo > 1) {
        const int32_t step = (hi - lo + 32) / 33;
        const int32_t at = lo + (lane + 1) * step;
        const bool below = at < hi && off[at] <= tok;
        const int32_t n = __popc(__ballot_sync(0xffffffffu, below));
        hi = min(hi, lo + (n + 1) * step);
        lo += n * step;
    }
    first = off[lo];
    end = off[lo + 1];
    return first <= tok && tok < end ? lo : -1;
}

template <bool kFp8>
__global__ void __launch_bounds__(32 * kAppendWarps) mla_cache_append_kernel(const AppendParams P) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    ptx::pdl_wait_prior();
    ptx::pdl_launch_dependents();
    if (blockIdx.x == 0) {   // the offsets as a whole
        bool bad = false;
        for (int32_t b = threadIdx.x; b < P.batch; b += 32 * kAppendWarps)
            bad |= P.offsets[b] > P.offsets[b + 1] || (b == 0 && P.offsets[0] != 0) ||
                   (b == P.batch - 1 && P.offsets[P.batch] > P.tokens);
        if (bad) atomicOr(P.status, MLA_DEV_BAD_OFFSETS);
    }
    const float g_hi = P.rope_table[lane], g_lo = P.rope_table[kPairs + lane];
    float ga[8], gb[8];
    unpack8(reinterpret_cast<const uint4 *>(P.gamma)[lane], ga);
    unpack8(reinterpret_cast<const uint4 *>(P.gamma)[lane + 32], gb);
    for (int32_t tok = blockIdx.x * kAppendWarps + warp; tok < P.tokens; tok += gridDim.x * kAppendWarps) {
        const uint4 *src = reinterpret_cast<const uint4 *>(P.kv_latent + tok * P.latent_stride);
        const uint4 va = src[lane], vb = src[lane + 32];
        const uint32_t kv = reinterpret_cast<const uint32_t *>(P.k_pe + tok * P.k_pe_stride)[lane];
        const int32_t given = P.positions ? P.positions[tok] : 0;
        int32_t first, end;
        const int32_t b = find_request(P.offsets, P.batch, tok, lane, first, end);
        if (b < 0 || given < 0) continue;
        const int64_t slot = (int64_t)P.seq_lens[b] - end + tok;
        if (slot < 0 || slot >= (int64_t)P.max_pages * kPage) {
            if (lane == 0) atomicOr(P.status, MLA_DEV_BAD_SEQ_LEN);
            continue;
        }
        const int32_t page = P.block_table[(size_t)b * P.max_pages + slot / kPage];
        if (page < 0 || page >= P.num_pages) {
            if (lane == 0) atomicOr(P.status, MLA_DEV_BAD_PAGE);
            continue;
        }
        float a[8], c[8];
        unpack8(va, a);
        unpack8(vb, c);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(a[j], a[j], fmaf(c[j], c[j], ss));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(ss * (1.0f / kDl) + P.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) {   // x * gamma: exact, a product of two bf16 values has 16 bits
            a[j] *= ga[j];
            c[j] *= gb[j];
        }
        float sn, cs;
        rope_sincos(P.positions ? given : (int32_t)slot, g_hi, g_lo, sn, cs);
        const float2 k = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&kv));
        const float k0 = k.x * cs - k.y * sn, k1 = k.x * sn + k.y * cs;
        const size_t row = (size_t)page * kPage + slot % kPage;
        if constexpr (kFp8) {
            // the row's maximum by its bits: a NaN's are above every number's, so one NaN is kept
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                top = max(top, max(__float_as_uint(fabsf(a[j])), __float_as_uint(fabsf(c[j]))));
            const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, top));
            // The norm's factor cancels in c / s = 448 (x gamma) / max |x gamma|: both sides of the
            // division are exact, so each code is the correctly rounded quotient's.  s is 0 for a zero
            // row (all of x gamma, or a norm past fp32's range, as in bf16).  It is no finite number if
            // the latent is none (NaN or infinities in x or gamma; 0 / 0 without eps): the row then holds
            // NaN codes and a NaN scale, and spoils what sees it as such a bf16 row does.
            float s = __fdiv_rn(amax * inv, 448.f);
            const bool lost = !(s < INFINITY), zero = s == 0.f;
            if (zero) s = 1.f;
            if (lost) s = __int_as_float(0x7fffffff);
            auto codes = [&](const float (&f)[8]) {
                if (lost) return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
                return zero ? make_uint2(0, 0) : codes8(f, amax);
            };
            uint8_t *dst = P.cache + row * MLA_FP8_ROW_BYTES;
            reinterpret_cast<uint2 *>(dst)[lane] = codes(a);
            reinterpret_cast<uint2 *>(dst)[lane + 32] = codes(c);
            reinterpret_cast<uint32_t *>(dst + kDl)[lane] = pack_bf16x2(__fdiv_rn(k0, s), __fdiv_rn(k1, s));
            if (lane < 4) reinterpret_cast<uint32_t *>(dst + kDl + 2 * kDr)[lane] = lane == 0 ? __float_as_uint(s) : 0u;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a[j] *= inv;
                c[j] *= inv;
            }
            uint8_t *dst = P.cache + row * (kDrow * 2);
            reinterpret_cast<uint4 *>(dst)[lane] = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                                              pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7]));
            reinterpret_cast<uint4 *>(dst)[lane + 32] = make_uint4(pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3]),
                                                                   pack_bf16x2(c[4], c[5]), pack_bf16x2(c[6], c[7]));
            reinterpret_cast<uint32_t *>(dst + 2 * kDl)[lane] = pack_bf16x2(k0, k1);
        }
    }
}

bool aligned(const void *p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

mla_status append(const mla_ragged *prob, const void *kv_latent, int64_t latent_stride, const void *k_pe,
                  int64_t k_pe_stride, const void *kv_norm_weight, float rms_eps, const float *rope_table,
                  const int32_t *positions, void *kv_cache, int64_t num_pages, const int32_t *block_table,
                  const int32_t *seq_lens, const int32_t *token_offsets, int32_t *device_status, bool fp8,
                  mla_stream_t stream) {
    const mla_status st = check_ragged(prob, 0);
    if (st != MLA_OK) return st;
    if (!aligned(kv_latent, 16) || !aligned(k_pe, 16) || !aligned(kv_norm_weight, 16) || !aligned(kv_cache, 16) ||
        !aligned(rope_table, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(token_offsets, 4) ||
        !aligned(device_status, 4) || (reinterpret_cast<uintptr_t>(positions) & 3u))
        return MLA_ERR_INVALID_ARG;
    if (latent_stride < 1 || latent_stride % 8 || k_pe_stride < 1 || k_pe_stride % 8 ||
        latent_stride >= (int64_t)1 << 31 || k_pe_stride >= (int64_t)1 << 31)
        return MLA_ERR_INVALID_ARG;
    if (num_pages < 1 || num_pages >= (int64_t)1 << 31 || !std::isfinite(rms_eps) || rms_eps < 0.f)
        return MLA_ERR_INVALID_ARG;
    AppendParams p;
    p.kv_latent = static_cast<const __nv_bfloat16 *>(kv_latent);
    p.k_pe = static_cast<const __nv_bfloat16 *>(k_pe);
    p.gamma = static_cast<const __nv_bfloat16 *>(kv_norm_weight);
    p.rope_table = rope_table;
    p.positions = positions;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.offsets = token_offsets;
    p.cache = static_cast<uint8_t *>(kv_cache);
    p.status = device_status;
    p.latent_stride = latent_stride;
    p.k_pe_stride = k_pe_stride;
    p.num_pages = num_pages;
    p.eps = rms_eps;
    p.batch = prob->batch;
    p.tokens = prob->tokens;
    p.max_pages = prob->max_pages_per_seq;
    const int ctas = (prob->tokens + kAppendWarps - 1) / kAppendWarps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas < kAppendGrid ? ctas : kAppendGrid));
    cfg.blockDim = dim3(32 * kAppendWarps);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = fp8 ? cudaLaunchKernelEx(&cfg, mla_cache_append_kernel<true>, p)
                              : cudaLaunchKernelEx(&cfg, mla_cache_append_kernel<false>, p);
    return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace

// Checks of a ragged problem that make no CUDA call (flags: those allowed).
mla_status check_ragged(const mla_ragged *p, int32_t flags) {
    if (!p || p->batch < 1 || p->tokens < 1 || p->max_pages_per_seq < 1 || (p->flags & ~flags) != 0)
        return MLA_ERR_INVALID_ARG;
    if (p->num_heads != MLA_NUM_HEADS || p->page_size != MLA_PAGE_SIZE) return MLA_ERR_UNSUPPORTED;
    if ((int64_t)p->batch * p->max_pages_per_seq >= (int64_t)1 << 31) return MLA_ERR_UNSUPPORTED;
    if ((int64_t)p->max_pages_per_seq * MLA_PAGE_SIZE >= (int64_t)1 << 31) return MLA_ERR_UNSUPPORTED;
    if (p->batch > 1 << 24) return MLA_ERR_UNSUPPORTED;
    if ((int64_t)p->tokens * MLA_NUM_HEADS >= (int64_t)1 << 31) return MLA_ERR_UNSUPPORTED;
    return MLA_OK;
}

}  // namespace mla

extern "C" mla_status mla_cache_append(const mla_ragged *prob, const void *kv_latent, int64_t latent_stride,
                                       const void *k_pe, int64_t k_pe_stride, const void *kv_norm_weight,
                                       float rms_eps, const float *rope_table, const int32_t *positions,
                                       void *kv_cache, int64_t num_pages, const int32_t *block_table,
                                       const int32_t *seq_lens, const int32_t *token_offsets,
                                       int32_t *device_status, mla_stream_t stream) {
    mla::NvtxRange nvtx_range("mla_cache_append");
    return mla::append(prob, kv_latent, latent_stride, k_pe, k_pe_stride, kv_norm_weight, rms_eps, rope_table,
                       positions, kv_cache, num_pages, block_table, seq_lens, token_offsets, device_status, false,
                       stream);
}

extern "C" mla_status mla_cache_append_fp8(const mla_ragged *prob, const void *kv_latent, int64_t latent_stride,
                                           const void *k_pe, int64_t k_pe_stride, const void *kv_norm_weight,
                                           float rms_eps, const float *rope_table, const int32_t *positions,
                                           void *kv_cache_fp8, int64_t num_pages, const int32_t *block_table,
                                           const int32_t *seq_lens, const int32_t *token_offsets,
                                           int32_t *device_status, mla_stream_t stream) {
    mla::NvtxRange nvtx_range("mla_cache_append_fp8");
    return mla::append(prob, kv_latent, latent_stride, k_pe, k_pe_stride, kv_norm_weight, rms_eps, rope_table,
                       positions, kv_cache_fp8, num_pages, block_table, seq_lens, token_offsets, device_status, true,
                       stream);
}
