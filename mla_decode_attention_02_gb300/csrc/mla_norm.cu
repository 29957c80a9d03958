// The layer's boundary (include/mla_chunk.h): residual addition and RMSNorm, the
// result in bf16 or in 8 bits with a scale per 128 values or per row.
//
//   z = x + residual,  y = z / sqrt(mean z^2 + eps) * weight
//   fp8: s = max |y| / 448 over the group,  code = e4m3(y / s)
//
// One CTA per row (8191 rows of 7168 to e4m3: 62.3 us, 6.6 TB/s; with CTAs that stay and take row after
// row 65 to 70, as their number fits the SMs or not).  A thread holds up to kMaxPer runs of eight values
// (16-byte loads, contiguous over a warp) from the load to the last store, so a row
// is read once; one block-wide sum, and for a scale per row one block-wide maximum.
// A group of 128 values is 16 neighbouring lanes' runs.  y / s = 448 (z w) / max |z w|: the
// norm's factor cancels, and one division a group is left.  Bound by memory: six bytes a value in and kept, one or
// two out (2049 rows to bf16: 19.4 us, 6.1 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "mla_chunk.h"
#include "mla_internal.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

constexpr int kNormThreads = 256;   // at most
constexpr int kMaxPer = 8;          // runs a thread holds at most: 8 x 8 x 256 = 16384 values a row
constexpr int kNormWarps = kNormThreads / 32;

struct NormParams {
    const __nv_bfloat16 *x, *residual, *weight;
    __nv_bfloat16 *out, *residual_out;
    uint8_t *codes;
    float *scales;
    int64_t x_stride, residual_stride;
    float eps, inv_hidden;
    int32_t tokens, hidden, groups;   // groups: scales a row
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

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

enum Output : int { kBf16 = 0, kRowScale = 1, kGroupScale = 2 };

// The scale of a group whose largest |z w| is amax, and what its z w take to become codes: first lift (a power
// of two, 1 unless 448 / amax would overflow), then factor.  s is 0 for a group of zeros (or a norm past fp32's
// range), whose scale is 1 and codes 0; it is no finite number if a value is none.
__device__ __forceinline__ float group_scale(float amax, float inv, float &lift, float &factor) {
    float s = __fdiv_rn(amax * inv, 448.f);
    lift = amax < 1e-30f ? 0x1p100f : 1.f;
    factor = __fdiv_rn(448.f, amax * lift);
    if (s == 0.f) {
        s = 1.f;
        factor = 0.f;
    }
    if (!(s < INFINITY)) s = factor = __int_as_float(0x7fffffff);
    return s;
}

__device__ __forceinline__ uint2 codes8(const float (&f)[8], float factor) {
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c[j] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * j] * factor, f[2 * j + 1] * factor), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

template <int kPer, Output kOut>
__global__ void __launch_bounds__(kNormThreads) mla_residual_norm_kernel(const NormParams P) {
    __shared__ float sums[kNormWarps];
    __shared__ uint32_t tops[kNormWarps];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, threads = blockDim.x, warps = threads >> 5;
    const int runs = P.hidden / 8;
    ptx::pdl_wait_prior();
    ptx::pdl_launch_dependents();
    const int64_t row = blockIdx.x;
    const uint4 *x = reinterpret_cast<const uint4 *>(P.x + row * P.x_stride);
    const uint4 *r = P.residual ? reinterpret_cast<const uint4 *>(P.residual + row * P.residual_stride) : nullptr;
    uint4 xv[kPer], rv[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int at = t + i * threads;
        xv[i] = at < runs ? x[at] : make_uint4(0, 0, 0, 0);
        rv[i] = r && at < runs ? r[at] : make_uint4(0, 0, 0, 0);
    }
    float z[kPer][8];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        float a[8];
        unpack8(xv[i], a);
        unpack8(rv[i], z[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            z[i][j] = r ? a[j] + z[i][j] : a[j];   // (x alone keeps its negative zeros)
            sum = fmaf(z[i][j], z[i][j], sum);
        }
        const int at = t + i * threads;
        if (P.residual_out && at < runs)
            reinterpret_cast<uint4 *>(P.residual_out + row * P.hidden)[at] = pack8(z[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    // z w, and its largest magnitude by its bits: a NaN's are above every number's
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int at = t + i * threads;
        float w[8];
        unpack8(at < runs ? reinterpret_cast<const uint4 *>(P.weight)[at] : make_uint4(0, 0, 0, 0), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            z[i][j] *= w[j];
            if constexpr (kOut == kRowScale) top = max(top, __float_as_uint(fabsf(z[i][j])));
        }
    }
    if constexpr (kOut == kRowScale) top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) {
        sums[warp] = sum;
        if constexpr (kOut == kRowScale) tops[warp] = top;
    }
    __syncthreads();
    sum = 0.f;
    for (int w = 0; w < warps; ++w) {
        sum += sums[w];
        if constexpr (kOut == kRowScale) top = max(top, tops[w]);
    }
    const float inv = rsqrtf(sum * P.inv_hidden + P.eps);
    if constexpr (kOut == kBf16) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = t + i * threads;
#pragma unroll
            for (int j = 0; j < 8; ++j) z[i][j] *= inv;
            if (at < runs) reinterpret_cast<uint4 *>(P.out + row * P.hidden)[at] = pack8(z[i]);
        }
    } else {
        float lift = 1.f, factor = 0.f;
        if constexpr (kOut == kRowScale) {
            const float s = group_scale(__uint_as_float(top), inv, lift, factor);
            if (t == 0) P.scales[row] = s;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = t + i * threads;
            if constexpr (kOut == kGroupScale) {
                uint32_t g = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) g = max(g, __float_as_uint(fabsf(z[i][j])));
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) g = max(g, __shfl_xor_sync(0xffffffffu, g, o));
                const float s = group_scale(__uint_as_float(g), inv, lift, factor);
                if ((lane & 15) == 0 && at < runs) P.scales[row * P.groups + at / 16] = s;
            }
            if (lift != 1.f) {
#pragma unroll
                for (int j = 0; j < 8; ++j) z[i][j] *= lift;
            }
            if (at < runs)
                reinterpret_cast<uint2 *>(P.codes + row * P.hidden)[at] = codes8(z[i], factor);
        }
    }
}

bool aligned(const void *p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <int kPer>
cudaError_t launch_norm(const cudaLaunchConfig_t &cfg, const NormParams &p, Output out) {
    return out == kBf16       ? cudaLaunchKernelEx(&cfg, mla_residual_norm_kernel<kPer, kBf16>, p)
           : out == kRowScale ? cudaLaunchKernelEx(&cfg, mla_residual_norm_kernel<kPer, kRowScale>, p)
                              : cudaLaunchKernelEx(&cfg, mla_residual_norm_kernel<kPer, kGroupScale>, p);
}

mla_status residual_norm(int32_t tokens, int32_t hidden, const void *x, int64_t x_stride, const void *residual,
                         int64_t residual_stride, const void *weight, float rms_eps, void *out, void *codes,
                         float *scales, Output kind, void *residual_out, mla_stream_t stream) {
    if (tokens < 1 || hidden < 8 || !std::isfinite(rms_eps) || rms_eps < 0.f) return MLA_ERR_INVALID_ARG;
    if (hidden % 8 || hidden > 8 * kMaxPer * kNormThreads) return MLA_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(weight, 16) || (residual && !aligned(residual, 16)) ||
        (residual_out && !aligned(residual_out, 16)))
        return MLA_ERR_INVALID_ARG;
    if (kind == kBf16 ? !aligned(out, 16) : !aligned(codes, 8) || !aligned(scales, 4)) return MLA_ERR_INVALID_ARG;
    for (const int64_t s : {x_stride, residual ? residual_stride : 8})
        if (s < 1 || s % 8 || s >= (int64_t)1 << 31) return MLA_ERR_INVALID_ARG;
    NormParams p;
    p.x = static_cast<const __nv_bfloat16 *>(x);
    p.residual = static_cast<const __nv_bfloat16 *>(residual);
    p.weight = static_cast<const __nv_bfloat16 *>(weight);
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.residual_out = static_cast<__nv_bfloat16 *>(residual_out);
    p.codes = static_cast<uint8_t *>(codes);
    p.scales = scales;
    p.x_stride = x_stride;
    p.residual_stride = residual_stride;
    p.eps = rms_eps;
    p.inv_hidden = 1.0f / (float)hidden;
    p.tokens = tokens;
    p.hidden = hidden;
    p.groups = (hidden + 127) / 128;
    // as few runs a thread as 256 threads allow, and no more warps than those runs need
    const int runs = hidden / 8, per = (runs + kNormThreads - 1) / kNormThreads;
    const int threads = ((runs + per - 1) / per + 31) / 32 * 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)tokens);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    switch (per) {
        case 1: e = launch_norm<1>(cfg, p, kind); break;
        case 2: e = launch_norm<2>(cfg, p, kind); break;
        case 3: e = launch_norm<3>(cfg, p, kind); break;
        case 4: e = launch_norm<4>(cfg, p, kind); break;
        case 5: e = launch_norm<5>(cfg, p, kind); break;
        case 6: e = launch_norm<6>(cfg, p, kind); break;
        case 7: e = launch_norm<7>(cfg, p, kind); break;
        default: e = launch_norm<8>(cfg, p, kind); break;
    }
    return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace
}  // namespace mla

extern "C" mla_status mla_residual_norm(int32_t tokens, int32_t hidden, const void *x, int64_t x_stride,
                                        const void *residual, int64_t residual_stride, const void *weight,
                                        float rms_eps, void *out, void *residual_out, mla_stream_t stream) {
    mla::NvtxRange nvtx_range("mla_residual_norm");
    return mla::residual_norm(tokens, hidden, x, x_stride, residual, residual_stride, weight, rms_eps, out, nullptr,
                              nullptr, mla::kBf16, residual_out, stream);
}

extern "C" mla_status mla_residual_norm_fp8(int32_t tokens, int32_t hidden, const void *x, int64_t x_stride,
                                            const void *residual, int64_t residual_stride, const void *weight,
                                            float rms_eps, int32_t group, void *codes, float *scales,
                                            void *residual_out, mla_stream_t stream) {
    mla::NvtxRange nvtx_range("mla_residual_norm_fp8");
    if (group != 0 && group != 128) return MLA_ERR_UNSUPPORTED;
    return mla::residual_norm(tokens, hidden, x, x_stride, residual, residual_stride, weight, rms_eps, nullptr, codes,
                              scales, group ? mla::kGroupScale : mla::kRowScale, residual_out, stream);
}
