// Rotary positions of queries or keys on their own (include/mla_chunk.h): the
// rotation of part of each head in either layout, and the rotary table of a model
// whose positions are scaled for long contexts.
//
//   y_a = m (x_a cos - x_b sin),  y_b = m (x_a sin + x_b cos)   for each pair (a, b), angle pos * rate
//
// A thread owns eight pairs of a token (16 values: one 32-byte run of the interleaved
// layout, two 16-byte runs of the half layout), works their angles out once and
// turns them in up to four heads, all eight loads in flight; a warp's share of a token is
// 128 / (dims / 16) heads (32 of 64 dims).
// Bound by memory: four bytes a value (4097 tokens of 128 x 64 values out of rows of 192: 23.7 us in a graph,
// 5.7 TB/s; 1 token 2.4 us, the launch and two dependent loads).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "mla_chunk.h"
#include "mla_internal.h"
#include "mla_rope.cuh"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

constexpr int kRotateWarps = 4;
constexpr int kRotateGrid = 152 * 16;   // CTAs at most (between 6 and 16 an SM: 4097 tokens within 4%)

struct RotateParams {
    const __nv_bfloat16 *x;
    __nv_bfloat16 *out;
    const int32_t *positions;
    const float *table;
    int64_t x_token, x_head, out_token, out_head;
    float magnitude, sign;
    int32_t tokens, heads, dims;
    int32_t parts;   // warps' shares of a token's heads
};

// Two bf16 values of one run against two of the other (the half layout's pairs).
__device__ __forceinline__ void turn_halves(uint32_t &a, uint32_t &b, const float (&s)[8], const float (&c)[8], int j) {
    const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&a));
    const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&b));
    a = pack_bf16x2(x.x * c[j] - y.x * s[j], x.y * c[j + 1] - y.y * s[j + 1]);
    b = pack_bf16x2(x.x * s[j] + y.x * c[j], x.y * s[j + 1] + y.y * c[j + 1]);
}

template <bool kHalf>
__global__ void __launch_bounds__(32 * kRotateWarps) mla_rotate_kernel(const RotateParams P) {
    const int lane = threadIdx.x & 31;
    const int per_head = P.dims / 16;          // threads of a head: a power of two
    const int sub = lane & (per_head - 1), first = lane / per_head, step = 32 / per_head;
    const int pairs = P.dims / 2;
    // in elements from the head's start: this thread's two runs of eight values
    const int run0 = kHalf ? sub * 8 : sub * 16, run1 = kHalf ? pairs + sub * 8 : run0 + 8;
    ptx::pdl_wait_prior();
    ptx::pdl_launch_dependents();
    const int64_t units = (int64_t)P.tokens * P.parts;
    for (int64_t u = (int64_t)blockIdx.x * kRotateWarps + (threadIdx.x >> 5); u < units;
         u += (int64_t)gridDim.x * kRotateWarps) {
        const int32_t tok = (int32_t)(u / P.parts), part = (int32_t)(u % P.parts);
        const int32_t pos = P.positions[tok];
        if (pos < 0) continue;
        const int h0 = (int)((int64_t)P.heads * part / P.parts), h1 = (int)((int64_t)P.heads * (part + 1) / P.parts);
        float s[8], c[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            rope_sincos(pos, P.table[sub * 8 + j], P.table[pairs + sub * 8 + j], s[j], c[j]);
            s[j] *= P.sign;
            c[j] *= P.magnitude;
        }
        const __nv_bfloat16 *src = P.x + tok * P.x_token;
        __nv_bfloat16 *dst = P.out + tok * P.out_token;
#pragma unroll 1
        for (int h = h0 + first; h < h1; h += 4 * step) {
            uint4 a[4], b[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (h + k * step < h1) {
                    const __nv_bfloat16 *at = src + (h + k * step) * P.x_head;
                    a[k] = *reinterpret_cast<const uint4 *>(at + run0);
                    b[k] = *reinterpret_cast<const uint4 *>(at + run1);
                }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (h + k * step < h1) {
                    if constexpr (kHalf) {
                        turn_halves(a[k].x, b[k].x, s, c, 0);
                        turn_halves(a[k].y, b[k].y, s, c, 2);
                        turn_halves(a[k].z, b[k].z, s, c, 4);
                        turn_halves(a[k].w, b[k].w, s, c, 6);
                    } else {
                        a[k] = make_uint4(turn2(a[k].x, s[0], c[0]), turn2(a[k].y, s[1], c[1]),
                                          turn2(a[k].z, s[2], c[2]), turn2(a[k].w, s[3], c[3]));
                        b[k] = make_uint4(turn2(b[k].x, s[4], c[4]), turn2(b[k].y, s[5], c[5]),
                                          turn2(b[k].z, s[6], c[6]), turn2(b[k].w, s[7], c[7]));
                    }
                    __nv_bfloat16 *at = dst + (h + k * step) * P.out_head;
                    *reinterpret_cast<uint4 *>(at + run0) = a[k];
                    *reinterpret_cast<uint4 *>(at + run1) = b[k];
                }
        }
    }
}

// Turns per position in fp64, as hi + lo floats (see mla_prolog.cu).
__global__ void __launch_bounds__(128) mla_rope_table_scaled_kernel(double base, int dims, double factor, double low,
                                                                    double high, float *table) {
    const int i = threadIdx.x;
    const double rate = pow(base, -(double)(2 * i) / dims);
    double w = (i - low) / (high - low);
    w = w < 0.0 ? 0.0 : w > 1.0 ? 1.0 : w;
    const double turns = (rate * (1.0 - w) + rate / factor * w) * 0.15915494309189535;
    const float hi = (float)turns;
    table[i] = hi;
    table[dims / 2 + i] = (float)(turns - (double)hi);
}

bool aligned(const void *p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool legal_dims(int32_t d) { return d == 16 || d == 32 || d == 64 || d == 128 || d == 256; }

}  // namespace
}  // namespace mla

extern "C" mla_status mla_rope_table_scaled(double rope_base, int32_t dims, double factor, int32_t original_positions,
                                            double beta_fast, double beta_slow, float *table, mla_stream_t stream) {
    if (!std::isfinite(rope_base) || !(rope_base > 1.0) || !mla::legal_dims(dims) || !std::isfinite(factor) ||
        !(factor >= 1.0) || original_positions < 1 || !std::isfinite(beta_fast) || !(beta_slow > 0.0) ||
        !(beta_fast >= beta_slow) || !mla::aligned(table, 4))
        return MLA_ERR_INVALID_ARG;
    auto pair_of = [&](double turns) {
        return dims * std::log(original_positions / (turns * 6.283185307179586)) / (2.0 * std::log(rope_base));
    };
    double low = std::floor(pair_of(beta_fast)), high = std::ceil(pair_of(beta_slow));
    low = low < 0.0 ? 0.0 : low;
    high = high > dims - 1.0 ? dims - 1.0 : high;
    if (high - low < 0.001) high = low + 0.001;
    mla::mla_rope_table_scaled_kernel<<<1, dims / 2, 0, reinterpret_cast<cudaStream_t>(stream)>>>(rope_base, dims, factor,
                                                                                               low, high, table);
    return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

extern "C" mla_status mla_rotate(int32_t tokens, int32_t heads, int32_t dims, const void *x, int64_t x_token_stride,
                                 int64_t x_head_stride, const int32_t *positions, const float *table, int32_t layout,
                                 int32_t inverse, float magnitude, void *out, int64_t out_token_stride,
                                 int64_t out_head_stride, mla_stream_t stream) {
    mla::NvtxRange nvtx_range("mla_rotate");
    using namespace mla;
    if (tokens < 1 || heads < 1 || (layout != MLA_LAYOUT_INTERLEAVED && layout != MLA_LAYOUT_HALF) ||
        (inverse != 0 && inverse != 1) || !std::isfinite(magnitude))
        return MLA_ERR_INVALID_ARG;
    if (!legal_dims(dims) || (int64_t)tokens * heads >= (int64_t)1 << 31) return MLA_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(positions, 4) || !aligned(table, 4)) return MLA_ERR_INVALID_ARG;
    for (const int64_t s : {x_token_stride, x_head_stride, out_token_stride, out_head_stride})
        if (s < 1 || s % 8 || s >= (int64_t)1 << 31) return MLA_ERR_INVALID_ARG;
    if (x == out && (x_token_stride != out_token_stride || x_head_stride != out_head_stride)) return MLA_ERR_INVALID_ARG;
    RotateParams p;
    p.x = static_cast<const __nv_bfloat16 *>(x);
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.positions = positions;
    p.table = table;
    p.x_token = x_token_stride;
    p.x_head = x_head_stride;
    p.out_token = out_token_stride;
    p.out_head = out_head_stride;
    p.magnitude = magnitude;
    p.sign = inverse ? -magnitude : magnitude;
    p.tokens = tokens;
    p.heads = heads;
    p.dims = dims;
    // A warp turns 32 / (dims / 16) heads at a time, four times per round: a share of a token's heads is one
    // round.
    const int share = 4 * 32 / (dims / 16);
    p.parts = (heads + share - 1) / share;
    const int64_t units = (int64_t)tokens * p.parts, ctas = (units + kRotateWarps - 1) / kRotateWarps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas < kRotateGrid ? ctas : kRotateGrid));
    cfg.blockDim = dim3(32 * kRotateWarps);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = layout == MLA_LAYOUT_HALF ? cudaLaunchKernelEx(&cfg, mla_rotate_kernel<true>, p)
                                                    : cudaLaunchKernelEx(&cfg, mla_rotate_kernel<false>, p);
    return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
