// The rotary embedding shared by the prolog, query and append kernels: angles
// of far positions in fp32 double-float arithmetic (see mla_prolog.cu for the
// error bound) and the rotation of bf16 pairs.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "mla_internal.h"

namespace mla {

constexpr int kPairs = kDr / 2;           // RoPE pairs per 64-dim vector

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}

// sin and cos of the angle pos * 2 pi (g_hi + g_lo), 0 <= pos < 2^31 (see the notes in mla_prolog.cu).
__device__ __forceinline__ void rope_sincos(int32_t pos, float g_hi, float g_lo, float &s, float &c) {
    const float ph = (float)(pos >> 16), pl = (float)(pos & 0xffff);   // both exact
    const float gh16 = g_hi * 65536.f, gl16 = g_lo * 65536.f;          // exact scalings
    const float a1 = ph * gh16, e1 = fmaf(ph, gh16, -a1);             // ph * gh16 = a1 + e1 exactly
    const float a2 = pl * g_hi, e2 = fmaf(pl, g_hi, -a2);
    float r = (a1 - rintf(a1)) + (a2 - rintf(a2));                      // fractions of the big terms
    r += e1 + e2 + fmaf(ph, gl16, pl * g_lo);
    r -= rintf(r);
    __sincosf(r * 6.28318530717958648f, &s, &c);
}

// Rotate a pair of bf16 values by the angle of this sine and cosine.
__device__ __forceinline__ uint32_t turn2(uint32_t v, float s, float c) {
    const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v));
    return pack_bf16x2(x.x * c - x.y * s, x.x * s + x.y * c);
}

// Rotate the four pairs held by eight consecutive bf16 values by angles given as sines and cosines.
__device__ __forceinline__ uint4 turn8(uint4 v, const float (&s)[4], const float (&c)[4]) {
    return make_uint4(turn2(v.x, s[0], c[0]), turn2(v.y, s[1], c[1]), turn2(v.z, s[2], c[2]), turn2(v.w, s[3], c[3]));
}

// Rotate the four pairs held by eight consecutive bf16 values, pairs p0 .. p0 + 3.
__device__ __forceinline__ uint4 rope8(uint4 v, int32_t pos, int p0, const float *g_hi,
                                       const float *g_lo) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float s, c;
        rope_sincos(pos, g_hi[p0 + j], g_lo[p0 + j], s, c);
        w[j] = turn2(w[j], s, c);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace mla
