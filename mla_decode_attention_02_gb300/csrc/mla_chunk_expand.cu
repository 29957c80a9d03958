// The keys and values of a step's chunks (include/mla_chunk.h): every cached row
// that the chunks read, through W_UK and W_UV of a range of heads, into scratch.
//
//   K[h][j] = W_UK[h] r_j[0:512],  V[h][j] = W_UV[h] r_j[0:512]      512 -> 128 + 128
//
// Keys are rounded to bf16, the queries' type; values to fp16, which has three bits more (the product with the
// weights would be the larger part of the output's error: 700 keys 2.9e-3 of its norm with bf16 values and
// weights) and reaches 65504; the key of a value beyond that is NaN, so that it shows.
//
// A row's keys and values are worked out once, for all tokens that see them: 2 x
// 131072 flops a head and row.  Left to the attention kernel they would be worked
// out again for every tile of 256 tokens, more than doubling its products.
//
// GB300 design.  An SM pair holds 256 rows (four pages, 128 KB a CTA) as the A operand in
// shared memory and runs heads against them: tcgen05.mma of both SMs (cta_group::2,
// M = 256 rows, N = 256: the even CTA holds W_UK[h]'s half of B, the odd one W_UV[h]'s), so
// that each SM takes in 16 KB of weights per 512 clocks of MMA; one SM alone would have to take in 32 KB.
//   warp 0       this CTA's half of the weights: 64-value K blocks through a ring of six
//   warp 1       MMAs (even CTA): eight K blocks an item into one of two TMEM accumulators
//   warps 2-3    the rows: by TMA from the pages (bf16), or expanded from e4m3 codes (exact), whose
//                row scale multiplies the sums instead
//   warps 4-11   the previous item's epilogue: TMEM -> 16 bits -> the thread's row of scratch, 32 bytes (a whole
//                sector) a store; the first four take the keys, the others the values
// Pages are packed one behind the other over all requests, so no row of the MMAs is wasted but in the last
// pair's tile.  Rows past a request's end become zeros, so that a zero weight times them is zero; the
// key of a row that is not finite, or has a value beyond fp16, becomes NaN and its values zeros, so that it spoils
// what sees it and nothing else.
// Bound by its stores, 64 KB a row: 32768 rows (2.1 GB) in 651 us, 3.3 TB/s where a fill of as much memory takes
// 4.06, and 1.7 PFLOP/s; without the stores 510.  Staging in shared memory and a ring of four took 795; arrivals between
// the CTAs with release semantics, which wait for the stores, 1475.  No gain: TMA stores (836), clusters of two pairs that
// share the weights by multicast (835: 36 of them fit, 144 SMs), the rows in tensor memory with a ring of fourteen (658, and
// 700 rows 41 us instead of 27).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <mutex>

#include "mla_chunk.cuh"
#include "mla_fp8.h"
#include "mla_internal.h"
#include "mla_rope.cuh"
#include "sm103_ptx.cuh"

namespace mla {
bool encode_bf16_4d(CUtensorMap *m, const void *base, cuuint64_t d1, cuuint64_t d2, cuuint64_t d3,
                    cuuint64_t s1, cuuint64_t s2, cuuint64_t s3, cuuint32_t rows, cuuint32_t blocks);
cudaError_t main_units(int32_t *units);
namespace {
using namespace ptx;

constexpr int kKBlocks = kDl / 64;
constexpr int kStages = 6;
constexpr int kEpiWarps = 8;
constexpr int kExpandThreads = 32 * (4 + kEpiWarps);
constexpr uint32_t kBlk = 128 * 128;                   // 128 rows x 64 values
constexpr uint32_t kABytes = kKBlocks * kBlk;          // 128 KB
constexpr uint32_t kOffB = kABytes;
constexpr uint32_t kExpandSmem = kOffB + kStages * kBlk + 1024;
constexpr uint64_t kExpandWaitNs = 2000000000ull, kSettleNs = 1000000ull;
static_assert(kExpandSmem <= 232448 - 1024, "shared memory budget");
static_assert(kDn == 128 && kDv == 128, "a CTA's half of B is one weight matrix's 128 rows");

struct ExpandParams {
    CUtensorMap tm_rows;   // bf16 cache as (64 dims, 64 tokens, 9 dim blocks, pages), box 64 x 64 x 1 x 1
    CUtensorMap tm_uk;     // W_UK, W_UV as (64 values, 128 rows, 8 K blocks, heads), box 64 x 128 x 1 x 1
    CUtensorMap tm_uv;
    const uint8_t *cache;
    const int32_t *block_table;
    uint8_t *ws;
    __nv_bfloat16 *rope, *kv;
    int64_t num_pages, rows, kv_tokens;
    int32_t batch, tokens, max_pages;
    int32_t head0, heads;  // this pass's
};

struct Wait {
    volatile int *abort;
    int32_t *status;
};

// Bounded wait; on time-out flags the CTA (every other wait then gives up at once).  What the other CTA of the
// pair completes carries data in one case only, the expanded rows, which is waited for at cluster scope.
template <bool kCluster>
__device__ __noinline__ bool wait_slow(const Wait w, uint32_t bar, uint32_t parity) {
    uint64_t t0 = 0;
    for (uint32_t i = 0;; ++i) {
        if (kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
        if ((i & 63) == 63) {
            if (*w.abort) return false;
            const uint64_t t = globaltimer_ns();
            if (t0 == 0) t0 = t;
            else if (t - t0 > kExpandWaitNs) {
                *w.abort = 1;
                atomicOr(w.status, MLA_DEV_TIMEOUT);
                return false;
            }
        }
    }
}

__device__ __forceinline__ bool expand_wait(const Wait &w, uint32_t bar, uint32_t parity) {
    return mbar_try_wait(bar, parity) || wait_slow<false>(w, bar, parity);
}

// Two e4m3 codes -> two bf16 values (exact).
__device__ __forceinline__ uint32_t codes2(uint32_t codes) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xFFFFu), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    return pack_bf16x2(f.x, f.y);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ void st_shared_v4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Maxima of two pairs (NaN if either is).
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Stores whose lines leave L2 before others: the scratch is larger than L2 in the cases that take long, and
// would drive out the weights that every group of rows reads again.
__device__ __forceinline__ uint64_t l2_evict_first() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

__device__ __forceinline__ void st_global_first(void *at, const uint32_t *x, uint64_t policy) {
    asm volatile("st.global.L2::cache_hint.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8}, %9;" ::"l"(at), "r"(x[0]),
                 "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "l"(policy)
                 : "memory");
}

// A warp's share of the items: 32 accumulator rows (lane: one row), the keys' 128 columns (kPart 0) or the
// values' (1).  The accumulator is given back as soon as it is in registers, rounded; what is not an ordinary
// row (a value not finite or beyond fp16) is mended there, in a branch that no other takes.
template <bool kFp8, int kPart>
__device__ __forceinline__ void epilogue(const ExpandParams &P, const Wait &w, const ChunkPage *pages, int32_t num_pages,
                                         int64_t i0, int64_t i1, uint32_t rank, int row, uint32_t acc, uint32_t b_acc,
                                         uint32_t b_free, uint32_t b_bad, uint8_t *bad) {
    const int lane = row & 31;
    bool there = false, spoilt = false;
    float s_row = 1.f;
    const uint64_t policy = l2_evict_first();
    int32_t group = (int32_t)(i0 / P.heads), hl = (int32_t)(i0 % P.heads);
    bool fresh = true;
    for (uint32_t k = 0; k < (uint32_t)(i1 - i0); ++k) {
        const uint32_t buf = k & 1;
        const int64_t row0 = (int64_t)group * kPairRows + rank * 128 + (row - lane);   // the warp's first scratch row
        if (fresh) {
            fresh = false;
            const int32_t p = group * 4 + (int32_t)rank * 2 + (row >> 6), r = row & 63;
            there = spoilt = false;
            s_row = 1.f;
            int32_t page = -1;
            if (p < num_pages) {
                const ChunkPage e = pages[p];
                page = P.block_table[e.entry];
                there = r < e.valid;
                spoilt = there && (page < 0 || page >= P.num_pages);
                if (spoilt) atomicOr(w.status, MLA_DEV_BAD_PAGE);
            }
            const bool read = there && !spoilt;
            const uint8_t *src = P.cache + ((size_t)(read ? page : 0) * kPage + r) * (kFp8 ? MLA_FP8_ROW_BYTES : 2 * kDrow);
            if (kFp8 && read) s_row = *reinterpret_cast<const float *>(src + kDl + 2 * kDr);
            if (kPart == 0 && P.head0 == 0 && hl == 0) {   // the rotary part, once for all heads
                uint4 v[kDr / 8];
#pragma unroll
                for (int q = 0; q < kDr / 8; ++q)
                    v[q] = read ? reinterpret_cast<const uint4 *>(src + (kFp8 ? kDl : 2 * kDl))[q] : make_uint4(0, 0, 0, 0);
                uint4 *dst = reinterpret_cast<uint4 *>(P.rope + (row0 + lane) * kDr);
#pragma unroll
                for (int q = 0; q < kDr / 8; ++q) {
                    if constexpr (kFp8) {
                        uint32_t *x = reinterpret_cast<uint32_t *>(&v[q]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&x[e]));
                            x[e] = pack_bf16x2(f.x * s_row, f.y * s_row);
                        }
                    }
                    dst[q] = v[q];
                }
            }
        }
        if (!__all_sync(0xffffffffu, expand_wait(w, b_acc + 8 * buf, (k / 2) & 1))) break;
        tc_fence_after();
        uint32_t x[64];
        bool odd = !there || spoilt;   // a row that is no ordinary one, or holds a value that is not finite
        uint32_t top[2] = {0, 0};   // the largest magnitudes, NaN above all
        constexpr int kAt = 2;   // pieces of 32 columns at a time
#pragma unroll
        for (int c = 0; c < 4; c += kAt) {
            uint32_t r[kAt][32];
#pragma unroll
            for (int d = 0; d < kAt; ++d) tmem_ld32(acc + buf * 256 + (c + d) * 32, r[d]);
#pragma unroll
            for (int d = 0; d < kAt; ++d) tmem_wait_ld(r[d]);
#pragma unroll
            for (int d = 0; d < kAt; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float a = __uint_as_float(r[d][2 * e]), b = __uint_as_float(r[d][2 * e + 1]);
                    if constexpr (kFp8) {
                        a *= s_row;
                        b *= s_row;
                    }
                    const uint32_t v = kPart == 0 ? pack_bf16x2(a, b) : pack_f16x2(a, b);
                    x[(c + d) * 16 + e] = v;
                    top[e & 1] = kPart == 0 ? max_bf16x2(top[e & 1], v & 0x7fff7fffu) : max_f16x2(top[e & 1], v & 0x7fff7fffu);
                }
        }
        constexpr uint32_t kInf = kPart == 0 ? 0x7f80u : 0x7c00u;
        top[0] = kPart == 0 ? max_bf16x2(top[0], top[1]) : max_f16x2(top[0], top[1]);
        odd |= (top[0] & 0xffffu) >= kInf || (top[0] >> 16) >= kInf;
        // The values' warp tells the keys' warp of the same rows.  (That one gives the accumulator back after it has
        // read this, so the flags are not written again before.)
        uint8_t *flag = &bad[buf * 128 + row];
        const uint32_t b_told = b_bad + 8 * (2 * (row >> 5) + buf);
        if constexpr (kPart == 1) {
            *flag = odd;
            __syncwarp();
            if (lane == 0) mbar_arrive(b_told);
        } else {
            if (!__all_sync(0xffffffffu, expand_wait(w, b_told, (k / 2) & 1))) break;
            odd |= *flag != 0;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_signal_cluster(b_free + 8 * buf);
        if (__any_sync(0xffffffffu, odd) && odd) {
            // a row that is not there: zeros; else the key is NaN, and the values are numbers
            const uint32_t fill = kPart == 0 && there ? 0x7fff7fffu : 0u;
#pragma unroll
            for (int e = 0; e < 64; ++e) x[e] = fill;
        }
        // a row's 256 bytes as eight whole sectors
        __nv_bfloat16 *out = P.kv + ((size_t)hl * P.rows + row0 + lane) * (kDn + kDv) + kPart * 128;
#pragma unroll
        for (int q = 0; q < 8; ++q) st_global_first(out + q * 16, &x[q * 8], policy);
        if (++hl == P.heads) {
            hl = 0;
            ++group;
            fresh = true;
        }
    }
}

template <bool kFp8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kExpandThreads, 1)
mla_chunk_expand_kernel(const __grid_constant__ ExpandParams P) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 15];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ uint8_t s_bad[2 * 128];   // by item parity: rows whose values are out of range
    const uint32_t s_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    // full, rows landed and accumulator free are the even CTA's (both CTAs arrive there); the others are
    // each CTA's own, which the MMAs' commits reach in both
    enum { B_FULL = 0, B_EMPTY = kStages, B_AFULL = 2 * kStages, B_AFREE, B_ACC, B_ACCFREE = B_ACC + 2,
           B_BAD = B_ACCFREE + 2, B_DRAIN = B_BAD + 8 };
    static_assert(B_DRAIN + 1 == 2 * kStages + 15, "barriers");
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    auto even = [&](int i) { return mapa(smem_u32(&bars[i]), 0); };
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar(B_FULL + s), 2);
            mbar_init(bar(B_EMPTY + s), 1);
        }
        mbar_init(bar(B_AFULL), kFp8 ? 4 : 2);
        mbar_init(bar(B_AFREE), 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(B_ACC + b), 1);
            mbar_init(bar(B_ACCFREE + b), 2 * kEpiWarps);
        }
        for (int b = 0; b < 8; ++b) mbar_init(bar(B_BAD + b), 1);
        mbar_init(bar(B_DRAIN), 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc_pair(smem_u32(&tmem_slot), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // the pair's barriers are set up
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait_prior();
    pdl_launch_dependents();

    PlanHeader *hdr = reinterpret_cast<PlanHeader *>(P.ws);
    const Wait w = {&abort_flag, &hdr->status};
    const bool fits = hdr->magic == kChunkMagic && hdr->batch == P.batch && hdr->s_q == P.tokens &&
                      hdr->max_pages == P.max_pages && hdr->total_cost == P.kv_tokens;   // (else flagged by the attention)
    const int32_t num_pages = fits ? hdr->num_parts : 0;
    if (fits && blockIdx.x == 0 && threadIdx.x == 0) hdr->target = 0;   // the attention's items taken so far
    const ChunkPage *pages =
        reinterpret_cast<const ChunkPage *>(P.ws + chunk_layout(P.batch, P.tokens, P.kv_tokens).pages);
    // An item is one head of four pages (of which the last may be the page of zeros).  Each pair takes a contiguous run,
    // so that it loads rows a few times only.
    const int32_t groups = num_pages > 0 ? num_pages / 4 + 1 : 0;
    const int64_t items = (int64_t)groups * P.heads, pairs = gridDim.x / 2, c = blockIdx.x / 2;
    const int64_t i0 = items * c / pairs, i1 = items * (c + 1) / pairs;

    if (warp == 0) {
        if (elect_one()) {
            const CUtensorMap *tm = rank == 0 ? &P.tm_uk : &P.tm_uv;
            prefetch_tmap(tm);
            uint32_t n = 0;
            bool ok = true;
            int hl = (int)(i0 % P.heads);
            for (int64_t i = i0; i < i1 && ok; ++i, hl = hl + 1 == P.heads ? 0 : hl + 1) {
                const int h = P.head0 + hl;
                for (int kb = 0; kb < kKBlocks; ++kb, ++n) {
                    const uint32_t s = n % kStages;
                    if (n >= kStages && !expand_wait(w, bar(B_EMPTY + s), (n / kStages - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    mbar_expect_tx_cluster(even(B_FULL + s), kBlk);
                    tma_load_4d_pair(s_base + kOffB + s * kBlk, tm, 0, 0, kb, h, even(B_FULL + s));
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            constexpr uint32_t idesc = idesc_bf16(256, 256, 0, 0);
            uint32_t n = 0, loads = 0;
            int hl = (int)(i0 % P.heads);
            bool ok = true;
            for (int64_t i = i0; i < i1 && ok; ++i, hl = hl + 1 == P.heads ? 0 : hl + 1) {
                const uint32_t k = (uint32_t)(i - i0), buf = k & 1;
                if (i == i0 || hl == 0) ok = wait_slow<kFp8>(w, bar(B_AFULL), loads++ & 1);
                if (k >= 2) ok = ok && expand_wait(w, bar(B_ACCFREE + buf), (k / 2 - 1) & 1);
                for (int kb = 0; kb < kKBlocks && ok; ++kb, ++n) {
                    const uint32_t s = n % kStages;
                    ok = expand_wait(w, bar(B_FULL + s), (n / kStages) & 1);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_ss_pair(tmem + buf * 256, smem_desc(s_base + kb * kBlk + ks * 32, 16, 1024, 2),
                                    smem_desc(s_base + kOffB + s * kBlk + ks * 32, 16, 1024, 2), idesc,
                                    (kb | ks) ? 1u : 0u);
                    mma_commit_pair(bar(B_EMPTY + s));
                }
                if (!ok) break;
                mma_commit_pair(bar(B_ACC + buf));
                if (i + 1 == i1 || hl + 1 == P.heads) mma_commit_pair(bar(B_AFREE));
            }
            // every MMA is done before the CTAs give their memory up
            mma_commit_pair(bar(B_DRAIN));
        }
        __syncwarp();
    } else if (warp < 4) {
        // ---- the rows of each group of pages
        uint32_t loads = 0;
        for (int64_t i = i0; i < i1; i = (i / P.heads + 1) * P.heads, ++loads) {
            if (loads > 0 && !__all_sync(0xffffffffu, expand_wait(w, bar(B_AFREE), (loads - 1) & 1))) break;
            const int32_t p0 = (int32_t)(i / P.heads) * 4 + (int32_t)rank * 2;
            int32_t page[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                page[q] = p0 + q < num_pages ? P.block_table[pages[p0 + q].entry] : -1;
                if (page[q] >= P.num_pages) page[q] = -1;
            }
            if constexpr (!kFp8) {
                if (warp == 2 && elect_one()) {
                    const uint32_t there = (page[0] >= 0) + (page[1] >= 0);
                    mbar_expect_tx_cluster(even(B_AFULL), there * (kABytes / 2));
                    for (int kb = 0; kb < kKBlocks; ++kb)
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            if (page[q] >= 0)
                                tma_load_4d_pair(s_base + kb * kBlk + q * (kBlk / 2), &P.tm_rows, 0, 0, kb, page[q],
                                                 even(B_AFULL));
                }
                __syncwarp();
            } else {
                // a row a warp at a time: lane l expands codes 16 l .. 16 l + 15
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (page[q] < 0) continue;
                    const uint8_t *src = P.cache + (size_t)page[q] * kPage * MLA_FP8_ROW_BYTES;
#pragma unroll 8
                    for (int r = warp - 2; r < kPage; r += 2) {
                        const uint4 v = reinterpret_cast<const uint4 *>(src + r * MLA_FP8_ROW_BYTES)[lane];
                        const uint32_t at = s_base + (lane >> 2) * kBlk + (q * kPage + r) * 128;
                        const uint32_t u = (lane & 3) * 2, x = r & 7;
                        st_shared_v4(at + ((u ^ x) << 4), codes2(v.x), codes2(v.x >> 16), codes2(v.y), codes2(v.y >> 16));
                        st_shared_v4(at + (((u + 1) ^ x) << 4), codes2(v.z), codes2(v.z >> 16), codes2(v.w),
                                     codes2(v.w >> 16));
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(even(B_AFULL));
            }
        }
    } else {
        // ---- accumulator rows [32 quarter, +32), the keys' or the values' 128 columns
        const int quarter = warp & 3, row = quarter * 32 + lane;
        if (warp < 8)
            epilogue<kFp8, 0>(P, w, pages, num_pages, i0, i1, rank, row, tmem + ((uint32_t)(quarter * 32) << 16), bar(B_ACC),
                              even(B_ACCFREE), bar(B_BAD), s_bad);
        else
            epilogue<kFp8, 1>(P, w, pages, num_pages, i0, i1, rank, row, tmem + ((uint32_t)(quarter * 32) << 16) + 128,
                              bar(B_ACC), even(B_ACCFREE), bar(B_BAD), s_bad);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        expand_wait(w, bar(B_DRAIN), 0);
        if (abort_flag) {   // copies may be in flight: they land within microseconds
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < kSettleNs) {
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // the other CTA reads nothing of this one's any more
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

std::mutex g_expand_mutex;
bool g_expand_attr[64];

}  // namespace

// head0 .. head0 + heads - 1 of every page of the plan in ws, into kv (and the rotary parts into rope, with head 0).
cudaError_t launch_chunk_expand(const mla_chunk *prob, const void *w_uk, const void *w_uv, const void *cache, bool fp8,
                                int64_t num_pages, const int32_t *block_table, void *ws, void *rope, void *kv,
                                int32_t head0, int32_t heads, cudaStream_t stream) {
    int dev = 0;
    int32_t units = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if ((e = main_units(&units)) != cudaSuccess) return e;
    auto *kernel = fp8 ? mla_chunk_expand_kernel<true> : mla_chunk_expand_kernel<false>;
    {
        std::lock_guard<std::mutex> lock(g_expand_mutex);
        if (!g_expand_attr[dev]) {
            for (auto *k : {mla_chunk_expand_kernel<true>, mla_chunk_expand_kernel<false>})
                if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kExpandSmem)) !=
                    cudaSuccess)
                    return e;
            g_expand_attr[dev] = true;
        }
    }
    ExpandParams p{};
    if ((!fp8 && !encode_bf16_4d(&p.tm_rows, cache, kPage, kDrow / 64, (cuuint64_t)num_pages, kDrow * 2, 128,
                                 (cuuint64_t)kPage * kDrow * 2, kPage, 1)) ||
        !encode_bf16_4d(&p.tm_uk, w_uk, kDn, kKBlocks, kHeads, kDl * 2, 128, (cuuint64_t)kDn * kDl * 2, kDn, 1) ||
        !encode_bf16_4d(&p.tm_uv, w_uv, kDv, kKBlocks, kHeads, kDl * 2, 128, (cuuint64_t)kDv * kDl * 2, kDv, 1))
        return cudaErrorInvalidValue;
    p.cache = static_cast<const uint8_t *>(cache);
    p.block_table = block_table;
    p.ws = static_cast<uint8_t *>(ws);
    p.rope = static_cast<__nv_bfloat16 *>(rope);
    p.kv = static_cast<__nv_bfloat16 *>(kv);
    p.num_pages = num_pages;
    p.rows = chunk_rows(prob->kv_tokens);
    p.kv_tokens = prob->kv_tokens;
    p.batch = prob->batch;
    p.tokens = prob->tokens;
    p.max_pages = prob->max_pages_per_seq;
    p.head0 = head0;
    p.heads = heads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * units));   // an SM pair per unit
    cfg.blockDim = dim3(kExpandThreads);
    cfg.dynamicSmemBytes = kExpandSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace mla
