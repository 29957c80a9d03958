// Absorbed and rotated queries of many tokens (include/mla_tree.h, mla_query):
//
//   q_latent[t][h] = q_nope[t][h] . W_UK[h]  (128 -> 512),   q_rope[t][h] = RoPE(q_pe[t][h], positions[t])
//
// A persistent kernel for more than a few token tiles.  An item is one 128-token
// tile of one head and one half (256) of the latent columns; each CTA (one per
// SM) runs the tiles of one head-half after another, so W_UK's half (64 KB)
// stays in shared memory over them while the next one loads beside it (with one
// buffer 129 tokens took 11.5 us instead of 10.5, 512 24.8 instead of 21.6).  Per item the tile's q_nope
// (32 KB, two stages) comes by TMA, eight tcgen05.mma (M=128, N=256, K=16) fill one
// of two TMEM accumulators, and the epilogue of the previous item runs meanwhile:
//   warp 0      loads and MMAs (one elected lane)
//   warps 1-8   TMEM -> bf16 -> the warp's own 4 KB of swizzled staging -> 128-byte row pieces
//   warps 9-12  q_pe, apart from the items: whole tokens, a quarter of the heads at a time
// Bound by memory: 384 bytes in and 1152 out per token and head (the outputs are
// three quarters), against 2 x 128 x 512 flops: 1537 tokens in 59.6 us, 5.4 TB/s.  q_pe by
// items (each CTA its head's share, angles anew for every head) had cost ten us more in an earlier form
// (79.8 against 69.5).  The small-tile kernel of mla_prolog.cu
// (one CTA per item of a quarter) does few tokens in one wave; from a few tiles on its
// CTAs spend their time on latency: each loads, multiplies and stores once.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <mutex>

#include "mla_internal.h"
#include "mla_prolog.h"
#include "mla_rope.cuh"
#include "mla_tree.h"
#include "sm103_ptx.cuh"

namespace mla {
bool encode_bf16_4d(CUtensorMap *m, const void *base, cuuint64_t d1, cuuint64_t d2, cuuint64_t d3,
                    cuuint64_t s1, cuuint64_t s2, cuuint64_t s3, cuuint32_t rows, cuuint32_t blocks);
cudaError_t main_units(int32_t *units);
mla_status launch_query_small(int32_t tokens, const void *q_nope, int64_t nope_token_stride, int64_t nope_head_stride,
                              const void *q_pe, int64_t pe_token_stride, int64_t pe_head_stride, const void *w_uk,
                              const float *rope_table, const int32_t *positions, void *q_latent, void *q_rope,
                              int32_t *device_status, mla_stream_t stream);
namespace {
using namespace ptx;

constexpr int kTile = 128;                      // tokens per item (MMA M)
constexpr int kCols = 256;                      // latent columns per item (MMA N)
constexpr int kHalves = kDl / kCols;
constexpr int kDimN = MLA_D_NOPE;               // 128: the contraction, eight K=16 steps
constexpr int kEpiWarps = 8, kRopeWarps = 4;
constexpr int kQueryThreads = 32 * (1 + kEpiWarps + kRopeWarps);
constexpr uint32_t kWBlk = kDimN * 128;         // one 64-column block of W_UK: 128 rows x 128 B
constexpr uint32_t kWBytes = kCols / 64 * kWBlk;        // 64 KB
constexpr uint32_t kABlk = kTile * 128;         // one 64-dim block of q_nope
constexpr uint32_t kABytes = kDimN / 64 * kABlk;        // 32 KB
constexpr uint32_t kStageBytes = 32 * 128;      // a warp's staging: 32 rows x 64 columns
constexpr uint32_t kOffA = 2 * kWBytes, kOffStage = kOffA + 2 * kABytes;
constexpr uint32_t kQuerySmem = kOffStage + kEpiWarps * kStageBytes + 1024;
constexpr uint64_t kQueryWaitNs = 2000000000ull;
static_assert(kQuerySmem <= 232448 - 1024, "shared memory budget");

struct QueryParams {
    CUtensorMap tm_a;    // q_nope as (64 dims, tokens, 2 dim blocks, heads), box 64 x 128 x 2 x 1
    CUtensorMap tm_w;    // W_UK as (64 columns, 128 dims, 8 column blocks, heads), box 64 x 128 x 4 x 1
    const __nv_bfloat16 *q_pe;
    const float *rope_table;
    const int32_t *positions;
    __nv_bfloat16 *q_latent, *q_rope;
    int32_t *status;
    int64_t pe_token, pe_head;
    int32_t tokens, tiles;
    TreePlanRef plan;    // of a mixed step: only tiles with a row in it (a position that is not negative)
};

constexpr int kMaxPlanTiles = 128;   // (a tree schedule's planner takes some 10,000 rows)

// Bounded wait; on time-out flags the CTA (every other wait then gives up at once).
__device__ __noinline__ bool query_wait(uint32_t bar, uint32_t parity, volatile int *abort, int32_t *status) {
    uint64_t t0 = 0;
    for (uint32_t i = 0;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63) == 63) {
            if (*abort) return false;
            const uint64_t t = globaltimer_ns();
            if (t0 == 0) t0 = t;
            else if (t - t0 > kQueryWaitNs) {
                *abort = 1;
                atomicOr(status, MLA_DEV_TIMEOUT);
                return false;
            }
        }
    }
}

// Teardown: what is in flight lands, whatever the abort flag says (bounded).
__device__ __noinline__ void query_landed(uint32_t bar, uint32_t parity, int32_t *status) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (globaltimer_ns() - t0 > kQueryWaitNs) {
            atomicOr(status, MLA_DEV_TIMEOUT);
            return;
        }
    }
}

// kSparse: of a mixed step over chunks (P.plan).
template <bool kSparse>
__global__ void __launch_bounds__(kQueryThreads, 1) mla_query_kernel(const __grid_constant__ QueryParams P) {
    if constexpr (kSparse) {
        pdl_wait_prior();   // (what follows starts only once this kernel's CTAs have their tensor memory, or are gone)
        if (tree_plan_idle(P.plan)) return;
    }
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[11];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag, live_tiles;
    __shared__ uint8_t live[kSparse ? kMaxPlanTiles : 1];
    const uint32_t s_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    // barriers (two each): A landed, A read by the MMAs, accumulator full, accumulator read, W landed; then drain
    enum { B_AFULL = 0, B_AFREE = 2, B_CFULL = 4, B_CFREE = 6, B_W = 8, B_DRAIN = 10 };
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(B_AFULL + b), 1);
            mbar_init(bar(B_AFREE + b), 1);
            mbar_init(bar(B_CFULL + b), 1);
            mbar_init(bar(B_CFREE + b), kEpiWarps);
            mbar_init(bar(B_W + b), 1);
        }
        mbar_init(bar(B_DRAIN), 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(&tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait_prior();
    pdl_launch_dependents();

    int tiles = P.tiles;
    if constexpr (kSparse) {
        const bool any = tree_plan_there(P.plan);
        for (int t = warp; t < P.tiles; t += kQueryThreads / 32) {
            bool has = false;
            if (any)
                for (int r = t * kTile + lane; r < (t + 1) * kTile && r < P.tokens; r += 32) has |= P.positions[r] >= 0;
            has = __any_sync(0xffffffffu, has);
            if (lane == 0) live[t] = has;
        }
        __syncthreads();
        if (threadIdx.x == 0) {   // the tiles with rows, in order
            int n = 0;
            for (int t = 0; t < P.tiles; ++t)
                if (live[t]) live[n++] = (uint8_t)t;
            live_tiles = n;
        }
        __syncthreads();
        tiles = live_tiles;
    }

    // Items: CTA c takes head-half c over all tiles, so that the CTAs move along the tokens together
    // and write neighbouring rows at the same time (1537 tokens: 59.4 us against 67.0 with one contiguous
    // run of (head, half, tile) per CTA), then a share of the other head-halves' items.
    const int64_t rest = ((int64_t)kHeads * kHalves - gridDim.x) * tiles;
    const int64_t r0 = rest * blockIdx.x / gridDim.x - tiles;
    const int n = (int)(rest * (blockIdx.x + 1) / gridDim.x - r0);
    auto head_half = [&](int i) { return i < tiles ? (int)blockIdx.x : (int)(gridDim.x + (r0 + i) / tiles); };
    auto place_of = [&](int i) { return i < tiles ? i : (int)((r0 + i) % tiles); };
    auto tile_of = [&](int i) { return kSparse ? (int)live[place_of(i)] : place_of(i); };

    if (warp == 0) {
        if (elect_one()) {
            prefetch_tmap(&P.tm_a);
            prefetch_tmap(&P.tm_w);
            constexpr uint32_t idesc = idesc_bf16(kTile, kCols, 0, 1);
            // W_UK's halves in the order of the items: each is loaded when the one before it comes
            // into use, and the MMAs that read the one before that are done
            int w_loads = 0, w_used = 0;
            auto load_w = [&](int i) {   // the half of item i
                const int hh = head_half(i);
                const uint32_t full = bar(B_W + (w_loads & 1));
                mbar_arrive_expect_tx(full, kWBytes);
                tma_load_4d(s_base + (w_loads & 1) * kWBytes, &P.tm_w, 0, 0, hh % kHalves * (kCols / 64), hh / kHalves,
                            full);
                ++w_loads;
            };
            int loaded = 0, next_w = 0;   // next_w: the first item of the next half
            bool ok = true;
            auto load_a = [&](int i) {
                const uint32_t full = bar(B_AFULL + (i & 1));
                mbar_arrive_expect_tx(full, kABytes);
                tma_load_4d(s_base + kOffA + (i & 1) * kABytes, &P.tm_a, 0, tile_of(i) * kTile, 0,
                            head_half(i) / kHalves, full);
                loaded = i + 1;
            };
            if (n > 0) {
                load_w(0);
                load_a(0);
            }
            for (int i = 0; i < n && ok; ++i) {
                // the next item's tile, once the MMAs of the item before this one have read its stage
                if (i >= 1) ok = query_wait(bar(B_AFREE + ((i - 1) & 1)), ((i - 1) >> 1) & 1, &abort_flag, P.status);
                if (!ok) break;
                if (i + 1 < n) load_a(i + 1);
                if (i == next_w) {   // (every MMA of the items before is done: waited above)
                    next_w = i + tiles - place_of(i);
                    if (next_w < n) load_w(next_w);
                    ok = query_wait(bar(B_W + (w_used & 1)), (w_used >> 1) & 1, &abort_flag, P.status);
                    ++w_used;
                }
                const uint32_t s_w = s_base + ((w_used - 1) & 1) * kWBytes;
                ok = ok && query_wait(bar(B_AFULL + (i & 1)), (i >> 1) & 1, &abort_flag, P.status) &&
                     (i < 2 || query_wait(bar(B_CFREE + (i & 1)), ((i >> 1) - 1) & 1, &abort_flag, P.status));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < kDimN / 16; ++ks)
                    mma_ss(tmem + (i & 1) * kCols,
                           smem_desc(s_base + kOffA + (i & 1) * kABytes + (ks / 4) * kABlk + (ks % 4) * 32, 16, 1024, 2),
                           smem_desc(s_w + ks * 2048, kWBlk, 1024, 2), idesc, ks > 0 ? 1u : 0u);
                mma_commit(bar(B_AFREE + (i & 1)));
                mma_commit(bar(B_CFULL + (i & 1)));
            }
            // every copy has landed and every MMA is done before the CTA gives its memory up
            for (int i = loaded > 2 ? loaded - 2 : 0; i < loaded; ++i)
                query_landed(bar(B_AFULL + (i & 1)), (i >> 1) & 1, P.status);
            for (int w = w_loads > 2 ? w_loads - 2 : 0; w < w_loads; ++w)
                query_landed(bar(B_W + (w & 1)), (w >> 1) & 1, P.status);
            mma_commit(bar(B_DRAIN));
            query_landed(bar(B_DRAIN), 0, P.status);
        }
        __syncwarp();
    } else if (warp <= kEpiWarps) {
        // ---- accumulator rows [32 quarter, +32), columns [128 part, +128) of the item's half
        const int quarter = warp & 3, part = (warp - 1) >> 2;
        const uint32_t stage = s_base + kOffStage + (warp - 1) * kStageBytes;
        const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16) + part * 128;
        for (int i = 0; i < n; ++i) {
            const int hh = head_half(i), tok0 = tile_of(i) * kTile + quarter * 32;
            const int32_t pos = tok0 + lane < P.tokens ? P.positions[tok0 + lane] : -1;
            const unsigned wanted = __ballot_sync(0xffffffffu, pos >= 0);
            if (!__all_sync(0xffffffffu, query_wait(bar(B_CFULL + (i & 1)), (i >> 1) & 1, &abort_flag, P.status))) break;
            tc_fence_after();
            const int j = lane & 7;
            __nv_bfloat16 *out = P.q_latent + ((size_t)tok0 * kHeads + hh / kHalves) * kDl + hh % kHalves * kCols +
                                 part * 128 + j * 8;
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {   // 64 columns at a time
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    uint32_t r[32];
                    tmem_ld32(acc + (i & 1) * kCols + c * 64 + d * 32, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t at = stage + lane * 128 + (((d * 4 + q) ^ (lane & 7)) << 4);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at),
                                     "r"(pack_bf16x2(__uint_as_float(r[8 * q]), __uint_as_float(r[8 * q + 1]))),
                                     "r"(pack_bf16x2(__uint_as_float(r[8 * q + 2]), __uint_as_float(r[8 * q + 3]))),
                                     "r"(pack_bf16x2(__uint_as_float(r[8 * q + 4]), __uint_as_float(r[8 * q + 5]))),
                                     "r"(pack_bf16x2(__uint_as_float(r[8 * q + 6]), __uint_as_float(r[8 * q + 7])))
                                     : "memory");
                    }
                }
                if (c == 1) tc_fence_before();
                __syncwarp();
                if (c == 1 && lane == 0) mbar_arrive(bar(B_CFREE + (i & 1)));
#pragma unroll
                for (int k = 0; k < 8; ++k) {   // four rows' 128 bytes at a time
                    const int row = 4 * k + (lane >> 3);
                    uint4 v;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                 : "r"(stage + row * 128 + ((j ^ (row & 7)) << 4))
                                 : "memory");
                    if (wanted >> row & 1) *reinterpret_cast<uint4 *>(out + c * 64 + (size_t)row * kHeads * kDl) = v;
                }
                __syncwarp();   // the staging is read before the next rows go in
            }
        }
    } else {
        // ---- q_pe: a unit is a token's 32 heads [32 (u % 4), +32), a warp's units a contiguous run.
        // Lane l rotates dims [8 (l % 8), +8) of four heads at a time, with the token's four angles
        // in registers: they are worked out once for 32 heads.
        const int pair0 = (lane & 7) * 4;
        float gh[4], gl[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            gh[j] = P.rope_table[pair0 + j];
            gl[j] = P.rope_table[kPairs + pair0 + j];
        }
        const int64_t units = (kSparse ? (int64_t)tiles * kTile : (int64_t)P.tokens) * 4;
        const int64_t warps = (int64_t)gridDim.x * kRopeWarps;
        const int64_t w = (int64_t)blockIdx.x * kRopeWarps + warp - 1 - kEpiWarps;
        for (int64_t u = units * w / warps, end = units * (w + 1) / warps; u < end; ++u) {
            int tok = (int)(u >> 2);
            const int h0 = (int)(u & 3) * 32 + (lane >> 3);
            if constexpr (kSparse) {
                tok = live[tok / kTile] * kTile + tok % kTile;
                if (tok >= P.tokens || P.positions[tok] < 0) continue;
            }
            const __nv_bfloat16 *src = P.q_pe + tok * P.pe_token + h0 * P.pe_head + pair0 * 2;
            uint4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = *reinterpret_cast<const uint4 *>(src + 4 * k * P.pe_head);
            const int32_t pos = P.positions[tok];
            if (pos < 0) continue;
            float sn[4], cs[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) rope_sincos(pos, gh[j], gl[j], sn[j], cs[j]);
            uint4 *dst = reinterpret_cast<uint4 *>(P.q_rope + ((size_t)tok * kHeads + h0) * kDr + pair0 * 2);
#pragma unroll
            for (int k = 0; k < 8; ++k) dst[4 * k * (kDr / 8)] = turn8(v[k], sn, cs);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

std::mutex g_query_mutex;
bool g_query_attr[64];

bool aligned(const void *p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

// mla_query; of a mixed step (plan.sparse), more than kQuerySmall tokens and kMaxPlanTiles tiles at most, for its rows only.
mla_status launch_query(int32_t tokens, const void *q_nope, int64_t nope_token_stride, int64_t nope_head_stride,
                        const void *q_pe, int64_t pe_token_stride, int64_t pe_head_stride, const void *w_uk,
                        const float *rope_table, const int32_t *positions, void *q_latent, void *q_rope,
                        int32_t *device_status, const TreePlanRef &plan, mla_stream_t stream) {
    if (tokens < 1) return MLA_ERR_INVALID_ARG;
    if ((int64_t)tokens * kHeads >= (int64_t)1 << 31) return MLA_ERR_UNSUPPORTED;
    if (!aligned(q_nope, 16) || !aligned(q_pe, 16) || !aligned(w_uk, 16) || !aligned(q_latent, 16) ||
        !aligned(q_rope, 16) || !aligned(rope_table, 4) || !aligned(positions, 4) || !aligned(device_status, 4))
        return MLA_ERR_INVALID_ARG;
    for (const int64_t s : {nope_token_stride, nope_head_stride, pe_token_stride, pe_head_stride})
        if (s < 1 || s % 8 || s >= (int64_t)1 << 31) return MLA_ERR_INVALID_ARG;
    if (plan.sparse && (tokens <= kQuerySmall || (tokens - 1) / kTile >= kMaxPlanTiles)) return MLA_ERR_UNSUPPORTED;
    if (tokens <= kQuerySmall)
        return launch_query_small(tokens, q_nope, nope_token_stride, nope_head_stride, q_pe, pe_token_stride,
                                  pe_head_stride, w_uk, rope_table, positions, q_latent, q_rope, device_status, stream);
    int dev = 0;
    int32_t units = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MLA_ERR_CUDA;
    if (main_units(&units) != cudaSuccess) return MLA_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lock(g_query_mutex);
        if (!g_query_attr[dev]) {
            for (auto *k : {mla_query_kernel<false>, mla_query_kernel<true>})
                if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kQuerySmem) != cudaSuccess)
                    return MLA_ERR_CUDA;
            g_query_attr[dev] = true;
        }
    }
    QueryParams p{};
    if (!encode_bf16_4d(&p.tm_a, q_nope, (cuuint64_t)tokens, kDimN / 64, kHeads, (cuuint64_t)nope_token_stride * 2, 128,
                        (cuuint64_t)nope_head_stride * 2, kTile, kDimN / 64) ||
        !encode_bf16_4d(&p.tm_w, w_uk, kDimN, kDl / 64, kHeads, kDl * 2, 128, (cuuint64_t)kDimN * kDl * 2, kDimN,
                        kCols / 64))
        return MLA_ERR_CUDA;
    p.q_pe = static_cast<const __nv_bfloat16 *>(q_pe);
    p.pe_token = pe_token_stride;
    p.pe_head = pe_head_stride;
    p.positions = positions;
    p.rope_table = rope_table;
    p.q_latent = static_cast<__nv_bfloat16 *>(q_latent);
    p.q_rope = static_cast<__nv_bfloat16 *>(q_rope);
    p.status = device_status;
    p.tokens = tokens;
    p.tiles = (tokens + kTile - 1) / kTile;
    p.plan = plan;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * units < kHeads * kHalves ? 2 * units : kHeads * kHalves));   // one CTA per SM
    cfg.blockDim = dim3(kQueryThreads);
    cfg.dynamicSmemBytes = kQuerySmem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    auto *kernel = plan.sparse ? mla_query_kernel<true> : mla_query_kernel<false>;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace mla

extern "C" mla_status mla_query(int32_t tokens, const void *q_nope, int64_t nope_token_stride,
                                int64_t nope_head_stride, const void *q_pe, int64_t pe_token_stride,
                                int64_t pe_head_stride, const void *w_uk, const float *rope_table,
                                const int32_t *positions, void *q_latent, void *q_rope, int32_t *device_status,
                                mla_stream_t stream) {
    mla::NvtxRange nvtx_range("mla_query");
    return mla::launch_query(tokens, q_nope, nope_token_stride, nope_head_stride, q_pe, pe_token_stride, pe_head_stride,
                             w_uk, rope_table, positions, q_latent, q_rope, device_status, {}, stream);
}
