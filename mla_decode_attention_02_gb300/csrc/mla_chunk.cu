// Attention of a step's chunks over the heads' keys and values (include/mla_chunk.h):
//
//   o[t][h] = sum_j softmax(scale q[t][h] . k[j][h])_j v[j][h]      192-value scores, 128-value outputs,
//   j from the first slot of t's request to t's own
//
// An item is one head of one tile of 256 tokens (mla_chunk_plan.cu), taken as two MMA tiles
// of 128 tokens that share every key tile of 128; a tile of up to 128 tokens as two halves of its
// keys, merged at the end.  GB300 design, one CTA per SM:
//   warp 8      TMA: the queries (96 KB), then keys and values as 16 KB blocks of 64 dims through a ring
//               of eight (a key tile's three blocks, its two value blocks, the next key tile's ...)
//   warp 9      MMAs of 128 x 128: S = q K^T (K = 192) into TMEM, and O += P V (K = 64 twice) with P read from
//               TMEM; the two tiles take turns, so that one's softmax runs while the other's products do
//   warps 0-3   softmax of the first tile, one thread a row, 64 keys at a time: S from TMEM, the running maximum and
//   warps 4-7   sum in registers, P as fp16 back over S and each half handed over; the second tile's likewise
// TMEM: S and O of both tiles, 4 x 128 columns, all of it.  A thread whose row's maximum grows by more than 2^8
// rescales the row's O itself, which waits for the product before; smaller growth leaves the reference as it
// is (exact: the reference is a shift).  Weights and values are fp16 for their product, three bits
// more than bf16; the sum is taken of the unrounded weights.
// fp16 has those bits down to 2^-14 only and ends at 2^-25, while a row whose first key draws nearly all the weight has
// thousands of others far below it.  So the weights stand 2^7 above the reference (at most 2^15), and where 64 keys in a row
// have none within 2^-20 of the reference it falls to their largest (once in eight key tiles at most, so that scores that
// go up and down cost little, and 2^40 below its highest at most, which fp32's range bears).  32768 keys of which one draws
// 0.9986 of the weight, with a value of zero: this rounding is without both 0.33 of the output's norm, with the lift alone 2e-3,
// with both 3e-4; a lift of 2^11 (then raised at 2^4) does as well but takes 11 to 35% longer where scores are twice as
// wide or more.
// Bound by the tensor cores, 81,920 flops a (token, key) pair and 128 heads, and by the power they draw: 2048 tokens over
// 32768 keys 3.04 ms (1.76 PFLOP/s; without the softmax's arithmetic 2.72, with keys from L2 alone 2.91), a prompt of 4096
// 460 us (1.5, the diagonal's masked halves and 13 items' beginnings and ends a CTA; tensor pipe 71% of the clocks).
// Measured on the way: items by index instead of in turn 705 -> 552 us (prompt), maxima in eight chains 523, weights before
// the maximum is known 505, requests together and the last heads tile by tile 480, halves 457; value products as two of
// 64 columns 3200 instead of 3030 us (long), with run-time loops around the MMAs 4170 (their issue then takes longer than
// they do), S in pieces of 16 columns 3215.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
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
cudaError_t launch_chunk_expand(const mla_chunk *prob, const void *w_uk, const void *w_uv, const void *cache, bool fp8,
                                int64_t num_pages, const int32_t *block_table, void *ws, void *rope, void *kv,
                                int32_t head0, int32_t heads, cudaStream_t stream);
namespace {
using namespace ptx;

constexpr int kSoftWarps = 8, kTmaWarp = 8, kMmaWarp = 9;
constexpr int kChunkThreads = 32 * 10;
constexpr int kSlots = 8;
constexpr int kKeys = 128;                              // keys of a tile
constexpr uint32_t kBlk = 128 * 128;                    // 128 rows x 64 dims
constexpr uint32_t kQTile = 3 * kBlk;                   // 128 tokens x 192 dims
constexpr uint32_t kOffRing = 2 * kQTile;
constexpr uint32_t kChunkSmem = kOffRing + kSlots * kBlk + 1024;
constexpr uint32_t kColS = 0, kColO = 256;              // + 128 per tile
constexpr uint64_t kChunkWaitNs = 2000000000ull;
constexpr float kRescale = 8.0f, kLift = 7.0f;          // log2 units
static_assert(kRescale + kLift <= 15.0f, "a weight is an fp16 value");
constexpr float kLow = 20.0f, kFall = 40.0f;
constexpr int kLowEvery = 8;
static_assert(kChunkSmem <= 232448 - 1024, "shared memory budget");

struct ChunkParams {
    CUtensorMap tm_qn, tm_qr;   // queries as (64 dims, tokens, dim blocks, heads), box 64 x 128 x 2 (1) x 1
    CUtensorMap tm_kv;          // scratch as (64 dims, rows, 4 blocks, heads), box 64 x 128 x 1 x 1
    CUtensorMap tm_kr;          // its rotary parts as (64 dims, rows, 1, 1), box 64 x 128 x 1 x 1
    uint8_t *ws;
    __nv_bfloat16 *out;
    float *lse;
    int64_t kv_tokens;
    float scale_log2;
    int32_t batch, tokens, max_pages, head0, heads;
};

// One head of a tile, on its way from the TMA warp to the others (head < 0: there are no more).
struct ChunkItem {
    ChunkTile tile;
    int32_t head, pad[3];
};

struct Wait {
    volatile int *abort;
    int32_t *status;
};

// Bounded wait; on time-out flags the CTA (every other wait then gives up at once).
__device__ __noinline__ bool wait_slow(const Wait w, uint32_t bar, uint32_t parity) {
    uint64_t t0 = 0;
    for (uint32_t i = 0;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63) == 63) {
            if (*w.abort) return false;
            const uint64_t t = globaltimer_ns();
            if (t0 == 0) t0 = t;
            else if (t - t0 > kChunkWaitNs) {
                *w.abort = 1;
                atomicOr(w.status, MLA_DEV_TIMEOUT);
                return false;
            }
        }
    }
}

__device__ __forceinline__ bool wait(const Wait &w, uint32_t bar, uint32_t parity) {
    return mbar_try_wait(bar, parity) || wait_slow(w, bar, parity);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Teardown: what is in flight lands, whatever the abort flag says (bounded).
__device__ __noinline__ void wait_landed(const Wait w, uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (globaltimer_ns() - t0 > kChunkWaitNs) {
            atomicOr(w.status, MLA_DEV_TIMEOUT);
            return;
        }
    }
}

// 32 bytes: a sector at once if they are one.
__device__ __forceinline__ void st_global_v8(void *at, const uint32_t *x, bool whole) {
    if (!whole) {
        reinterpret_cast<uint4 *>(at)[0] = make_uint4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<uint4 *>(at)[1] = make_uint4(x[4], x[5], x[6], x[7]);
        return;
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                 "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

// Multiply a row's 128 output values in TMEM.
__device__ __noinline__ void rescale(uint32_t col, float f) {
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        uint32_t r[32];
        tmem_ld32(col + c * 32, r);
        tmem_wait_ld(r);
#pragma unroll
        for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
        tmem_st32(col + c * 32, r);
    }
    tmem_wait_st();
}

// A row's 128 output values in TMEM times f0, with f1 times those of the other half 128 columns on added.
__device__ __noinline__ void add_half(uint32_t col, float f0, float f1) {
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        uint32_t r[32], x[32];
        tmem_ld32(col + c * 32, r);
        tmem_ld32(col + 128 + c * 32, x);
        tmem_wait_ld(r);
        tmem_wait_ld(x);
#pragma unroll
        for (int e = 0; e < 32; ++e)
            r[e] = __float_as_uint(fmaf(__uint_as_float(x[e]), f1, __uint_as_float(r[e]) * f0));
        tmem_st32(col + c * 32, r);
    }
    tmem_wait_st();
}

// A tile in error: its rows' outputs are NaN.
__device__ __noinline__ void write_nan(const ChunkParams &P, const ChunkTile t, int head, int thread, int threads) {
    const uint32_t nan2 = 0x7fff7fffu;
    for (int i = thread; i < t.count * (kDv / 8); i += threads) {
        const int row = t.t0 + i / (kDv / 8);
        reinterpret_cast<uint4 *>(P.out + ((size_t)row * kHeads + head) * kDv)[i % (kDv / 8)] =
            make_uint4(nan2, nan2, nan2, nan2);
    }
    if (P.lse)
        for (int i = thread; i < t.count; i += threads)
            P.lse[(size_t)(t.t0 + i) * kHeads + head] = __int_as_float(0x7fffffff);
}

__global__ void __launch_bounds__(kChunkThreads, 1) mla_chunk_kernel(const __grid_constant__ ChunkParams P) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * kSlots + 21];
    __shared__ ChunkItem s_item[2];
    __shared__ float2 s_stat[128];   // maximum and sum of the second half's rows
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const uint32_t s_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // + ring slot: landed, read; + tile: queries landed, queries read, S complete; + 2 half + tile: P written, product
    // done (of half a key tile);
    // + item parity: item there, item read; the second half's rows handed over, merged
    enum { B_FULL = 0, B_EMPTY = kSlots, B_QFULL = 2 * kSlots, B_QFREE = B_QFULL + 2, B_S = B_QFREE + 2, B_P = B_S + 2,
           B_PV = B_P + 4, B_ITEM = B_PV + 4, B_TAKEN = B_ITEM + 2, B_HALF = B_TAKEN + 2, B_MERGED,
           B_DRAIN };
    static_assert(B_DRAIN + 1 == 2 * kSlots + 21, "barriers");
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(bar(B_FULL + s), 1);
            mbar_init(bar(B_EMPTY + s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(B_QFULL + s), 1);
            mbar_init(bar(B_QFREE + s), 1);
            mbar_init(bar(B_S + s), 1);
            for (int half = 0; half < 2; ++half) {
                mbar_init(bar(B_P + 2 * half + s), kSoftWarps / 2);
                mbar_init(bar(B_PV + 2 * half + s), 1);
            }
            mbar_init(bar(B_ITEM + s), 1);
            mbar_init(bar(B_TAKEN + s), 1 + kSoftWarps);
        }
        mbar_init(bar(B_HALF), kSoftWarps / 2);
        mbar_init(bar(B_MERGED), kSoftWarps / 2);
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

    PlanHeader *hdr = reinterpret_cast<PlanHeader *>(P.ws);
    const Wait w = {&abort_flag, &hdr->status};
    const bool fits = hdr->magic == kChunkMagic && hdr->batch == P.batch && hdr->s_q == P.tokens &&
                      hdr->max_pages == P.max_pages && hdr->total_cost == P.kv_tokens;
    if (!fits && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&hdr->status, MLA_DEV_BAD_PLAN);
    const ChunkTile *tiles = reinterpret_cast<const ChunkTile *>(P.ws + chunk_layout(P.batch, P.tokens, P.kv_tokens).tiles);
    // Items: request by request, and head by head a request's tiles together (they read the same keys).  The last
    // request's last heads go tile by tile, the longest first, so that all CTAs end with short items.  A CTA begins with
    // the item of its index and then takes whatever is next.
    const int32_t num_tiles = fits ? hdr->num_items : 0;
    const int64_t items = (int64_t)num_tiles * P.heads;
    auto item_at = [&](int64_t i) {
        ChunkItem it;
        it.head = -1;
        if (i >= items) return it;
        const ChunkTile any = tiles[(int32_t)(i / P.heads)];
        const int32_t nt = any.end - any.first;
        int64_t at = i - (int64_t)any.first * P.heads;
        const int32_t few = ((int32_t)gridDim.x + nt - 1) / nt, late = any.end < num_tiles || few > P.heads ? 0 : few;
        const int64_t split = (int64_t)(P.heads - late) * nt;
        int32_t tile;
        if (at < split) {
            it.head = (int32_t)(at / nt);
            tile = (int32_t)(at % nt);
        } else {
            at -= split;
            it.head = P.heads - late + (int32_t)(at % late);
            tile = (int32_t)(at / late);
        }
        it.tile = tiles[any.first + tile];
        return it;
    };
    // Key tiles of one MMA tile of tokens: up to the one with its last token's slot.  An item of one such tile (up to 128
    // tokens) is run as two, which take its key tiles in turn and are merged at the end.
    auto key_tiles = [](const ChunkTile &t, int s) {
        const bool split = t.count <= 128;
        const int last = (split || t.count < 128 * (s + 1) ? t.count : 128 * (s + 1)) - 1, n = (t.slot0 + last) / kKeys + 1;
        return split ? (n + 1 - s) / 2 : n;
    };
    // The k-th item of this CTA, as the MMA thread or a softmax warp sees it.
    auto item_of = [&](uint32_t k, bool &ok) {
        ChunkItem it;
        it.head = -1;
        if (ok) ok = wait(w, bar(B_ITEM + (k & 1)), (k >> 1) & 1);
        if (ok) it = s_item[k & 1];
        return it;
    };

    if (warp == kTmaWarp) {
        if (elect_one()) {
            prefetch_tmap(&P.tm_qn);
            prefetch_tmap(&P.tm_qr);
            prefetch_tmap(&P.tm_kv);
            prefetch_tmap(&P.tm_kr);
            uint32_t n = 0, loads[2] = {0, 0};
            bool ok = true;
            // blocks [b0, b1) of a key tile: its keys' two, their rotary part, its values' two
            auto load = [&](int row, int hl, int b0, int b1) {
#pragma unroll 1
                for (int b = b0; b < b1; ++b) {
                    const uint32_t s = n % kSlots;
                    if (n >= kSlots) ok = ok && wait(w, bar(B_EMPTY + s), (n / kSlots - 1) & 1);
                    if (!ok) return;
                    mbar_arrive_expect_tx(bar(B_FULL + s), kBlk);
                    // (a pair of value blocks that wraps around the ring is swapped: the first 64 dims lie lower)
                    const bool swap = b >= 3 && (n - (b - 3)) % kSlots == kSlots - 1;
                    const int blk = b < 2 ? b : b == 2 ? 0 : swap ? 6 - b : b - 1;
                    tma_load_4d(s_base + kOffRing + s * kBlk, b == 2 ? &P.tm_kr : &P.tm_kv, 0, row, blk, b == 2 ? 0 : hl,
                                bar(B_FULL + s));
                    ++n;
                }
            };
            int64_t i = blockIdx.x;
            for (uint32_t k = 0; ok; ++k) {
                const ChunkItem it = item_at(i);
                if (k >= 2) ok = wait(w, bar(B_TAKEN + (k & 1)), ((k >> 1) - 1) & 1);
                if (!ok) break;
                s_item[k & 1] = it;
                mbar_arrive(bar(B_ITEM + (k & 1)));
                if (it.head < 0) break;
                i = gridDim.x + (int64_t)atomicAdd(reinterpret_cast<unsigned long long *>(&hdr->target), 1ull);
                const ChunkTile &t = it.tile;
                if (t.slot0 < 0) continue;
                const int hl = it.head, h = P.head0 + hl;
                const int n0 = key_tiles(t, 0), n1 = key_tiles(t, 1);
                // in the order of their use: of two halves, a tile's products come after the next tile's scores
                const bool split = t.count <= 128;
                const int tiles_of_keys = split ? n0 + n1 : n1, behind = split;
                for (int j = 0; j < tiles_of_keys + behind && ok; ++j) {
                    if (j < tiles_of_keys) load(t.base + j * kKeys, hl, 0, 3);
                    if (j == 0) {   // the queries, once the item before has read its own
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            if (s == 1 && split) break;
                            if (loads[s]) ok = ok && wait(w, bar(B_QFREE + s), (loads[s] - 1) & 1);
                            if (!ok) break;
                            mbar_arrive_expect_tx(bar(B_QFULL + s), kQTile);
                            tma_load_4d(s_base + s * kQTile, &P.tm_qn, 0, t.t0 + 128 * s, 0, h, bar(B_QFULL + s));
                            tma_load_4d(s_base + s * kQTile + 2 * kBlk, &P.tm_qr, 0, t.t0 + 128 * s, 0, h, bar(B_QFULL + s));
                            ++loads[s];
                        }
                    }
                    if (j >= behind) load(t.base + (j - behind) * kKeys, hl, 3, 5);
                }
            }
            // every copy has landed before the CTA gives its memory up
            for (uint32_t k = n > kSlots ? n - kSlots : 0; k < n; ++k)
                wait_landed(w, bar(B_FULL + k % kSlots), (k / kSlots) & 1);
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (loads[s]) wait_landed(w, bar(B_QFULL + s), (loads[s] - 1) & 1);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        if (elect_one()) {
            constexpr uint32_t idesc_s = idesc_bf16(128, kKeys, 0, 0), idesc_o = idesc_f16(128, kDv, 0, 1);
            uint32_t n = 0, q_phase = 0, p_phase = 0;   // n: ring blocks before this item's; phases: bit s is tile s's
            bool ok = true;
            for (uint32_t item = 0; ok; ++item) {
                const ChunkItem it = item_of(item, ok);
                if (it.head < 0) break;
                mbar_arrive(bar(B_TAKEN + (item & 1)));
                const ChunkTile &t = it.tile;
                if (t.slot0 < 0) continue;
                const int n0 = key_tiles(t, 0), n1 = key_tiles(t, 1), most = n0 > n1 ? n0 : n1;
                const bool split = t.count <= 128;
                // The two tiles in turn: the products of key tile j, then the scores of the next, so that one's softmax runs
                // while the other's products do.  Two tiles of tokens share every block; two halves of the keys have their own,
                // in this order.
                uint32_t next = n;
#pragma unroll 1
                for (int j = -1; j < most && ok; ++j) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const int nk = s ? n1 : n0;
                        if (j >= 0 && j < nk) {   // O (+)= P V
                            const uint32_t k = split ? next : n + 5 * j + 3, a = k % kSlots, b = (k + 1) % kSlots;
                            next += 2;
                            // (the first 64 dims are in the lower of the two slots)
                            const uint64_t d = smem_desc(s_base + kOffRing + (a < b ? a : b) * kBlk, a < b ? kBlk : 7 * kBlk,
                                                         1024, 2);
                            ok = wait(w, bar(B_FULL + a), (k / kSlots) & 1) && wait(w, bar(B_FULL + b), ((k + 1) / kSlots) & 1);
#pragma unroll
                            for (int half = 0; half < 2; ++half) {   // 64 keys each, as their weights come
                                ok = ok && wait(w, bar(B_P + 2 * half + s), p_phase >> s & 1);
                                if (!ok) break;
                                tc_fence_after();
#pragma unroll
                                for (int ks = 4 * half; ks < 4 * half + 4; ++ks)
                                    mma_ts(tmem + kColO + s * 128, tmem + kColS + s * 128 + ks * 8, d + ks * (2048 >> 4),
                                           idesc_o, (j > 0 || ks) ? 1u : 0u);
                                mma_commit(bar(B_PV + 2 * half + s));
                            }
                            p_phase ^= 1u << s;
                            if (!ok) break;
                            if (split || s == 1) {
                                mma_commit(bar(B_EMPTY + a));
                                mma_commit(bar(B_EMPTY + b));
                            }
                        }
                        if (j + 1 < nk) {   // S = q K^T
                            const uint32_t k = split ? next : n + 5 * (j + 1);
                            next += 3;
                            if (j < 0 && (s == 0 || !split)) {
                                ok = wait(w, bar(B_QFULL + s), q_phase >> s & 1);
                                q_phase ^= 1u << s;
                            }
                            const uint64_t dq = smem_desc(s_base + (split ? 0 : s) * kQTile, 16, 1024, 2);
#pragma unroll
                            for (int b = 0; b < 3; ++b) {
                                const uint32_t slot = (k + b) % kSlots;
                                ok = ok && wait(w, bar(B_FULL + slot), ((k + b) / kSlots) & 1);
                                if (!ok) break;
                                tc_fence_after();
                                const uint64_t d = smem_desc(s_base + kOffRing + slot * kBlk, 16, 1024, 2);
#pragma unroll
                                for (int ks = 0; ks < 4; ++ks)
                                    mma_ss(tmem + kColS + s * 128, dq + b * (kBlk >> 4) + ks * 2, d + ks * 2, idesc_s,
                                           (b | ks) ? 1u : 0u);
                                if (split || s == 1) mma_commit(bar(B_EMPTY + slot));
                            }
                            if (!ok) break;
                            mma_commit(bar(B_S + s));
                            // the last scores of a tile's queries (two halves have one tile: n1 is n0 or one less)
                            if (split ? j + 1 == (n1 == n0 ? n1 : n0) - 1 && s == (n1 == n0) : j + 2 == nk)
                                mma_commit(bar(B_QFREE + (split ? 0 : s)));
                        }
                    }
                }
                n += split ? 5 * (n0 + n1) : 5 * n1;
            }
            mma_commit(bar(B_DRAIN));   // every MMA is done before the CTA gives its memory up
            wait_landed(w, bar(B_DRAIN), 0);
        }
        __syncwarp();
    } else {
        // ---- softmax of MMA tile s: a thread's row is accumulator lane 32 quarter + lane
        const int s = warp >> 2, quarter = warp & 3;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t col_s = lanes + kColS + s * 128, col_o = lanes + kColO + s * 128;
        uint32_t phase = 0, merges = 0;   // key tiles and merges before this item's
        bool ok = true;
        for (uint32_t item = 0; ok; ++item) {
            const ChunkItem it = item_of(item, ok);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || it.head < 0) break;
            if (lane == 0) mbar_arrive(bar(B_TAKEN + (item & 1)));
            const ChunkTile &t = it.tile;
            const int h = P.head0 + it.head;
            if (t.slot0 < 0) {
                write_nan(P, t, h, threadIdx.x, 32 * kSoftWarps);
                continue;
            }
            const bool split = t.count <= 128;
            const int nk = key_tiles(t, s), row = (split ? 0 : 128 * s) + quarter * 32 + lane;
            const bool mine = row < t.count;
            const int slot = t.slot0 + (mine ? row : t.count - 1);   // (a row past the tile's end: any legal slot)
            const int least = __shfl_sync(0xffffffffu, slot, 0);     // the warp's first row sees the fewest keys
            float m = -INFINITY, sum = 0.f;   // the reference, the weights' sum by it
            float peak = -INFINITY;           // the highest reference so far
            int low_from = 1;                 // the key tile from which on references may fall (the same for a warp)
            for (int j = 0; j < nk; ++j, ++phase) {
                if (!__all_sync(0xffffffffu, wait(w, bar(B_S + s), phase & 1))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int first = (split ? 2 * j + s : j) * kKeys;
                const int limit = slot - first;   // the last key of the tile that the row sees
                const bool masked = least - first < kKeys - 1;
                // Half of the tile at a time.  The weights by the reference as it is, while the half's maximum is found: it
                // is read once.  If the reference has to be raised (always at a row's first tile, seldom later) or falls it
                // is read again.
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    uint32_t wgt[32];
                    float2 all;
                    const int seen = limit - 64 * half;
                    for (;;) {
                        // (no key seen so far: weights of 0)
                        const float neg = m == -INFINITY ? 0.f : fmaf(-m, P.scale_log2, kLift);
                        const uint64_t scale2 = pair(P.scale_log2, P.scale_log2), shift2 = pair(neg, neg);
                        uint64_t part[2] = {0, 0};
                        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                        uint32_t r[2][32];
                        tmem_ld32(col_s + 64 * half, r[0]);
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t(&x)[32] = r[c];
                            tmem_wait_ld(x);
                            if (c == 0) tmem_ld32(col_s + 64 * half + 32, r[1]);
                            if (masked) {
#pragma unroll
                                for (int e = 0; e < 32; ++e) x[e] = c * 32 + e <= seen ? x[e] : 0xff800000u;
                            }
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
#pragma unroll
                                for (int g = 0; g < 4; ++g)
                                    tops[g] =
                                        fmaxf(fmaxf(tops[g], __uint_as_float(x[e + g])), __uint_as_float(x[e + 4 + g]));
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float2 y = unpair(fma_pair(
                                    pair(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), scale2, shift2));
                                const float a = ex2(y.x), b = ex2(y.y);
                                part[e & 1] = add_pair(part[e & 1], pair(a, b));
                                wgt[c * 16 + e] = pack_f16x2(a, b);
                            }
                        }
                        all = unpair(add_pair(part[0], part[1]));
                        const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                        const float over = (top - m) * P.scale_log2;
                        const bool raise = over > kRescale;
                        const bool fall = j >= low_from && over < -kLow && top > -INFINITY;
                        if (!__any_sync(0xffffffffu, raise || fall)) break;
                        if (__any_sync(0xffffffffu, fall)) low_from = j + kLowEvery;
                        float f = 1.f;
                        if (raise || fall) {
                            const float to = raise ? top : fmaxf(top, peak - kFall / P.scale_log2);
                            f = ex2((m - to) * P.scale_log2);
                            m = to;
                            peak = fmaxf(peak, m);
                            sum *= f;
                        }
                        // O holds what came before: once its last product is done
                        if (j > 0 || half > 0) {
                            if (!__all_sync(0xffffffffu, half ? wait(w, bar(B_PV + s), phase & 1)
                                                              : wait(w, bar(B_PV + 2 + s), (phase - 1) & 1))) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            rescale(col_o, f);
                        }
                    }
                    if (!ok) break;
                    sum += all.x + all.y;
                    tmem_st32(col_s + 32 * half, wgt);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_P + 2 * half + s));
                }
                if (!ok) break;
            }
            if (!ok || !nk) continue;
            // ---- the item's output, once its last product is done
            if (!__all_sync(0xffffffffu, wait(w, bar(B_PV + 2 + s), (phase - 1) & 1))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const bool merge = split && key_tiles(t, 1) > 0;
            if (merge) {
                float2 *stat = &s_stat[quarter * 32 + lane];
                if (s == 1) {   // hands its row over and goes on when it has been read
                    *stat = make_float2(m, sum);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_HALF));
                    ok = __all_sync(0xffffffffu, wait(w, bar(B_MERGED), merges++ & 1));
                    continue;
                }
                if (!__all_sync(0xffffffffu, wait(w, bar(B_HALF), merges++ & 1))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float2 other = *stat;   // (its maximum is -infinity if the row sees none of its keys)
                const float top = fmaxf(m, other.x);
                const float f0 = ex2((m - top) * P.scale_log2), f1 = ex2((other.x - top) * P.scale_log2);
                sum = sum * f0 + other.y * f1;
                m = top;
                add_half(col_o, f0, f1);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_MERGED));
            }
            const float inv = 1.f / sum;
            __nv_bfloat16 *dst = P.out + ((size_t)(t.t0 + row) * kHeads + h) * kDv;
            const bool whole = (reinterpret_cast<uintptr_t>(P.out) & 31) == 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {   // (in whole sectors)
                uint32_t r[32];
                tmem_ld32(col_o + c * 32, r);
                tmem_wait_ld(r);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    r[e] = pack_bf16x2(__uint_as_float(r[2 * e]) * inv, __uint_as_float(r[2 * e + 1]) * inv);
                if (mine) {
                    st_global_v8(dst + c * 32, &r[0], whole);
                    st_global_v8(dst + c * 32 + 16, &r[8], whole);
                }
            }
            if (mine && P.lse)
                P.lse[(size_t)(t.t0 + row) * kHeads + h] = (m * P.scale_log2 + (log2f(sum) - kLift)) * 0.6931471805599453f;
            tc_fence_before();   // the next item's first product writes over O: after its P, which these threads write
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

std::mutex g_chunk_mutex;
bool g_chunk_attr[64];

bool aligned(const void *p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

mla_status attend(const mla_chunk *prob, const void *q_nope, int64_t nope_token, int64_t nope_head, const void *q_rope,
                  int64_t rope_token, int64_t rope_head, const void *w_uk, const void *w_uv, const void *cache, bool fp8,
                  int64_t num_pages, const int32_t *block_table, float scale, void *out, float *lse, void *workspace,
                  size_t workspace_bytes, void *scratch, size_t scratch_bytes, mla_stream_t stream) {
    const mla_status st = check_chunk(prob);
    if (st != MLA_OK) return st;
    if (!aligned(q_nope, 16) || !aligned(q_rope, 16) || !aligned(w_uk, 16) || !aligned(w_uv, 16) || !aligned(cache, 16) ||
        !aligned(block_table, 4) || !aligned(out, 16) || (reinterpret_cast<uintptr_t>(lse) & 3u) ||
        !aligned(workspace, 16) || !aligned(scratch, 128))
        return MLA_ERR_INVALID_ARG;
    for (const int64_t s : {nope_token, nope_head, rope_token, rope_head})
        if (s < 1 || s % 8 || s >= (int64_t)1 << 31) return MLA_ERR_INVALID_ARG;
    if (num_pages < 1 || num_pages >= (int64_t)1 << 31 || !std::isfinite(scale) || !(scale > 0.f))
        return MLA_ERR_INVALID_ARG;
    int dev = 0;
    int32_t units = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MLA_ERR_CUDA;
    if (main_units(&units) != cudaSuccess) return MLA_ERR_CUDA;
    const ChunkForm form = chunk_form(prob, units);
    if (workspace_bytes < chunk_workspace_bytes(prob, form, units)) return MLA_ERR_WORKSPACE;
    const size_t rope_bytes = chunk_rope_bytes(prob->kv_tokens), head_bytes = chunk_head_bytes(prob->kv_tokens);
    const size_t least = form == ChunkForm::kAbsorbed ? 0 : rope_bytes + head_bytes;
    // the scratch: the absorbed form's, its expanded pages if there is room, the whole form's
    uint8_t *const ws = static_cast<uint8_t *>(workspace), *const few_space = static_cast<uint8_t *>(scratch);
    uint8_t *space = few_space, *expanded = nullptr;
    if (form != ChunkForm::kWhole) {
        const size_t rows = absorbed_scratch_bytes(prob), pages = fp8 ? absorbed_expanded_bytes(prob) : 0;
        if (scratch_bytes < rows + least) return MLA_ERR_WORKSPACE;
        space += rows;
        if (pages && scratch_bytes - rows - least >= pages) {
            expanded = space;
            space += pages;
        }
        scratch_bytes -= (size_t)(space - few_space);
    }
    auto few = [&]() {
        const bool mixed = form == ChunkForm::kMixed;
        return absorbed_attend(prob, q_nope, nope_token, nope_head, q_rope, rope_token, rope_head, w_uk, w_uv, cache, fp8,
                               num_pages, block_table, scale, out, lse, mixed ? ws + mixed_tree(prob) : ws, mixed,
                               &reinterpret_cast<PlanHeader *>(ws)->status, few_space, expanded, units, stream);
    };
    if (form == ChunkForm::kAbsorbed) return few();
    if (scratch_bytes < least) return MLA_ERR_WORKSPACE;
    const size_t room = (scratch_bytes - rope_bytes) / head_bytes;
    const int32_t fit = room < (size_t)kHeads ? (int32_t)room : kHeads;
    const int32_t passes = (kHeads + fit - 1) / fit;
    {
        std::lock_guard<std::mutex> lock(g_chunk_mutex);
        if (!g_chunk_attr[dev]) {
            if (cudaFuncSetAttribute(mla_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kChunkSmem) !=
                cudaSuccess)
                return MLA_ERR_CUDA;
            g_chunk_attr[dev] = true;
        }
    }
    uint8_t *rope = space, *kv = rope + rope_bytes;
    const cuuint64_t rows = (cuuint64_t)chunk_rows(prob->kv_tokens), T = (cuuint64_t)prob->tokens;
    ChunkParams p{};
    if (!encode_bf16_4d(&p.tm_qn, q_nope, T, kDn / 64, kHeads, (cuuint64_t)nope_token * 2, 128, (cuuint64_t)nope_head * 2,
                        128, kDn / 64) ||
        !encode_bf16_4d(&p.tm_qr, q_rope, T, 1, kHeads, (cuuint64_t)rope_token * 2, 128, (cuuint64_t)rope_head * 2, 128, 1) ||
        !encode_bf16_4d(&p.tm_kr, rope, rows, 1, 1, kDr * 2, rows * kDr * 2, rows * kDr * 2, 128, 1) ||
        !encode_bf16_4d(&p.tm_kv, kv, rows, 4, (cuuint64_t)fit, (kDn + kDv) * 2, 128, rows * (kDn + kDv) * 2, 128, 1))
        return MLA_ERR_CUDA;
    p.ws = ws;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse = lse;
    p.kv_tokens = prob->kv_tokens;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.batch = prob->batch;
    p.tokens = prob->tokens;
    p.max_pages = prob->max_pages_per_seq;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * units));   // one CTA per SM
    cfg.blockDim = dim3(kChunkThreads);
    cfg.dynamicSmemBytes = kChunkSmem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    // passes of about the same number of heads
    for (int32_t pass = 0; pass < passes; ++pass) {
        p.head0 = (int32_t)((int64_t)kHeads * pass / passes);
        p.heads = (int32_t)((int64_t)kHeads * (pass + 1) / passes) - p.head0;
        if (launch_chunk_expand(prob, w_uk, w_uv, cache, fp8, num_pages, block_table, workspace, rope, kv, p.head0, p.heads,
                                cfg.stream) != cudaSuccess ||
            cudaLaunchKernelEx(&cfg, mla_chunk_kernel, p) != cudaSuccess)
            return MLA_ERR_CUDA;
    }
    return form == ChunkForm::kMixed ? few() : MLA_OK;
}

}  // namespace
}  // namespace mla

extern "C" mla_status mla_chunk_scratch_size(const mla_chunk *prob, int32_t heads, int32_t fp8, size_t *bytes) {
    const mla_status st = mla::check_chunk(prob);
    if (st != MLA_OK) return st;
    if (!bytes || heads < 1 || heads > mla::kHeads || (fp8 != 0 && fp8 != 1)) return MLA_ERR_INVALID_ARG;
    int32_t units = 0;
    if (mla::main_units(&units) != cudaSuccess) return MLA_ERR_CUDA;
    const mla::ChunkForm form = mla::chunk_form(prob, units);
    *bytes = 0;
    if (form != mla::ChunkForm::kWhole)
        *bytes += mla::absorbed_scratch_bytes(prob) + (fp8 ? mla::absorbed_expanded_bytes(prob) : 0);
    if (form != mla::ChunkForm::kAbsorbed)
        *bytes += mla::chunk_rope_bytes(prob->kv_tokens) + (size_t)heads * mla::chunk_head_bytes(prob->kv_tokens);
    return MLA_OK;
}

extern "C" mla_status mla_chunk_attend(const mla_chunk *prob, const void *q_nope, int64_t nope_token_stride,
                                       int64_t nope_head_stride, const void *q_rope, int64_t rope_token_stride,
                                       int64_t rope_head_stride, const void *w_uk, const void *w_uv,
                                       const void *kv_cache, int64_t num_pages, const int32_t *block_table, float scale,
                                       void *out, float *lse, void *workspace, size_t workspace_bytes, void *scratch,
                                       size_t scratch_bytes, mla_stream_t stream) {
    mla::NvtxRange nvtx_range("mla_chunk_attend");
    return mla::attend(prob, q_nope, nope_token_stride, nope_head_stride, q_rope, rope_token_stride, rope_head_stride, w_uk,
                       w_uv, kv_cache, false, num_pages, block_table, scale, out, lse, workspace, workspace_bytes,
                       scratch, scratch_bytes, stream);
}

extern "C" mla_status mla_chunk_attend_fp8(const mla_chunk *prob, const void *q_nope, int64_t nope_token_stride,
                                           int64_t nope_head_stride, const void *q_rope, int64_t rope_token_stride,
                                           int64_t rope_head_stride, const void *w_uk, const void *w_uv,
                                           const void *kv_cache_fp8, int64_t num_pages, const int32_t *block_table,
                                           float scale, void *out, float *lse, void *workspace, size_t workspace_bytes,
                                           void *scratch, size_t scratch_bytes, mla_stream_t stream) {
    mla::NvtxRange nvtx_range("mla_chunk_attend_fp8");
    return mla::attend(prob, q_nope, nope_token_stride, nope_head_stride, q_rope, rope_token_stride, rope_head_stride, w_uk,
                       w_uv, kv_cache_fp8, true, num_pages, block_table, scale, out, lse, workspace, workspace_bytes,
                       scratch, scratch_bytes, stream);
}
