// Schedule of a batch of drafted trees (include/mla_tree.h, mla_tree_plan): one
// row per node, in token order, its keys ending at its last visible one.
//
// A row costs pages + kItemCost, as in mla_plan.cu.  Trees differ from single
// tokens in that there are many rows and those of a request read the same pages:
// what runs at the same time should be of few requests, so that pages are read
// from L2.  So every unit gets rows spread over the whole batch and runs them in
// token order: at any time all units are at about the same requests.
//
//  - Whole rows: the rows are dealt in waves of one row per unit, each wave's
//    longest row to the unit with the least work so far (ranks by counting,
//    ties to the lower index).  Taken when its largest load is within 1/32 of
//    what cutting would give.
//  - Even pieces: with no more rows than units, every row in pieces of one size (two
//    pages at least), as small as one piece per unit allows.  Taken up to 1/12 above the
//    cut load.
//  - Cut rows: the rows lie on a cost line, every units-th row together (in token
//    order when there are no more rows than units), and the line is cut into equal
//    stretches as in mla_plan.cu (cut_row); a unit then runs its pieces in token order.
//
// Measured (decode alone) against the line in token order: 64 requests of 16
// nodes over 4096 keys 1001 -> 957 us (whole rows), 268 nodes of 80 keys 52 -> 44,
// 138 nodes of mixed lengths 118 -> 114 (cut rows).  Even pieces against cut rows (at least
// four pages each), requests x nodes x keys, us in a short burst / in a run of a second:
//
//                      even           cut                              even           cut
//   1 x 8 x 700      20.2 / 19.4   22.4 / 21.7     1 x 64 x 8192    142.8 / 141.3  137.0 / 136.0
//   1 x 16 x 1500    26.4 / 25.4   29.3 / 28.6     2 x 12 x 32768   189.3 / 191.3  185.6 / 191.5
//   1 x 1 x 8192     21.4 / 20.6   24.0 / 23.3     1 x 24 x 65536   359.3 / 366.5  348.6 / 364.3
//   3 x 5 x 5000     37.4 / 36.5   40.9 / 39.9     2 x 12 x 131072  701.5 / 725.5  687.3 / 744.6
//   1 x 8 x 16384    49.7 / 48.5   48.9 / 47.7
//   4 x 8 x 8192     82.2 / 80.6   77.9 / 76.8
//
// So they win up to 13% where a unit has a few pages, and lose 1 to 5% of a burst from some ten
// pages a unit on.  In the longest runs, under the power cap, a request's nodes at the same pages
// (a twelfth of the DRAM reads) win 2.6%.  The 1/12 decides 1 x 64 x 8192, 1 x 24 x 65536 and
// 2 x 12 x 131072, which would be cut without it.
//
// One CTA; every choice is a function of the inputs alone, and the host twin
// below makes the same ones.
// Without masks the rows are those of chunks of prompts (mla_chunk_absorbed.cu): any
// number of tokens a request, each seeing the slots up to its own; of a mixed step (forms) only the
// requests in that form, the rows of the others left as those behind the last.  For such chunks the planner also lays
// down the positions and the rotary table of zeros by which mla_query packs their queries (-1: a row without keys).
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>
#include <vector>

#include "mla_internal.h"
#include "mla_prolog.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

constexpr int kTreeThreads = 512;
constexpr int kMaxUnits = 96;   // units at most that whole rows are dealt to 
// Ranks compare 32-bit keys of a load or cost and an index below 256, so the loads of
// the dealt waves stay below 2^23 (a total far beyond what fits one step).
constexpr int64_t kMaxDealt = (int64_t)1 << 23;
static_assert(kMaxUnits <= 256 && 4 * kMaxUnits <= kTreeThreads && kMaxUnits % 32 == 0, "rank keys");
constexpr size_t kMaxTreeSmem = 200 * 1024;      // working set of the planner kernel

// Pages of rows that have no work items (their row_nparts follow).
constexpr int32_t kNoneUnused = 0, kNoneBad = -1, kNoneEmpty = -2;
MLA_HD int32_t none_parts(int32_t pages) {
    return pages == kNoneBad ? 0 : pages == kNoneEmpty ? kRowEmpty : kRowUnused;
}

// A node's row and its pages: pages to read, or one of the kNone codes.
MLA_HD int32_t tree_row(int32_t seq_len, int32_t nodes, int32_t req, uint64_t mask, int32_t max_pages, TreeRow *row) {
    const bool ok = seq_len >= nodes && seq_len <= (int64_t)max_pages * kPage;
    row->mask = ok ? (nodes < 64 ? mask & ((1ull << nodes) - 1) : mask) : 0;
    row->context = ok ? seq_len - nodes : 0;
    row->req = req;
    if (!ok) return kNoneBad;
    const int32_t end = tree_end(row->context, row->mask);
    return end > 0 ? (end + kPage - 1) / kPage : kNoneEmpty;
}

// Whether request b's stretch of the token array is sound.
MLA_HD bool tree_offsets_ok(int32_t o0, int32_t o1, int32_t b, int32_t tokens) {
    return o0 >= 0 && o0 <= o1 && o1 <= tokens && (b > 0 || o0 == 0) && (int64_t)o1 - o0 <= MLA_TREE_MAX_NODES;
}

// The i-th token of a chunk (no masks): every slot up to its own is context.
__device__ __forceinline__ int32_t chunk_row(int32_t seq_len, int32_t tokens, int32_t i, int32_t req, int32_t max_pages,
                                             TreeRow *row) {
    const int32_t p = tree_row(seq_len, tokens, req, 0, max_pages, row);
    if (p == kNoneBad) return p;
    row->context += i + 1;
    return (row->context - 1) / kPage + 1;
}

// Row at position k of the cost line: every units-th row together.
MLA_HD int32_t tree_line(int32_t k, int32_t rows, int32_t units) {
    const int32_t q = rows / units, rem = rows % units, head = rem * (q + 1);
    if (q == 0) return k;
    return k < head ? k / (q + 1) + k % (q + 1) * units : rem + (k - head) / q + (k - head) % q * units;
}

// Whether dealing whole rows is tried at all: the longest alone would be too much, or the keys too small.
MLA_HD bool keep_whole(int64_t max_load, int64_t target);
MLA_HD bool try_whole(int32_t units, int64_t longest, int64_t total, int64_t target) {
    return units <= kMaxUnits && total < kMaxDealt && keep_whole(longest, target);
}

// Whether rows stay whole, given the largest load of the dealt waves.
MLA_HD bool keep_whole(int64_t max_load, int64_t target) {
    return max_load <= target + kItemCost + kSplitPenalty + target / 32;
}

// Pieces of a row when pieces have `cap` pages at most, and the first page of piece i of k.
constexpr int32_t kEvenPages = 2;
MLA_HD int32_t even_pieces(int32_t pages, int32_t cap) { return pages > 0 ? (pages - 1) / cap + 1 : 0; }
// The largest cap that even pieces are taken with: up to 1/12 above the cut line's load, since a
// request's nodes then read the same pages at the same time.
MLA_HD int32_t even_most(int64_t longest, int64_t target) {
    const int64_t cap = target + kSplitPenalty + target / 12;
    return (int32_t)(cap < longest ? cap : longest);
}
MLA_HD int32_t even_page(int32_t pages, int32_t i, int32_t k) { return (int32_t)((int64_t)pages * i / k); }

size_t tree_plan_smem(int32_t R, int32_t U) {
    return 8 * (size_t)R + 4 * (3 * (size_t)R + 2 * (size_t)U) + 4 * (3 * (size_t)U + 2);
}

// Inclusive block-wide sum of one int64 per thread.
__device__ int64_t block_scan(int64_t v, int64_t *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t n = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += n;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    int64_t before = 0;
#pragma unroll
    for (int w = 0; w < kTreeThreads / 32; ++w) before += w < warp ? warp_sums[w] : 0;
    __syncthreads();
    return v + before;
}

// kChunk: of chunks (no masks).
template <bool kChunk>
__global__ void __launch_bounds__(kTreeThreads, 1)
mla_tree_plan_kernel(const int32_t *__restrict__ seq_lens, const int32_t *__restrict__ offsets,
                     const uint64_t *__restrict__ masks, const uint8_t *forms, int32_t *zeros, uint8_t *__restrict__ ws,
                     int32_t batch, int32_t tokens, int32_t max_pages, int32_t num_units) {
    __shared__ int64_t warp_sums[kTreeThreads / 32], warp_most[kTreeThreads / 32];
    __shared__ int64_t carry, carry_parts;
    __shared__ __align__(16) uint32_t unit_key[kMaxUnits];
    __shared__ int32_t bad, special, even_cap;   // even_cap: 0 for no even pieces
    extern __shared__ int64_t smem[];
    const int32_t R = tokens, U = num_units, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const PlanLayout L = make_layout(R, U, batch);
    int64_t *s_pos = smem;                                       // [R] cost-line start (cut rows)
    int32_t *s_end = reinterpret_cast<int32_t *>(s_pos + R);     // [R] one past the last visible key, or a kNone code
    int32_t *s_unit = s_end + R;      // [R + U] unit of each row (whole) or piece on the line (cut)
    int32_t *s_row = s_unit + R + U;    // [R + U] the row's place in its unit, or the piece's row
    int32_t *s_count = s_row + R + U;   // [U]
    int32_t *s_rank = s_count + U;      // [U]
    int32_t *s_begin = s_rank + U;      // [U + 1]
    // a row's pages, or its kNone code
    auto pages = [&](int32_t r) { return s_end[r] > 0 ? (s_end[r] - 1) / kPage + 1 : s_end[r]; };
    PlanHeader *hdr = reinterpret_cast<PlanHeader *>(ws);
    WorkItem *items = reinterpret_cast<WorkItem *>(ws + L.items);
    int32_t *item_unit = reinterpret_cast<int32_t *>(ws + L.item_unit);
    int32_t *unit_begin = reinterpret_cast<int32_t *>(ws + L.unit_begin);
    int32_t *row_nparts = reinterpret_cast<int32_t *>(ws + L.row_nparts);
    int32_t *row_part0 = reinterpret_cast<int32_t *>(ws + L.row_part0);
    int32_t *row_item0 = reinterpret_cast<int32_t *>(ws + L.row_item0);
    TreeRow *tree_rows = reinterpret_cast<TreeRow *>(ws + L.tree_rows);
    TreeRow *tree_items = reinterpret_cast<TreeRow *>(ws + L.tree_items);
    int32_t *tree_pages = reinterpret_cast<int32_t *>(ws + L.tree_pages);

    if (tid == 0) {
        carry = carry_parts = 0;
        bad = special = even_cap = 0;
    }
    for (int32_t r = tid; r < R; r += kTreeThreads) s_end[r] = kNoneUnused;
    for (int32_t u = tid; u < U; u += kTreeThreads) s_count[u] = 0;
    ptx::pdl_wait_prior();
    // the main kernel may start its prologue now; it waits for this grid before it reads the schedule
    ptx::pdl_launch_dependents();

    if (kChunk && forms) {   // (none: no request, and so with bad offsets; the chunks' planner has just written them)
        bool any = false;
        for (int32_t b = tid; b < batch; b += kTreeThreads) any |= forms[b] != 0;
        if (!__syncthreads_or(any)) {
            for (int32_t v = tid; v <= U; v += kTreeThreads) unit_begin[v] = 0;
            if (tid == 0) {
                PlanHeader h = {};
                h.magic = kTreeMagic;
                h.batch = batch;
                h.s_q = tokens;
                h.max_pages = max_pages;
                h.num_units = U;
                *hdr = h;
            }
            return;
        }
    }

    // ---- every request's rows; with bad offsets no row belongs to any (all NaN)
    bool wrong = false;
    for (int32_t b = tid; b < batch; b += kTreeThreads) {
        const int32_t o0 = offsets[b], o1 = offsets[b + 1];
        // (a chunk's tokens are not counted)
        wrong |= !kChunk ? !tree_offsets_ok(o0, o1, b, R) : o0 < 0 || o0 > o1 || o1 > R || (b == 0 && o0 != 0);
    }
    wrong = __syncthreads_or(wrong) != 0;
    if (kChunk && !wrong) {   // a warp a request
        for (int32_t b = warp; b < batch; b += kTreeThreads / 32) {
            const int32_t o0 = offsets[b], n = forms && !forms[b] ? 0 : offsets[b + 1] - o0, len = seq_lens[b];
            int32_t most = 0;
            for (int32_t i = lane; i < n; i += 32) {
                TreeRow row;
                const int32_t p = chunk_row(len, n, i, b, max_pages, &row);
                tree_rows[o0 + i] = row;
                s_end[o0 + i] = p > 0 ? row.context : p;
                most = max(most, p);
                if (p == kNoneBad) {
                    bad = MLA_DEV_BAD_SEQ_LEN;
                    special = 1;
                }
            }
            most = __reduce_max_sync(0xffffffffu, most);
            if (lane == 0) tree_pages[b] = most;
        }
    } else if (wrong) {
        for (int32_t r = tid; r < R; r += kTreeThreads) s_end[r] = kNoneBad;
        for (int32_t b = tid; b < batch; b += kTreeThreads) tree_pages[b] = 0;
        if (tid == 0) {
            bad = MLA_DEV_BAD_OFFSETS;
            special = 1;
        }
    } else {
        // one warp per request, four requests in flight: lane i has its nodes i and i + 32
        constexpr int kFly = 4, kWarps = kTreeThreads / 32;
        for (int32_t b0 = warp; b0 < batch; b0 += kFly * kWarps) {
            int32_t o0[kFly], nodes[kFly], len[kFly];
            uint64_t mask[kFly][2];
#pragma unroll
            for (int j = 0; j < kFly; ++j) {
                const int32_t b = b0 + j * kWarps;
                o0[j] = b < batch ? offsets[b] : 0;
                nodes[j] = b < batch ? offsets[b + 1] - o0[j] : 0;
                len[j] = b < batch ? seq_lens[b] : 0;
            }
#pragma unroll
            for (int j = 0; j < kFly; ++j)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    mask[j][k] = lane + 32 * k < nodes[j] ? masks[o0[j] + lane + 32 * k] : 0;
#pragma unroll
            for (int j = 0; j < kFly; ++j) {
                const int32_t b = b0 + j * kWarps;
                int32_t most = 0;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int32_t i = lane + 32 * k;
                    if (i >= nodes[j]) continue;
                    TreeRow row;
                    const int32_t p = tree_row(len[j], nodes[j], b, mask[j][k], max_pages, &row);
                    tree_rows[o0[j] + i] = row;
                    s_end[o0[j] + i] = p > 0 ? tree_end(row.context, row.mask) : p;
                    most = max(most, p);
                    if (p == kNoneBad) bad = MLA_DEV_BAD_SEQ_LEN;
                    if (p < 0) special = 1;
                }
                most = __reduce_max_sync(0xffffffffu, most);
                if (lane == 0 && b < batch) tree_pages[b] = most;
            }
        }
    }
    __syncthreads();

    if constexpr (kChunk)
        for (int32_t r = tid; r < R + MLA_ROPE_TABLE_FLOATS; r += kTreeThreads) zeros[r] = r < R && s_end[r] <= 0 ? -1 : 0;

    // ---- total cost and largest row
    {
        int64_t sum = 0, most = 0;
        for (int32_t r = tid; r < R; r += kTreeThreads) {
            const int64_t c = row_cost(pages(r));
            sum += c;
            most = c > most ? c : most;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const int64_t m = __shfl_xor_sync(0xffffffffu, most, o);
            most = m > most ? m : most;
        }
        if (lane == 0) {
            warp_sums[warp] = sum;
            warp_most[warp] = most;
        }
    }
    __syncthreads();
    static_assert(kTreeThreads == 512, "16 warps' sums, twice over a warp");
    int64_t total = warp_sums[lane & 15], longest = warp_most[lane & 15];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, o);
        const int64_t m = __shfl_xor_sync(0xffffffffu, longest, o);
        longest = m > longest ? m : longest;
    }
    __syncthreads();
    const int64_t target = total > 0 ? (total + U - 1) / U : 1;

    // ---- whole rows: deal them in waves (not tried when one row alone is too long for it)
    bool whole = try_whole(U, longest, total, target);
    if (whole) {
        // keys: a unit's by load, a row's by cost; all distinct within a wave.  First every row's
        // rank in its wave, the longest first (the keys in s_row, the ranks in s_unit).
        for (int32_t r = tid; r < R; r += kTreeThreads)
            s_row[r] = (int32_t)((uint32_t)row_cost(pages(r)) << 8 | (uint32_t)(255 - r % U));
        if (tid < kMaxUnits) unit_key[tid] = tid < U ? (uint32_t)tid : 0xffffffffu;
        __syncthreads();
        for (int32_t r = tid; r < R; r += kTreeThreads) {
            const int32_t r0 = r / U * U, n = min(U, R - r0);
            const uint32_t mine = (uint32_t)s_row[r];
            int32_t rank = 0;
#pragma unroll 8
            for (int32_t j = 0; j < n; ++j) rank += (uint32_t)s_row[r0 + j] > mine;
            s_unit[r] = rank;
        }
        __syncthreads();
        for (int32_t r0 = 0; r0 < R; r0 += U) {
            // units by load: four threads each count a quarter of the keys
            if (tid < 4 * kMaxUnits) {
                const int32_t u = tid >> 2;
                const uint32_t mine = unit_key[u];
                int32_t rank = 0;
#pragma unroll
                for (int v = 0; v < kMaxUnits / 16; ++v) {
                    const uint4 k = reinterpret_cast<const uint4 *>(unit_key)[v * 4 + (tid & 3)];
                    rank += (k.x < mine) + (k.y < mine) + (k.z < mine) + (k.w < mine);
                }
                rank += __shfl_xor_sync(0xffffffffu, rank, 1);
                rank += __shfl_xor_sync(0xffffffffu, rank, 2);
                if ((tid & 3) == 0 && u < U) s_rank[rank] = u;
            }
            __syncthreads();
            const int32_t r = r0 + tid;
            if (tid < U && r < R) {
                const int32_t u = s_rank[s_unit[r]];
                s_unit[r] = u;
                if (pages(r) > 0) {
                    unit_key[u] += (uint32_t)s_row[r] & ~255u;
                    s_row[r] = s_count[u]++;
                }
            }
            __syncthreads();
        }
        uint32_t most = 0;
#pragma unroll 16
        for (int32_t u = 0; u < U; ++u) most = max(most, unit_key[u]);
        whole = keep_whole(most >> 8, target);
    }

    // ---- even pieces: the smallest cap under which every piece has a unit of its own
    if (!whole && R <= U && total > 0) {
        if (warp == 0) {
            int32_t lo = kEvenPages, hi = even_most(longest, target);
            auto fits = [&](int32_t c) {
                int32_t pieces = 0;
                for (int32_t r = lane; r < R; r += 32) pieces += even_pieces(pages(r), c);
                return __reduce_add_sync(0xffffffffu, pieces) <= U;
            };
            const bool ok = hi >= lo && fits(hi);
            while (ok && lo < hi) {
                const int32_t mid = lo + (hi - lo) / 2;
                if (fits(mid)) hi = mid;
                else lo = mid + 1;
            }
            if (lane == 0) even_cap = ok ? lo : 0;
        }
        __syncthreads();
    }
    const int32_t cap = even_cap;
    const bool even = cap > 0;

    // an item's place in the schedule
    auto put = [&](int32_t at, int32_t unit, int32_t r, int32_t pg0, int32_t pg1, int32_t end, int32_t part,
                   const TreeRow &row) {
        items[at] = WorkItem{r, pg0 * kPage, min(pg1 * kPage, end), part};
        item_unit[at] = unit;
        tree_items[at] = row;
    };
    int32_t num_items = 0, num_parts = 0;
    if (whole) {
        if (tid < U) {
            int32_t at = 0;
            for (int32_t u = 0; u < tid; ++u) at += s_count[u];
            s_begin[tid] = at;
            unit_begin[tid] = at;
            if (tid == U - 1) {
                s_begin[U] = at + s_count[tid];
                unit_begin[U] = s_begin[U];
            }
        }
        __syncthreads();
        num_items = s_begin[U];
        for (int32_t r = tid; r < R; r += kTreeThreads) {
            const int32_t p = pages(r);
            row_nparts[r] = p > 0 ? 1 : none_parts(p);
            row_part0[r] = -1;
            const int32_t at = p > 0 ? s_begin[s_unit[r]] + s_row[r] : -1;
            row_item0[r] = at;
            if (p > 0) put(at, s_unit[r], r, 0, p, s_end[r], -1, tree_rows[r]);
        }
    } else if (even) {
        // ---- even pieces, one per unit, in token order
        for (int32_t r = tid; r < R; r += kTreeThreads) s_row[r] = even_pieces(pages(r), cap);
        __syncthreads();
        for (int32_t r = tid; r < R; r += kTreeThreads) {
            const int32_t p = pages(r), k = s_row[r];
            TreeRow row = {};
            if (p > 0) row = tree_rows[r];
            int32_t first = 0, part0 = 0;
#pragma unroll 8
            for (int32_t j = 0; j < r; ++j) {
                first += s_row[j];
                part0 += s_row[j] > 1 ? s_row[j] : 0;
            }
            row_nparts[r] = p > 0 ? k : none_parts(p);
            row_part0[r] = k > 1 ? part0 : -1;
            row_item0[r] = p > 0 ? first : -1;
            for (int32_t i = 0; i < k; ++i)
                put(first + i, first + i, r, even_page(p, i, k), even_page(p, i + 1, k), s_end[r],
                    k > 1 ? part0 + i : -1, row);
            if (r == R - 1) {
                carry = first + k;
                carry_parts = part0 + (k > 1 ? k : 0);
            }
        }
        __syncthreads();
        num_items = (int32_t)carry;
        num_parts = (int32_t)carry_parts;
        for (int32_t v = tid; v <= U; v += kTreeThreads) unit_begin[v] = min(v, num_items);
    } else {
        // ---- cut rows: positions on the line
        for (int32_t base = 0; base < R; base += kTreeThreads) {
            const int32_t k = base + tid;
            const int32_t r = k < R ? tree_line(k, R, U) : 0;
            const int64_t c = k < R ? row_cost(pages(r)) : 0;
            const int64_t incl = block_scan(c, warp_sums);
            if (k < R) s_pos[r] = carry + incl - c;
            __syncthreads();
            if (tid == kTreeThreads - 1) carry += incl;
            __syncthreads();
        }
        if (tid == 0) carry = 0;
        __syncthreads();
        // the pieces in line order: their units and rows, and each row's first partial
        int32_t my_part0 = -1;   // of the thread's row, if it has one alone
        for (int32_t base = 0; base < R; base += kTreeThreads) {
            const int32_t k = base + tid;
            const int32_t r = k < R ? tree_line(k, R, U) : 0;
            const int32_t n = k < R ? cut_row(s_pos[r], pages(r), target, U, true, NoEmit{}) : 0;
            // pieces and partials in one sum (both far below 2^31)
            const int64_t both = (int64_t)n | (int64_t)(n > 1 ? n : 0) << 32;
            const int64_t incl = block_scan(both, warp_sums);
            if (k < R) {
                const int32_t first = (int32_t)carry + (int32_t)(incl & 0xffffffff) - n;
                my_part0 = n > 1 ? (int32_t)carry_parts + (int32_t)(incl >> 32) - n : -1;
                row_item0[r] = n > 0 ? first : -1;
                row_nparts[r] = n > 0 ? n : none_parts(pages(r));
                row_part0[r] = my_part0;
                cut_row(s_pos[r], pages(r), target, U, true, [&](int32_t i, int32_t, int32_t, int32_t unit) {
                    s_unit[first + i] = unit;
                    s_row[first + i] = r;
                });
            }
            __syncthreads();
            if (tid == kTreeThreads - 1) {
                carry += incl & 0xffffffff;
                carry_parts += incl >> 32;
            }
            __syncthreads();
        }
        num_items = (int32_t)carry;
        num_parts = (int32_t)carry_parts;
        // s_begin[u] = first piece whose unit is >= u (units are non-decreasing along the line)
        for (int32_t i = tid; i < num_items; i += kTreeThreads) {
            const int32_t u = s_unit[i], before = i > 0 ? s_unit[i - 1] : -1;
            for (int32_t v = before + 1; v <= u; ++v) s_begin[v] = i;
            if (i == num_items - 1)
                for (int32_t v = u + 1; v <= U; ++v) s_begin[v] = num_items;
        }
        if (num_items == 0)
            for (int32_t v = tid; v <= U; v += kTreeThreads) s_begin[v] = 0;
        __syncthreads();
        for (int32_t v = tid; v <= U; v += kTreeThreads) unit_begin[v] = s_begin[v];
        // each unit's pieces in token order (a unit has one piece of a row at most)
        for (int32_t k = tid; k < R; k += kTreeThreads) {
            const int32_t r = tree_line(k, R, U);
            if (pages(r) <= 0) continue;
            const TreeRow row = tree_rows[r];
            const int32_t end = s_end[r], part0 = R <= kTreeThreads ? my_part0 : row_part0[r];
            cut_row(s_pos[r], pages(r), target, U, true, [&](int32_t i, int32_t pg0, int32_t pg1, int32_t unit) {
                int32_t at = s_begin[unit];
                for (int32_t j = s_begin[unit]; j < s_begin[unit + 1]; ++j) at += s_row[j] < r;
                put(at, unit, r, pg0, pg1, end, part0 >= 0 ? part0 + i : -1, row);
            });
        }
    }
    if (tid == 0) {
        PlanHeader h;
        h.magic = kTreeMagic;
        h.batch = batch;
        h.s_q = tokens;
        h.max_pages = max_pages;
        h.num_units = U;
        h.num_rows = R;
        h.max_items = L.max_items;
        h.num_items = num_items;
        h.num_parts = num_parts;
        h.status = bad;
        h.split = (whole ? 0 : 1) | (special ? 2 : 0);
        h.min_split = kMinSplitPages;
        h.total_cost = total;
        h.target = target;
        *hdr = h;
    }
}

}  // namespace

// Host twin of mla_tree_plan_kernel (the same integer arithmetic, sequential).
mla_status tree_plan_host(const mla_ragged *prob, const int32_t *seq_lens, const int32_t *offsets,
                          const uint64_t *masks, int32_t num_units, uint8_t *ws) {
    const int32_t batch = prob->batch, R = prob->tokens, U = num_units;
    const PlanLayout L = make_layout(R, U, batch);
    WorkItem *items = reinterpret_cast<WorkItem *>(ws + L.items);
    int32_t *item_unit = reinterpret_cast<int32_t *>(ws + L.item_unit);
    int32_t *unit_begin = reinterpret_cast<int32_t *>(ws + L.unit_begin);
    int32_t *row_nparts = reinterpret_cast<int32_t *>(ws + L.row_nparts);
    int32_t *row_part0 = reinterpret_cast<int32_t *>(ws + L.row_part0);
    int32_t *row_item0 = reinterpret_cast<int32_t *>(ws + L.row_item0);
    TreeRow *rows = reinterpret_cast<TreeRow *>(ws + L.tree_rows);
    TreeRow *tree_items = reinterpret_cast<TreeRow *>(ws + L.tree_items);
    int32_t *tree_pages = reinterpret_cast<int32_t *>(ws + L.tree_pages);
    PlanHeader h = {};
    std::vector<int32_t> pages((size_t)R, kNoneUnused);
    bool wrong = false;
    for (int32_t b = 0; b < batch; ++b) wrong |= !tree_offsets_ok(offsets[b], offsets[b + 1], b, R);
    if (wrong) {
        h.status = MLA_DEV_BAD_OFFSETS;
        h.split = 2;
        std::fill(pages.begin(), pages.end(), kNoneBad);
    }
    for (int32_t b = 0; b < batch; ++b) {
        tree_pages[b] = 0;
        if (wrong) continue;
        const int32_t nodes = offsets[b + 1] - offsets[b];
        for (int32_t r = offsets[b]; r < offsets[b + 1]; ++r) {
            pages[r] = tree_row(seq_lens[b], nodes, b, masks[r], prob->max_pages_per_seq, &rows[r]);
            tree_pages[b] = std::max(tree_pages[b], pages[r]);
            if (pages[r] == kNoneBad) h.status = MLA_DEV_BAD_SEQ_LEN;
            if (pages[r] < 0) h.split = 2;
        }
    }
    int64_t total = 0, longest = 0;
    for (int32_t p : pages) {
        total += row_cost(p);
        longest = std::max(longest, row_cost(p));
    }
    const int64_t target = total > 0 ? (total + U - 1) / U : 1;
    std::vector<std::vector<WorkItem>> lists((size_t)U);
    std::vector<int64_t> load((size_t)U, 0);
    bool whole = try_whole(U, longest, total, target);
    if (whole) {
        std::vector<int32_t> units((size_t)U), wave;
        for (int32_t r0 = 0; r0 < R; r0 += U) {
            wave.clear();
            for (int32_t r = r0; r < std::min(R, r0 + U); ++r) wave.push_back(r);
            for (int32_t u = 0; u < U; ++u) units[u] = u;
            std::stable_sort(units.begin(), units.end(), [&](int32_t a, int32_t b) { return load[a] < load[b]; });
            std::stable_sort(wave.begin(), wave.end(),
                             [&](int32_t a, int32_t b) { return std::max(pages[a], 0) > std::max(pages[b], 0); });
            for (size_t i = 0; i < wave.size(); ++i) {
                const int32_t r = wave[i];
                if (pages[r] <= 0) continue;
                lists[units[i]].push_back({r, 0, tree_end(rows[r].context, rows[r].mask), -1});
                load[units[i]] += row_cost(pages[r]);
            }
        }
        whole = keep_whole(*std::max_element(load.begin(), load.end()), target);
    }
    bool even = !whole && R <= U && total > 0;
    int32_t cap = 0;
    if (even) {
        int32_t lo = kEvenPages, hi = even_most(longest, target);
        auto fits = [&](int32_t c) {
            int64_t pieces = 0;
            for (int32_t p : pages) pieces += even_pieces(p, c);
            return pieces <= U;
        };
        even = hi >= lo && fits(hi);
        while (even && lo < hi) {
            const int32_t mid = lo + (hi - lo) / 2;
            if (fits(mid)) hi = mid;
            else lo = mid + 1;
        }
        cap = lo;
    }
    for (int32_t r = 0; r < R; ++r) {
        row_nparts[r] = pages[r] > 0 ? 1 : none_parts(pages[r]);
        row_part0[r] = row_item0[r] = -1;
    }
    if (even) {
        for (auto &l : lists) l.clear();
        int32_t unit = 0;
        for (int32_t r = 0; r < R; ++r) {
            const int32_t p = pages[r], k = even_pieces(p, cap);
            if (k > 0) row_item0[r] = unit;
            if (k > 1) {
                row_nparts[r] = k;
                row_part0[r] = h.num_parts;
                h.num_parts += k;
            }
            const int32_t end = p > 0 ? tree_end(rows[r].context, rows[r].mask) : 0;
            for (int32_t i = 0; i < k; ++i)
                lists[unit++].push_back({r, even_page(p, i, k) * kPage, std::min(even_page(p, i + 1, k) * kPage, end),
                                         k > 1 ? row_part0[r] + i : -1});
        }
    } else if (!whole) {
        for (auto &l : lists) l.clear();
        int64_t at = 0;
        int32_t n_items = 0;
        for (int32_t k = 0; k < R; ++k) {
            const int32_t r = tree_line(k, R, U), p = pages[r];
            const int32_t n = cut_row(at, p, target, U, true, NoEmit{});
            if (n > 0) row_item0[r] = n_items;
            if (n > 1) {
                row_nparts[r] = n;
                row_part0[r] = h.num_parts;
                h.num_parts += n;
            }
            const int32_t end = p > 0 ? tree_end(rows[r].context, rows[r].mask) : 0;
            cut_row(at, p, target, U, true, [&](int32_t i, int32_t pg0, int32_t pg1, int32_t unit) {
                lists[unit].push_back({r, pg0 * kPage, std::min(pg1 * kPage, end), n > 1 ? row_part0[r] + i : -1});
            });
            n_items += n;
            at += row_cost(p);
        }
        for (auto &l : lists)
            std::sort(l.begin(), l.end(), [](const WorkItem &a, const WorkItem &b) { return a.row < b.row; });
    }
    for (int32_t u = 0; u < U; ++u) {
        unit_begin[u] = h.num_items;
        for (const WorkItem &it : lists[u]) {
            if (whole) row_item0[it.row] = h.num_items;
            items[h.num_items] = it;
            tree_items[h.num_items] = rows[it.row];
            item_unit[h.num_items++] = u;
        }
    }
    unit_begin[U] = h.num_items;
    h.magic = kTreeMagic;
    h.batch = batch;
    h.s_q = R;
    h.max_pages = prob->max_pages_per_seq;
    h.num_units = U;
    h.num_rows = R;
    h.max_items = L.max_items;
    h.split |= whole ? 0 : 1;
    h.min_split = kMinSplitPages;
    h.total_cost = total;
    h.target = target;
    *reinterpret_cast<PlanHeader *>(ws) = h;
    return MLA_OK;
}

bool tree_plan_fits(int32_t rows, int32_t units) { return tree_plan_smem(rows, units) <= kMaxTreeSmem; }

// forms, zeros: of chunks (masks null); zeros has room for a position per token and a rotary table.
cudaError_t launch_tree_plan(const int32_t *seq_lens, const int32_t *offsets, const uint64_t *masks, const uint8_t *forms,
                             int32_t *zeros, void *ws, int32_t batch, int32_t tokens, int32_t max_pages,
                             int32_t num_units, cudaStream_t stream) {
    if (!tree_plan_fits(tokens, num_units)) return cudaErrorInvalidValue;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    // the attribute belongs to the device: set once on each
    static std::mutex mutex;
    static bool set[64];
    {
        std::lock_guard<std::mutex> lock(mutex);
        if (!set[dev]) {
            for (auto *k : {mla_tree_plan_kernel<false>, mla_tree_plan_kernel<true>})
                if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxTreeSmem)) !=
                    cudaSuccess)
                    return e;
            set[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kTreeThreads);
    cfg.dynamicSmemBytes = tree_plan_smem(tokens, num_units);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    auto *kernel = masks ? mla_tree_plan_kernel<false> : mla_tree_plan_kernel<true>;
    return cudaLaunchKernelEx(&cfg, kernel, seq_lens, offsets, masks, forms, zeros,
                              static_cast<uint8_t *>(ws), batch, tokens, max_pages, num_units);
}

}  // namespace mla
