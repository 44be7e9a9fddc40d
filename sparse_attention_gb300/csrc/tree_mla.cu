// tree_mla.cu -- latent attention of a step's new rows over everything they
// see in a (paged or contiguous) cache: the committed rows and, by a bit mask,
// the drafted rows of the same sequence.
//
// With 64 heads on one cached stream, two new rows (nodes) make 128 query
// rows: the M of a CTA pair's tcgen05 tile.  A pair takes an item (sequence,
// node pair) and walks its cache in tiles of 128 positions:
//   S[128 q, 128 pos] = Q K^T     9 chunks of 64 dims; each CTA stages its
//                                 node's 64 query rows (72 KiB, resident) and
//                                 64 of the tile's positions
//   P = 2^(S c - m)               the running maximum m of a row moves only
//                                 when a score exceeds it by 2^8 (then O is
//                                 rescaled), so sums and weights stay far from
//                                 both ends of fp32
//                                 P is rounded to bf16 for the product, the
//                                 MMA's type, and its sum taken before, in
//                                 fp32: an error of half a bf16 step of a
//                                 weight, like the result's own rounding (fp32
//                                 weights would need TF32 MMAs of half the rate
//                                 and twice the shared memory)
//   O[128 q, 512] += P V          two N = 256 halves; each CTA stages, for all
//                                 128 positions, the 128 dims of each half
//                                 whose columns it supplies
// O (256 TMEM columns) and two S tiles (64 columns each) live in each CTA's
// TMEM: rows of its node, lanes 0-63 the first half of the columns, lanes
// 64-127 the second.  Nothing but barriers crosses between the CTAs, and each
// cached row feeds 128 query rows.  S of tile g + 1 is issued before PV of
// tile g, so the softmax of a tile runs under the tensor work of the next.
//
// The value half of a CTA's positions is staged twice (once as K, once in
// V's dims-by-position split): a pair's K and V differ in which operand half
// a CTA has to hold, and descriptors mean the same offset in both.
//
// Roles of a CTA's 9 warps: K and Q loads, MMA (rank 0 only), V loads,
// fix-up, four softmax / epilogue warps (a thread per TMEM lane, so two
// threads share a query row, 64 positions each), and one that walks the
// pair's share of the work and publishes its segments.  Tiles that reach
// past the committed rows go through the fix-up warp, which zeroes V rows past
// the sequence (a page's leftovers may hold anything, and 0 * NaN is NaN) and
// values of drafted rows that are not finite.  A row that does not see such a
// row gets nothing of it; one that does gets NaN through its score, which is
// NaN or infinite: +inf by the subtraction of the maximum, -inf (an infinity
// against the query's sign) by a look at the row itself.
//
// Work: the items' tiles, plus kItemCost tiles per item for its start and
// end, laid end to end and cut into equal shares, one per pair (after whole
// items in turn where that saves HBM reads, see plan_rounds).  An item cut by
// a share's end leaves fp32 partial results, which tree_merge_kernel joins in
// order.
//
// Bounds.  A row pair's tile is 36 MMAs of N = 128 (37 cycles each) and 16 of
// N = 256 (65): 2,372 cycles for 35.7 MFLOP, 92 % of the tensor rate; a single
// row leaves rank 1's half empty and is bound by HBM (121 flop a byte).
// Measured, in single calls and in a loop that the power cap slows: 16 trees
// of 64 over 8,192 rows 0.64-0.66 ms = 1,770-1,820 TFLOP/s (1,907 measured
// peak) and 0.73-0.75 ms = 1,560-1,600 (1,698 sustained); 64 single rows over
// 32,768 each 0.37-0.38 ms = 6.4-6.6 TB/s (6.78 measured copy) and 0.41-0.43
// ms; one tree of 8 over 1,500 rows 17 us with the merge.
#include <algorithm>
#include <atomic>

#include "internal.h"
#include "ptx.cuh"
#include "tree.h"

namespace dsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kTile = 128;                   // positions per tile
constexpr int kItemCost = 3;                 // an item's start and end, in tiles
constexpr int kThreads = 288;
constexpr int kChunkBytes = 64 * 128;        // 64 rows x 64 dims
constexpr int kQChunks = kDQK / 64;          // 9
constexpr int kGroup = 3;                    // chunks per K stage
constexpr int kKStages = 3;                  // a whole tile of K ..
constexpr int kVStages = 2;                  // .. and of V: a stage is 128 positions x 128 dims of one half
constexpr int kKBytes = kGroup * kChunkBytes, kVBytes = 4 * kChunkBytes;
constexpr uint32_t kOCol = 0, kSCol = 256;   // TMEM columns
constexpr int kMaxPairs = 96;                 // CTA pairs of a launch
constexpr int kPlanSeqs = 256;               // sequences of a call whose items may go round the pairs
constexpr int kSegs = 4;                     // segments published ahead
constexpr int64_t kSharedBytes = int64_t(48) << 20;   // cached rows that L2 keeps for pairs apart in a sequence
constexpr int kRoundPart = 48;               // units per pair below which rounds do not pay
constexpr float kRescale = 8.f;              // log2

struct Plan {
    int64_t lo[kMaxPairs + 1];   // pair k's share of the cut items: units [lo[k], lo[k + 1])
    int64_t start_u;             // the share's first sequence, and where its items begin
    int32_t start_b, rounds;     // whole items that every pair takes before
};

// One item's tiles [t0, t1) of a pair's chunk.
struct Seg {
    int32_t b, row, c, len, i0, rows, t0, t1, tiles;
    int64_t u0;                  // the unit of tile 0, for a piece of a cut item
    __device__ bool whole() const { return t0 == 0 && t1 == tiles; }
};

struct Smem {
    alignas(1024) uint8_t q[kQChunks * kChunkBytes];
    alignas(1024) uint8_t k[kKStages * kKBytes];
    alignas(1024) uint8_t v[kVStages * kVBytes];
    alignas(1024) uint8_t p[2 * kChunkBytes];
    alignas(8) uint64_t kfull[kKStages], kempty[kKStages], vfull[kVStages], vempty[kVStages], vloc[kVStages];
    uint64_t qfull, qempty, sfull[2], sempty[2], pfull, pvdone, ofree, segfull[kSegs], segempty[kSegs];
    Plan plan;
    Seg seg[kSegs];
    int64_t scan[kThreads / 32];
    int32_t longest[kThreads / 32];
    float xch[2][128];
    int32_t bad[4];
    uint32_t lost[4];            // softmax warps: 1 + the last segment with a score of -inf past the committed rows
    uint32_t tmem;
};
static_assert(sizeof(Smem) <= 232448, "one CTA's shared memory");

struct Args {
    BatchDev bd;
    PagesDev pg;
    const uint64_t* mask;
    const uint16_t* kv;
    float scale_log2;
    uint16_t* out;
    float* lse;
    int4* meta;          // [pairs]: row, rows, last and first pair of the cut item that a pair begins or lies in
    float* part_lse;     // [2 * pairs][128]
    float* part_o;       // [2 * pairs][2 CTAs][4 warps][64 groups of 4 columns][32 lanes][4]
    int32_t* status;
    int32_t rows_total;  // cache rows
    bool may_round;      // the bounds allow plan_rounds
    bool ahead;          // a sequence's rows are read by one pair only
};

__device__ __forceinline__ int64_t seq_units(const SeqInfo& s) {
    return (int64_t)((s.nq + 1) >> 1) * (((s.ctx + kTile - 1) / kTile) + kItemCost);
}

// Walks the segments of a pair (a warp; lanes hold 32 sequences' lengths):
// first every pairs-th item, whole, then its share of the others.
struct SegIter {
    const Args& a;
    const Plan& plan;
    const int32_t pair, pairs;
    int32_t round = 0, first = 0;        // round, and the first item of sequence b, while items are whole
    int32_t b = 0, p = 0, b0 = -64;
    int64_t u = 0;
    int32_t w_q0 = 0, w_nq = 0, w_ctx = 0;
    __device__ SegIter(const Args& args, const Plan& pl, int32_t pair_, int32_t pairs_)
        : a(args), plan(pl), pair(pair_), pairs(pairs_) {
        if (plan.rounds == 0) begin_share();
    }

    __device__ void begin_share() {
        b = plan.start_b;
        u = plan.start_u;
        p = 0;
    }

    // new rows, length and first packed row of sequence b
    __device__ void lengths(int32_t& nq, int32_t& ctx, int32_t& q0) {
        if (b < b0 || b >= b0 + 32) {
            b0 = b;
            const int mine = b0 + (int)lane_id();
            SeqInfo q{0, 0, 0};
            if (mine >= a.bd.B || !load_seq(a.bd, mine, nullptr, q)) q.nq = 0;
            w_q0 = q.q0, w_nq = q.nq, w_ctx = q.ctx;
        }
        nq = __shfl_sync(0xffffffffu, w_nq, b - b0);
        ctx = __shfl_sync(0xffffffffu, w_ctx, b - b0);
        q0 = __shfl_sync(0xffffffffu, w_q0, b - b0);
    }

    __device__ void fill(Seg& s, int32_t item, int32_t nq, int32_t ctx, int32_t q0) const {
        s.b = b;
        s.i0 = 2 * item;
        s.row = q0 + s.i0;
        s.rows = min(2, nq - s.i0);
        s.c = ctx - nq;
        s.len = ctx;
        s.tiles = (ctx + kTile - 1) / kTile;
    }

    __device__ bool next(Seg& s) {
        int32_t nq, ctx, q0;
        while (round < plan.rounds) {
            if (b >= a.bd.B) {                   // lengths that change under the call
                round = plan.rounds;
                begin_share();
                break;
            }
            lengths(nq, ctx, q0);
            const int32_t item = round * pairs + pair - first, items = (nq + 1) >> 1;
            if (item >= items) {
                first += items;
                ++b;
                continue;
            }
            fill(s, item, nq, ctx, q0);
            s.t0 = 0;
            s.t1 = s.tiles;
            if (++round == plan.rounds) begin_share();
            return true;
        }
        const int64_t lo = plan.lo[pair], hi = plan.lo[pair + 1];
        for (; b < a.bd.B; ++b, p = 0) {
            lengths(nq, ctx, q0);
            if (nq == 0) continue;
            const int32_t tiles = (ctx + kTile - 1) / kTile, per = tiles + kItemCost, items = (nq + 1) >> 1;
            if (p == 0 && lo > u) p = (uint32_t)(lo - u) / (uint32_t)per;   // < items: lo lies in the share's first sequence
            while (p < items) {
                const int64_t u0 = u + (int64_t)p * per + kItemCost;
                if (u0 - kItemCost >= hi) return false;
                s.t0 = (int32_t)max((int64_t)0, min((int64_t)tiles, lo - u0));
                s.t1 = (int32_t)max((int64_t)0, min((int64_t)tiles, hi - u0));
                ++p;
                if (s.t1 > s.t0) {
                    fill(s, p - 1, nq, ctx, q0);
                    s.u0 = u0;
                    return true;
                }
            }
            u += (int64_t)items * per;
        }
        return false;
    }
};

// The least work worth a pair of its own, in units: a tile takes 1.2 us (2 us
// among the first) and a piece 0.17 us more in the merge, so an item of N
// tiles alone on the GPU is done soonest in pieces of about sqrt(N / 4)
// (1 x 8,000 rows: 18.9 us in pieces of 4 tiles, 23.6 of 1; 1 x 1,500: 14.7 in
// pieces of 1, 16.9 of 2 and of 4).
__device__ __forceinline__ int least_chunk(int tiles) {
    int c = 1;
    while (4 * (c + 1) * (c + 1) <= tiles + 2) ++c;
    return c;
}

__device__ __forceinline__ int32_t warp_scan_i32(int32_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t n = __shfl_up_sync(0xffffffffu, v, o);
        if ((int)lane_id() >= o) v += n;
    }
    return v;
}

// Whole items go round the pairs first when several node pairs share a
// sequence and the caches exceed what L2 keeps: the pairs then walk the same
// one or two sequences side by side, and a cached row comes from HBM once (in
// equal contiguous shares every sequence is being read at the same time: 3.0
// GB of HBM reads for 0.23 GB of inputs, 16 trees of 64 over 8,192 rows 0.79
// ms; 0.66 with rounds; 64 trees of 4 over 1,000 rows, 18 units a pair, lose 4
// of 50 us).  The shares of the items left over even out what the rounds gave.
// All threads; kPlanSeqs sequences at most, a thread each with its units and
// those before it.  Sets S.plan's rounds, shares and start; false: no rounds.
__device__ bool plan_rounds(const Args& a, Smem& S, const SeqInfo& q, int64_t units_before, int64_t units, int64_t all,
                            int pair, int pairs) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // the V ring is not in use yet
    int32_t* first = reinterpret_cast<int32_t*>(S.v);            // [B + 1] items before a sequence
    int32_t* per = first + kThreads + 1;                         // [B] units of its items
    int32_t* sums = per + kThreads;                              // [3][warps]
    const int32_t items = (q.nq + 1) >> 1;
    const int32_t incl = warp_scan_i32(items);
    // cached rows (64 at a time) of sequences that several items read
    const uint32_t rows = __reduce_add_sync(0xffffffffu, items > 1 ? (uint32_t)q.ctx >> 6 : 0u);
    if (lane == 31) {
        sums[warp] = incl;
        sums[16 + warp] = (int32_t)min(rows, 1u << 26);
    }
    __syncthreads();
    int32_t before = 0, total = 0, cached = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
        cached += sums[16 + w];
    }
    // (all the same for every thread)
    const int64_t part = (all + pairs - 1) / pairs;
    if ((int64_t)cached * 64 * 2 * kDQK <= kSharedBytes || total < pairs || part < kRoundPart) return false;
    first[tid] = before + incl - items;
    per[tid] = (q.ctx + kTile - 1) / kTile + kItemCost;
    if (tid == 0) first[kThreads] = total;
    __syncthreads();
    // thread k: what the rounds give pair k, which takes as many of them as
    // leave it no more than a quarter above its part of all (up to there the
    // saved reads are worth more: 24 ragged trees of up to 13 over 7,001 rows
    // 119 -> 113 us); all pairs take as many as the one that takes fewest
    const int64_t most = part + part / 4;
    auto given_by = [&](int n, int64_t& load) -> int {     // the rounds of n that fit, and their load
        load = 0;
        int b = 0, top = a.bd.B;
        while (b + 1 < top) {                    // the sequence of item tid
            const int mid = (b + top) >> 1;
            if (first[mid] <= tid) b = mid;
            else top = mid;
        }
        for (int r = 0; r < n; ++r) {
            const int32_t item = r * pairs + tid;
            while (first[b + 1] <= item) ++b;
            if (load + per[b] > most) return r;
            load += per[b];
        }
        return n;
    };
    int64_t load = 0;
    int rounds = total / pairs;
    const int fit = __reduce_min_sync(0xffffffffu, tid < pairs ? given_by(rounds, load) : rounds);
    if (lane == 0) sums[32 + warp] = fit;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) rounds = min(rounds, sums[32 + w]);
    if (rounds == 0) return false;
    if (rounds < total / pairs && tid < pairs) given_by(rounds, load);
    // shares of the rest, one behind the other
    if (tid < kMaxPairs) {
        // one unit at least, so that no pair inside a cut item is without a piece
        int64_t sum = tid < pairs ? max((int64_t)1, part - load) : 0, given = tid < pairs ? load : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t n = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += n;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) given += __shfl_xor_sync(0xffffffffu, given, o);
        if (lane == 31) {
            S.scan[warp] = sum;
            S.scan[4 + warp] = given;
        }
        S.plan.lo[tid + 1] = sum;
    }
    __syncthreads();
    if (tid < kMaxPairs) {
        int64_t rest = all, lower = 0;
        for (int w = 0; w < kMaxPairs / 32; ++w) {
            rest -= S.scan[4 + w];
            if (w < warp) lower += S.scan[w];
        }
        S.plan.lo[tid + 1] = min(rest, S.plan.lo[tid + 1] + lower);
    }
    __syncthreads();
    // units before the first item left over, then the sequence in which the
    // pair's share begins
    const int32_t rest_item = rounds * pairs;
    if (first[tid] <= rest_item && rest_item < first[tid + 1])
        S.scan[0] = units_before + (int64_t)(rest_item - first[tid]) * per[tid];
    if (tid == 0) {
        S.plan.lo[0] = 0;
        S.plan.rounds = rounds;
        S.plan.start_b = a.bd.B;
        if (rest_item >= total) S.scan[0] = all;
    }
    __syncthreads();
    const int64_t u = units_before - S.scan[0], lo = S.plan.lo[pair];
    if (u <= lo && lo < u + units) {
        S.plan.start_b = tid;
        S.plan.start_u = u;
    }
    return true;
}

// The pair's part of the work, by all threads of the CTA.
__device__ void make_plan(const Args& a, Smem& S, int pair, int pairs) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.bd.B + kThreads - 1) / kThreads;
    const int b_lo = min(a.bd.B, tid * per), b_hi = min(a.bd.B, b_lo + per);
    int64_t sum = 0;
    int tiles = 0;
    SeqInfo mine{0, 0, 0};
    for (int b = b_lo; b < b_hi; ++b) {
        SeqInfo q;
        if (!load_seq(a.bd, b, a.status, q) || q.nq == 0) continue;
        sum += seq_units(q);
        tiles = max(tiles, (q.ctx + kTile - 1) / kTile);
        mine = q;
    }
    tiles = __reduce_max_sync(0xffffffffu, tiles);
    if (lane == 0) S.longest[warp] = tiles;
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) S.scan[warp] = incl;
    __syncthreads();
    int64_t before = incl - sum, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += S.scan[w];
        all += S.scan[w];
    }
    if (a.may_round && plan_rounds(a, S, mine, before, sum, all, pair, pairs)) return;
    const int64_t even = all < (int64_t(1) << 30) ? (int64_t)(((uint32_t)all + pairs - 1) / (uint32_t)pairs)
                                                  : (all + pairs - 1) / pairs;
    int longest = 0;
    for (int w = 0; w < kThreads / 32; ++w) longest = max(longest, S.longest[w]);
    const int64_t chunk = max(even, (int64_t)least_chunk(longest));
    const int64_t lo = min(all, pair * chunk);
    if (tid <= pairs) S.plan.lo[tid] = min(all, tid * chunk);
    if (tid == 0) {
        S.plan.rounds = 0;
        if (lo >= all) S.plan.start_b = a.bd.B;
    }
    if (before <= lo && lo < before + sum) {
        int64_t u = before;
        S.plan.start_b = b_lo;
        S.plan.start_u = u;
        for (int b = b_lo; b + 1 < b_hi; ++b) {
            SeqInfo q;
            const int64_t w = load_seq(a.bd, b, nullptr, q) ? seq_units(q) : 0;
            if (lo < u + w) break;
            u += w;
            S.plan.start_b = b + 1;
            S.plan.start_u = u;
        }
    }
}

// First cache row of a box of positions at pos; past the sequence, or on a
// page outside the pool, the rows behind the cache (TMA fills zeros).
__device__ __forceinline__ int32_t box_row(const Args& a, const Seg& s, int32_t pos, bool& bad) {
    if (pos >= s.len) return a.rows_total;
    const int32_t r = cache_row(a.bd, a.pg, s.b, pos);
    if (r >= 0) return r;
    bad = true;
    return a.rows_total;
}

__device__ __forceinline__ bool past_committed(const Seg& s, int32_t t) { return (t + 1) * kTile > s.c; }

// Whether one of the new rows `rows` in the segment's tiles holds a NaN or an
// infinity; all lanes.  Called when a row past the committed ones scored -inf,
// which is seldom; a call, since the code of it inside the softmax role costs
// long calls 1-2 %, out of the way 0.5 % (16 trees of 64 over 8,192 rows).
__device__ __noinline__ bool any_not_finite(const Args& a, const Seg& s, uint64_t rows) {
#pragma unroll 1
    for (; rows; rows &= rows - 1u) {
        const int32_t pos = s.c + __ffsll((long long)rows) - 1;
        if (pos < s.t0 * kTile || pos >= s.t1 * kTile) continue;
        const int32_t at = cache_row(a.bd, a.pg, s.b, pos);
        if (at < 0) continue;                    // a bad page: latched, and nothing is written
        const uint4* row = reinterpret_cast<const uint4*>(a.kv + (int64_t)at * kDQK);
        bool hit = false;
#pragma unroll 1
        for (int k = (int)lane_id(); k < kDQK / 8; k += 32) {
            const uint4 v = row[k];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
                hit = hit || (w[q] & 0x7F80u) == 0x7F80u || (w[q] & 0x7F800000u) == 0x7F800000u;
        }
        if (__any_sync(0xffffffffu, hit)) return true;
    }
    return false;
}

// kKRows, kVRows: positions of a K box (of one chunk, or of a stage's three)
// and of a V box (of two).  Pages of 64 rows and more, and contiguous caches:
// boxes of 64; pages of 32: of 32; pages of 16: K boxes of 8 rows x 3 chunks,
// whose 8-row groups stay evenly spaced in a stage as a descriptor needs them
// (24 K and 16 V boxes a tile; boxes of one chunk of 16 rows, 36 and 32: 0.94
// instead of 0.89 ms for 16 trees of 64 over 8,192 rows).
template <int kKRows, int kVRows>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    tree_mla_kernel(const Args a, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem& S = *reinterpret_cast<Smem*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    pdl_launch_dependents();
    if (smem_u32(smem_raw) & 1023u) {            // the swizzle goes by address bits
        if (tid == 0) latch_status(a.status, DSA_ERR_INTERNAL);
        return;                                  // both CTAs: the same launch, the same offset
    }
    if (tid == kThreads - 32) {
        for (int i = 0; i < kKStages; ++i) {
            mbar_init(smem_u32(&S.kfull[i]), 2);
            mbar_init(smem_u32(&S.kempty[i]), 1);
        }
        for (int i = 0; i < kVStages; ++i) {
            mbar_init(smem_u32(&S.vfull[i]), 2);
            mbar_init(smem_u32(&S.vempty[i]), 1);
            mbar_init(smem_u32(&S.vloc[i]), 1);
        }
        mbar_init(smem_u32(&S.qfull), 2);
        mbar_init(smem_u32(&S.qempty), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&S.sfull[i]), 1);
            mbar_init(smem_u32(&S.sempty[i]), 8);
        }
        mbar_init(smem_u32(&S.pfull), 8);
        mbar_init(smem_u32(&S.pvdone), 1);
        mbar_init(smem_u32(&S.ofree), 8);
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(smem_u32(&S.segfull[i]), 1);
            mbar_init(smem_u32(&S.segempty[i]), rank == 0 ? 8 : 7);   // the warps that read segments
        }
        fence_mbar_init();
    }
    if (tid < 4) S.lost[tid] = 0u;
    if (warp == 1) tmem_alloc_pair(smem_u32(&S.tmem), 512);
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    __syncwarp();
    cluster_arrive();                            // the peer may use this CTA's barriers and TMEM ..
    pdl_wait();                                  // lengths, tables and inputs, and the scratch of an earlier call
    make_plan(a, S, pair, pairs);
    if (a.may_round) fence_proxy_async_smem();   // plan_rounds used the V ring
    tc_fence_before();
    __syncthreads();
    cluster_wait();                              // .. and this CTA the peer's
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    Seg s;
    bool ok = true;
    // the barrier at `b`'s offset in the CTA of rank 0
    auto lead = [&](uint64_t& b) -> uint32_t { return map_to_cluster_rank(smem_u32(&b), 0); };
    // bounded; a thread whose wait expired waits for nothing any more
    auto wait = [&](uint64_t& b, uint32_t parity) -> bool {
        if (ok && !mbar_wait_rolled(smem_u32(&b), parity)) {
            ok = false;
            latch_status(a.status, DSA_ERR_TIMEOUT);
        }
        return ok;
    };
    // the next segment that warp 8 published; false behind the last
    uint32_t segs_read = 0;
    auto next_seg = [&](Seg& to) -> bool {
        const uint32_t slot = segs_read & (kSegs - 1);
        wait(S.segfull[slot], (segs_read / kSegs) & 1);
        ok = __all_sync(0xffffffffu, ok);
        to = S.seg[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&S.segempty[slot]));
        ++segs_read;
        return ok && to.t1 > to.t0;
    };
    constexpr int kboxes = 64 / kKRows, vboxes = kTile / kVRows;     // per stage's positions
    constexpr int kChunksPerBox = kKRows == 32 ? 1 : kGroup;

    // MMAs are issued by one elected lane, which also waits: the tensor pipe
    // takes a K chunk's four MMAs in 150 cycles, less than a warp that waits
    // together, votes and branches to its issuing lane needs (4.5 us a tile
    // that way, of 1.3 us in the pipe).  Loads have that time: lane 0 waits,
    // then each lane issues a box.
    if (warp == 0) {
        // Q and K loads
        uint32_t g0 = 0, seg = 0;                // tiles and segments before this one
        for (; next_seg(s); g0 += s.t1 - s.t0, ++seg) {
            // first rows of the segment's boxes, 32 at a time
            const int32_t n = (s.t1 - s.t0) * kboxes;
            for (int32_t x0 = 0; ok && x0 < n; x0 += 32) {
                bool bad = false;
                const int32_t x = x0 + lane;
                const int32_t row =
                    box_row(a, s, (s.t0 + x / kboxes) * kTile + 64 * (int)rank + (x % kboxes) * kKRows, bad);
                for (int32_t y = 0; ok && y < 32 && x0 + y < n; y += kboxes) {
                    if (x0 + y == 0) {
                        // No row for this CTA: zeros, from behind the queries.
                        // Whatever lay there would do as well, but its products
                        // cost power, which holds the clock (64 x 1 row over
                        // 32,768 in a long loop: 438 us, 407 with zeros).
                        const int32_t q_row = (int)rank < s.rows ? (s.row + (int)rank) * kH : a.bd.total_q * kH;
                        if (lane == 0 && (seg == 0 || wait(S.qempty, (seg - 1) & 1)))
                            mbar_arrive_expect_tx_pair(lead(S.qfull), (uint32_t)sizeof(S.q));
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                        if (ok && lane < kQChunks)
                            tma_load_2d_pair(smem_u32(S.q + lane * kChunkBytes), &tm_q, lead(S.qfull), 64 * lane, q_row);
                    }
                    const uint32_t g = g0 + (x0 + y) / kboxes;
                    const int e = lane % kboxes, c = (lane / kboxes) * kChunksPerBox;    // a box each
                    const int32_t r = __shfl_sync(0xffffffffu, row, y + e);
#pragma unroll 1
                    for (int gr = 0; ok && gr < kKStages; ++gr) {
                        const uint32_t bar = lead(S.kfull[gr]);
                        if (lane == 0 && (g == 0 || wait(S.kempty[gr], (g - 1) & 1)))
                            mbar_arrive_expect_tx_pair(bar, kKBytes);
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                        if (ok && c < kGroup)
                            tma_load_3d_pair(smem_u32(S.k + gr * kKBytes + c * kChunkBytes +
                                                      e * kKRows * 128 * kChunksPerBox),
                                             &tm_k, bar, 0, r, kGroup * gr + c);
                    }
                    // Rows that no other pair reads come from HBM: the next
                    // tile's are brought to L2 while this one's are loaded
                    // (64 x 1 row over 32,768: 416 -> 399 us; with rows that
                    // several pairs share the same costs 4-7 %).
                    if (a.ahead) {
                        const int32_t next = y + kboxes + lane;
                        const int32_t r2 = __shfl_sync(0xffffffffu, row, next & 31);
                        if (lane < kboxes && next < 32 && x0 + next < n && r2 < a.rows_total)
                            prefetch_l2_bulk(a.kv + (int64_t)r2 * kDQK, min(kKRows, a.rows_total - r2) * 2 * kDQK);
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // MMA: S of tile g + 1, then PV of tile g
            constexpr uint32_t kIdS = idesc_bf16_f32(128, kTile), kIdO = idesc_bf16_f32(128, 256, false, true);
            // K stages: three chunks of 64 rows, or (boxes of 8 rows) eight
            // groups of 8 rows x three chunks; V stages: boxes of two 64-dim
            // blocks of vrows rows
            constexpr uint32_t ksbo = kKRows == 8 ? 1024 * kGroup : 1024;
            constexpr uint32_t kcstep = (kKRows == 8 ? 1024 : kChunkBytes) >> 4;
            // S of tile g; first / last of its segment (number seg)
            auto issue_s = [&](uint32_t g, bool first, bool last, uint32_t seg) {
                if (first && !wait(S.qfull, seg & 1)) return;
                const uint32_t buf = g & 1;
                if (g >= 2 && !wait(S.sempty[buf], ((g >> 1) - 1) & 1)) return;
                const uint64_t dq = sdesc_sw128(smem_u32(S.q), 0, 1024), dk = sdesc_sw128(smem_u32(S.k), 0, ksbo);
#pragma unroll 1
                for (int gr = 0; gr < kKStages; ++gr) {
                    if (!wait(S.kfull[gr], g & 1)) return;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < kGroup; ++c) {
                        const uint64_t da = dq + (kGroup * gr + c) * (kChunkBytes >> 4);
                        const uint64_t db = dk + gr * (kKBytes >> 4) + c * kcstep;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16_ss_pair(tmem + kSCol + 64 * buf, da + 2 * k, db + 2 * k, kIdS,
                                             (gr | c | k) != 0);
                    }
                    mma_commit_pair(smem_u32(&S.kempty[gr]));
                }
                mma_commit_pair(smem_u32(&S.sfull[buf]));
                if (last) mma_commit_pair(smem_u32(&S.qempty));
            };
            auto issue_pv = [&](uint32_t g, bool first, uint32_t seg) {
                if (first && seg > 0 && !wait(S.ofree, (seg - 1) & 1)) return;
                if (!wait(S.pfull, g & 1)) return;
                tc_fence_after();
                const uint64_t dp = sdesc_sw128(smem_u32(S.p), 0, 1024), dv = sdesc_sw128(smem_u32(S.v), kVRows * 128, 1024);
#pragma unroll 1
                for (int j = 0; j < kVStages; ++j) {
                    if (!wait(S.vfull[j], g & 1)) return;
                    tc_fence_after();
                    const uint64_t db = dv + j * (kVBytes >> 4);
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        mma_bf16_ss_pair(tmem + kOCol + 128 * j, dp + (k >> 2) * (kChunkBytes >> 4) + 2 * (k & 3),
                                         db + 128 * k + 128 * ((16 * k) & -kVRows) / 16, kIdO, !first || k != 0);
                    mma_commit_pair(smem_u32(&S.vempty[j]));
                }
                mma_commit_pair(smem_u32(&S.pvdone));
            };
            Seg n;
            bool more = next_seg(n);
            uint32_t g = 0;
            if (more && elect_one()) issue_s(0, true, n.t1 - n.t0 == 1, 0);
            __syncwarp();
            ok = __all_sync(0xffffffffu, ok);
            for (uint32_t seg = 0; ok && more; ++seg) {
                s = n;
                more = next_seg(n);
                const int32_t tiles = s.t1 - s.t0;
                if (elect_one()) {
                    for (int32_t t = 0; ok && t < tiles; ++t) {
                        if (t + 1 < tiles) issue_s(g + t + 1, false, t + 2 == tiles, seg);
                        else if (more) issue_s(g + t + 1, true, n.t1 - n.t0 == 1, seg + 1);
                        if (ok) issue_pv(g + t, t == 0, seg);
                    }
                }
                __syncwarp();
                ok = __all_sync(0xffffffffu, ok);
                g += tiles;
            }
        }
    } else if (warp == 2) {
        // V loads
        uint32_t g0 = 0, seg = 0;
        for (; next_seg(s); g0 += s.t1 - s.t0, ++seg) {
            const int32_t n = (s.t1 - s.t0) * vboxes;
            bool bad = false;
            for (int32_t x0 = 0; ok && x0 < n; x0 += 32) {
                const int32_t x = x0 + lane;
                const int32_t row = box_row(a, s, s.t0 * kTile + x * kVRows, bad);
                const bool any_bad = __any_sync(0xffffffffu, bad);
                if (lane == 0) {
                    S.bad[seg & 3] = any_bad;
                    if (any_bad) latch_status(a.status, DSA_ERR_BAD_INDEX);
                }
                __syncwarp();
                for (int32_t y = 0; ok && y < 32 && x0 + y < n; y += vboxes) {
                    const int32_t tile = (x0 + y) / vboxes;
                    const bool fix = past_committed(s, s.t0 + tile);
                    const uint32_t g = g0 + tile;
                    const int32_t r = __shfl_sync(0xffffffffu, row, (y + lane) & 31);     // a box each
#pragma unroll 1
                    for (int j = 0; ok && j < kVStages; ++j) {
                        const uint32_t bar =
                            fix ? map_to_cluster_rank(smem_u32(&S.vloc[j]), rank) : lead(S.vfull[j]);
                        if (lane == 0 && (g == 0 || wait(S.vempty[j], (g - 1) & 1)))
                            mbar_arrive_expect_tx_pair(bar, kVBytes);
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                        if (ok && lane < vboxes)
                            tma_load_3d_pair(smem_u32(S.v + j * kVBytes + lane * kVRows * 256), &tm_v, bar, 0, r,
                                             4 * j + 2 * (int)rank);
                    }
                }
            }
        }
    } else if (warp == 3) {
        // fix-up of V tiles that reach past the committed rows
        uint32_t fixed = 0;
        while (next_seg(s)) {
            for (int32_t t = s.t0; t < s.t1; ++t) {
                if (!past_committed(s, t)) continue;
                const int32_t pos0 = t * kTile;
                for (int j = 0; j < kVStages; ++j) {
                    wait(S.vloc[j], fixed & 1);
                    __syncwarp();
                    // two rows at a time; boxes behind the last row are zero
                    const int32_t from = max(0, s.c - pos0) + (lane >> 4), live = min(kTile, s.len - pos0);
                    const int32_t end = (live + kVRows - 1) & -kVRows;
                    auto piece = [&](int32_t x) -> uint4* {
                        const int32_t in = x & (kVRows - 1), blk = (lane >> 3) & 1;
                        return reinterpret_cast<uint4*>(S.v + j * kVBytes + (x - in) * 256 +
                                                        (blk * kVRows + in) * 128 + (lane & 7) * 16);
                    };
#pragma unroll 1
                    for (int32_t x = max(from, live + ((live ^ from) & 1)); x < end; x += 2)
                        *piece(x) = make_uint4(0, 0, 0, 0);
                    // (four reads in flight; with one, 64 drafted rows held up
                    // an item's end by 13 K cycles)
#pragma unroll 1
                    for (int32_t x0 = from; x0 < live; x0 += 8) {
                        uint4 v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (x0 + 2 * k < live) v[k] = *piece(x0 + 2 * k);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (x0 + 2 * k >= live) break;
                            uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
                            bool hit = false;
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                if ((w[q] & 0x7F80u) == 0x7F80u) w[q] &= 0xFFFF0000u, hit = true;
                                if ((w[q] & 0x7F800000u) == 0x7F800000u) w[q] &= 0xFFFFu, hit = true;
                            }
                            if (hit) *piece(x0 + 2 * k) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_pair(lead(S.vfull[j]));
                }
                ++fixed;
            }
        }
    } else if (warp < 8) {
        // softmax and epilogue: TMEM lane = tid - 128
        const int ln = tid - 128, x = ln & 63, half = ln >> 6;
        const uint32_t tl = tmem + ((uint32_t)(ln & ~31) << 16);
        uint32_t g = 0, seg = 0, xb = 0;
        auto exchange = [&](float v) -> float {
            xb ^= 1;
            S.xch[xb][ln] = v;
            named_bar_sync(1, 128);
            return S.xch[xb][ln ^ 64];
        };
        // the four warps agree on each segment, since they meet at barriers
        while (!named_bar_or(1, 128, !next_seg(s))) {
            const bool mine = (int)rank < s.rows;
            const uint64_t bits =
                mine ? visible_bits(__ldg(reinterpret_cast<const unsigned long long*>(a.mask) + s.row + rank),
                                    s.i0 + (int)rank)
                     : 0u;
            if (!mine) {
                // P of the last segment is read; zeros for this one
#pragma unroll
                for (int k = 0; k < 8; ++k) reinterpret_cast<uint4*>(S.p)[128 * k + ln] = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
            }
            float m = -INFINITY, l = 0.f;
            for (int32_t t = s.t0; t < s.t1; ++t, ++g) {
                const uint32_t buf = g & 1;
                wait(S.sfull[buf], (g >> 1) & 1);
                __syncwarp();
                tc_fence_after();
                if (!mine) {
                    // no node here: its rows of S, P and O are nobody's
                    __syncwarp();
                    if (lane == 0) mbar_arrive_pair(lead(S.sempty[buf]));
                    if (g > 0) wait(S.pvdone, (g - 1) & 1);
                    __syncwarp();
                    if (lane == 0) mbar_arrive_pair(lead(S.pfull));
                    continue;
                }
                uint32_t r[2][32];
                tmem_ld_32x32b_x32(tl + kSCol + 64 * buf, r[0]);
                tmem_ld_32x32b_x32(tl + kSCol + 64 * buf + 32, r[1]);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(lead(S.sempty[buf]));
                if (past_committed(s, t)) {
                    const int32_t d = s.c - (t * kTile + 64 * half);     // committed columns of this thread's 64
                    uint64_t vis = d >= 64 ? ~0ull : d > 0 ? (1ull << d) - 1u : 0u;
                    vis |= d >= 64 ? 0u : d >= 0 ? bits << d : d > -64 ? bits >> -d : 0u;
                    float least = INFINITY;
#pragma unroll
                    for (int k = 0; k < 64; ++k) least = fminf(least, __uint_as_float(r[k >> 5][k & 31]));
                    if (least == -INFINITY) *reinterpret_cast<volatile uint32_t*>(&S.lost[warp - 4]) = seg + 1;
#pragma unroll
                    for (int k = 0; k < 64; ++k)
                        if (!((vis >> k) & 1u)) r[k >> 5][k & 31] = 0xFF800000u;
                }
                float mx = -INFINITY;
#pragma unroll
                for (int k = 0; k < 64; ++k) mx = fmaxf(mx, __uint_as_float(r[k >> 5][k & 31]));
                mx = fmaxf(mx, exchange(mx)) * a.scale_log2;
                const bool move = mx > m + kRescale || (m == -INFINITY && mx > m);
                const float m_new = move ? mx : m;
                const float f = move ? ex2_approx(m - m_new) : 1.f;
                const float off = m_new == -INFINITY ? 0.f : m_new;
                m = m_new;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                uint32_t pk[32];
#pragma unroll
                for (int k = 0; k < 64; k += 2) {
                    const float p0 = ex2_approx(fmaf(__uint_as_float(r[k >> 5][k & 31]), a.scale_log2, -off));
                    const float p1 = ex2_approx(fmaf(__uint_as_float(r[k >> 5][(k & 31) + 1]), a.scale_log2, -off));
                    sum[(k >> 1) & 3] += p0 + p1;
                    pk[k >> 1] = pack_bf16x2(p0, p1);
                }
                l = l * f + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
                if (g > 0) wait(S.pvdone, (g - 1) & 1);
                __syncwarp();
                tc_fence_after();
                if (t > s.t0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
                    for (uint32_t c = 0; c < 256; c += 16) {
                        uint32_t o[16];
                        tmem_ld_32x32b_x16(tl + kOCol + c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        tmem_st_32x32b_x16(tl + kOCol + c, o);
                    }
                    tmem_st_wait();
                }
                uint8_t* pr = S.p + half * kChunkBytes + x * 128;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<uint4*>(pr + ((k ^ (x & 7)) << 4)) =
                        make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(lead(S.pfull));
            }
            wait(S.pvdone, (g - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            const bool bad = *reinterpret_cast<volatile int32_t*>(&S.bad[seg & 3]) != 0;
            if (mine) {
                __syncwarp();
                if (*reinterpret_cast<volatile uint32_t*>(&S.lost[warp - 4]) == seg + 1 && any_not_finite(a, s, bits))
                    l = NAN;
                l += exchange(l);
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const float ls = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
                const int64_t head = (int64_t)(s.row + (int)rank) * kH;
                const bool whole = s.whole();
                const int64_t slot = 2 * (int64_t)pair + (s.t0 == 0 ? 1 : 0);
                if (half == 0 && ok) {
                    if (!whole) a.part_lse[slot * 128 + 64 * (int)rank + x] = bad ? INFINITY : ls;
                    else if (a.lse && !bad) a.lse[head + x] = ls;
                }
                // O through a 4 KiB piece of P's buffer per warp, so that a
                // store covers whole 128-byte lines of 4 rows (16 bytes of 32
                // rows at a time: 5.7 us an item instead of 1)
                uint8_t* stage = S.p + (warp - 4) * 4096;
                uint8_t* mine_at = stage + lane * 128;
                const int x0 = x & 32;
                auto flush = [&](uint8_t* to, int64_t pitch) {
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int row = 4 * k + (lane >> 3), at = lane & 7;
                        *reinterpret_cast<uint4*>(to + row * pitch + 16 * at) =
                            *reinterpret_cast<const uint4*>(stage + row * 128 + ((at ^ (row & 7)) << 4));
                    }
                    __syncwarp();
                };
                if (ok && whole && !bad) {
#pragma unroll 2
                    for (uint32_t c = 0; c < 256; c += 64) {
                        uint32_t o[2][32];
                        tmem_ld_32x32b_x32(tl + kOCol + c, o[0]);
                        tmem_ld_32x32b_x32(tl + kOCol + c + 32, o[1]);
                        tmem_ld_wait();
#pragma unroll
                        for (int v = 0; v < 8; ++v) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                w[k] = pack_bf16x2(__uint_as_float(o[v >> 2][8 * (v & 3) + 2 * k]) * inv,
                                                   __uint_as_float(o[v >> 2][8 * (v & 3) + 2 * k + 1]) * inv);
                            *reinterpret_cast<uint4*>(mine_at + ((v ^ (lane & 7)) << 4)) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        // dims 256 j + 128 half + ..
                        const uint32_t dim = 128 * half + (c & 127) + 2 * (c & 128);
                        flush(reinterpret_cast<uint8_t*>(a.out + (head + x0) * kDV + dim), 2 * kDV);
                    }
                } else if (ok && !whole) {
                    // partial results stay in TMEM's order, four columns of a
                    // warp's 32 lanes side by side
                    float4* part = reinterpret_cast<float4*>(a.part_o) +
                                   ((slot * 2 + (int)rank) * 4 + (warp - 4)) * 64 * 32 + lane;
#pragma unroll 2
                    for (uint32_t c = 0; c < 256; c += 32) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(tl + kOCol + c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            part[(c / 4 + v) * 32] =
                                make_float4(__uint_as_float(o[4 * v]) * inv, __uint_as_float(o[4 * v + 1]) * inv,
                                            __uint_as_float(o[4 * v + 2]) * inv, __uint_as_float(o[4 * v + 3]) * inv);
                    }
                }
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(lead(S.ofree));
            ++seg;
        }
    } else {
        // the segments, and what tree_merge_kernel has to know of a cut item
        SegIter it(a, S.plan, pair, pairs);
        // the pair whose share holds unit u: the last with lo <= u
        auto holder = [&](int64_t u) -> int {
            int k = 0;
            for (int x = 0; x < pairs; x += 32)
                k += __popc(__ballot_sync(0xffffffffu, x + lane < pairs && S.plan.lo[x + lane] <= u));
            return k - 1;
        };
        int4 meta = make_int4(0, 0, 0, 0);
        bool more = true;
        for (uint32_t n = 0; ok && more; ++n) {
            more = it.next(s);
            const uint32_t slot = n & (kSegs - 1);
            if (n >= kSegs) wait(S.segempty[slot], (n / kSegs - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!more) s.t0 = s.t1 = 0;
            if (lane == 0) {
                S.seg[slot] = s;
                mbar_arrive(smem_u32(&S.segfull[slot]));
            }
            __syncwarp();
            if (more && !s.whole()) meta = make_int4(s.row, s.rows, holder(s.u0 + s.tiles - 1), holder(s.u0));
        }
        if (rank == 0 && lane == 0) a.meta[pair] = meta;
    }
    if (!ok) {
        // let copies in flight land before the CTA's shared memory goes
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000u) __nanosleep(1000);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// Joins the partial results of the items that chunks cut.  A unit is 16 TMEM
// columns of a CTA's 32 lanes, a lane per query row.  Items of few pieces: the
// 16 blocks of the pair that begins the item take a unit per warp.  Items of
// many (one long sequence over the whole GPU: 10 MB of pieces): the blocks of
// the pairs inside it, which begin nothing, help; a block takes a unit, its
// warps every 8th piece (1 x 100,000 rows: 83 -> 30 us, merge included).
constexpr int kMergeBlocks = 16, kMergeWarps = 8;

__global__ void __launch_bounds__(32 * kMergeWarps)
    tree_merge_kernel(const int4* __restrict__ meta, const float* __restrict__ part_lse,
                      const float4* __restrict__ part_o, uint16_t* __restrict__ out, float* __restrict__ lse) {
    __shared__ float acc_s[kMergeWarps][18][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    pdl_wait();
    const int4 it = meta[blockIdx.x];
    const int pair = it.w, helper = (int)blockIdx.x - pair;
    if (it.y == 0) return;
    // its pieces: the first pair's slot 2 pair + 1, then slots 2 p of the pairs
    // behind it
    const int pieces = it.z - pair + 1;
    const bool wide = pieces > kMergeWarps;
    if (!wide && helper > 0) return;
    const int helpers = wide ? it.z - pair + (meta[it.z].w == pair ? 1 : 0) : 1;
    const int e0 = wide ? warp : 0, step = wide ? kMergeWarps : 1;
    const int units = 64 * it.y, stride = wide ? kMergeBlocks * helpers : units;
    auto slot = [&](int e) -> int64_t { return e == 0 ? 2 * (int64_t)pair + 1 : 2 * ((int64_t)pair + e); };
    for (int unit = wide ? kMergeBlocks * helper + (int)blockIdx.y : kMergeWarps * (int)blockIdx.y + warp; unit < units;
         unit += stride) {
        const int rank = unit >> 6, w = (unit >> 4) & 3, c = 16 * (unit & 15);
        const int x = 32 * (w & 1) + lane;           // the lane's head
        auto piece_lse = [&](int e) -> float { return part_lse[slot(e) * 128 + 64 * rank + x]; };
        // eight pieces' sums at a time, with a running maximum
        float acc[16], sum = 0.f, top = -INFINITY;
        bool bad = false, nan = false;
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[k] = 0.f;
#pragma unroll 1
        for (int e1 = e0; e1 < pieces; e1 += 8 * step) {
            float ls[8], mx = top;
#pragma unroll
            for (int q = 0; q < 8; ++q) ls[q] = e1 + q * step < pieces ? piece_lse(e1 + q * step) : -INFINITY;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                bad = bad || ls[q] == INFINITY;
                nan = nan || ls[q] != ls[q];
                mx = fmaxf(mx, ls[q]);
            }
            const float base = mx == -INFINITY ? 0.f : mx, down = ex2_approx((top - base) * kLog2e);
            top = mx;
            sum *= down;
#pragma unroll
            for (int k = 0; k < 16; ++k) acc[k] *= down;
#pragma unroll 2
            for (int q = 0; q < 8; ++q) {
                if (e1 + q * step >= pieces) break;
                const float f = ex2_approx((ls[q] - base) * kLog2e);
                const float4* o = part_o + (((slot(e1 + q * step) * 2 + rank) * 4 + w) * 64 + c / 4) * 32 + lane;
                sum += f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 v = o[32 * k];
                    acc[4 * k] += f * v.x;
                    acc[4 * k + 1] += f * v.y;
                    acc[4 * k + 2] += f * v.z;
                    acc[4 * k + 3] += f * v.w;
                }
            }
        }
        if (bad) top = INFINITY;
        else if (nan) top = NAN;
        if (wide) {
            // the warps' sums, in order
#pragma unroll
            for (int k = 0; k < 16; ++k) acc_s[warp][k][lane] = acc[k];
            acc_s[warp][16][lane] = sum;
            acc_s[warp][17][lane] = top;
            __syncthreads();
            if (warp == 0) {
                float mx = top;
#pragma unroll
                for (int v = 1; v < kMergeWarps; ++v) {
                    const float m = acc_s[v][17][lane];
                    if (mx != INFINITY) mx = m == INFINITY || m != m ? m : mx != mx ? mx : fmaxf(mx, m);
                }
                const float base = mx == -INFINITY ? 0.f : mx;
                const float own = ex2_approx((top - base) * kLog2e);
                sum *= own;
#pragma unroll
                for (int k = 0; k < 16; ++k) acc[k] *= own;
#pragma unroll
                for (int v = 1; v < kMergeWarps; ++v) {
                    const float f = ex2_approx((acc_s[v][17][lane] - base) * kLog2e);
#pragma unroll
                    for (int k = 0; k < 16; ++k) acc[k] += f * acc_s[v][k][lane];
                    sum += f * acc_s[v][16][lane];
                }
                top = mx;
            }
            __syncthreads();
            if (warp != 0) continue;
        }
        if (top == INFINITY) continue;           // a bad page in one of the pieces
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t head = (int64_t)(it.x + rank) * kH + x;
        uint4* to = reinterpret_cast<uint4*>(out + head * kDV + 128 * (w >> 1) + (c & 127) + 2 * (c & 128));
#pragma unroll
        for (int k = 0; k < 2; ++k)
            to[k] = make_uint4(pack_bf16x2(acc[8 * k] * inv, acc[8 * k + 1] * inv),
                               pack_bf16x2(acc[8 * k + 2] * inv, acc[8 * k + 3] * inv),
                               pack_bf16x2(acc[8 * k + 4] * inv, acc[8 * k + 5] * inv),
                               pack_bf16x2(acc[8 * k + 6] * inv, acc[8 * k + 7] * inv));
        if (lse && (w >> 1) == 0 && c == 0) lse[head] = sum == 0.f ? -INFINITY : top + log2f(sum) * kLn2;
    }
}

// CTA pairs that can be resident at once on the current device.
int max_pairs() {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> cache[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return kDefaultSMs / 2;
    }
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * num_sms());
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Smem);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(tree_mla_kernel<64, 64>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem)) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, tree_mla_kernel<64, 64>, &cfg) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        return num_sms() / 2;
    }
    n = std::min(n, std::min(num_sms() / 2, kMaxPairs));
    cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Pairs that a call launches: no more than its bounds give work to.
int pairs_for(const BatchDev& bd) {
    const int64_t items = (int64_t)bd.B * ((std::min(bd.max_q, DSA_MAX_TREE) + 1) / 2);
    const int64_t units = items * ((bd.max_ctx + kTile - 1) / kTile + kItemCost);
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min(num_sms() / 2, kMaxPairs), units));
}

}  // namespace

size_t tree_mla_scratch_bytes(const BatchDev& bd) {
    const size_t pairs = (size_t)pairs_for(bd);
    return pairs * (sizeof(int4) + 2 * 128 * sizeof(float) * (1 + (size_t)kDV)) + 256;
}

cudaError_t launch_tree_mla(const BatchDev& bd, const PagesDev& pg, const uint16_t* q, const uint16_t* kv,
                            const uint64_t* mask, float sm_scale, uint16_t* out, float* lse, void* scratch,
                            int32_t* status, cudaStream_t stream) {
    const size_t slots = 2 * (size_t)pairs_for(bd);
    const int pairs = std::min(pairs_for(bd), max_pairs());
    Args a{};
    a.bd = bd;
    a.pg = pg;
    a.mask = mask;
    a.kv = kv;
    a.ahead = bd.max_q <= 2;
    a.scale_log2 = sm_scale * kLog2e;
    a.out = out;
    a.lse = lse;
    a.status = status;
    a.part_o = static_cast<float*>(scratch);
    a.part_lse = a.part_o + slots * 128 * kDV;
    a.meta = reinterpret_cast<int4*>(a.part_lse + slots * 128);
    a.may_round = bd.B <= kPlanSeqs && bd.max_q > 2 && pairs <= kMaxPairs &&
                  (int64_t)bd.B * bd.max_ctx * 2 * kDQK > kSharedBytes;
    a.rows_total = pg.table ? pg.pool_pages << pg.shift : (int32_t)(bd.B * bd.stride);
    const int page = pg.table ? 1 << pg.shift : kTile;
    const uint32_t krows = page >= 64 ? 64 : page == 32 ? 32 : 8, kchunks = krows == 32 ? 1 : kGroup;
    const uint32_t vrows = (uint32_t)std::min(page, 64);
    CUtensorMap tm_q, tm_k, tm_v;
    if (!make_tmap_bf16_2d(&tm_q, q, kDQK, (uint64_t)bd.total_q * kH, 64, 64) ||
        !make_tmap_bf16_chunks(&tm_k, kv, kQChunks, (uint64_t)a.rows_total, krows, kchunks) ||
        !make_tmap_bf16_chunks(&tm_v, kv, kQChunks, (uint64_t)a.rows_total, vrows, 2))
        return cudaErrorInvalidValue;
    auto kernel = krows == 64   ? tree_mla_kernel<64, 64>
                  : krows == 32 ? tree_mla_kernel<32, 32>
                                : tree_mla_kernel<8, 16>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
    if (e != cudaSuccess) return e;
    // Both are programmatic dependents of the launch before them: they set up
    // while it drains and wait for it before they read anything.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)pairs);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, kernel, a, tm_q, tm_k, tm_v)) != cudaSuccess) return e;
    count_launches(1);
    cfg.gridDim = dim3((unsigned)pairs, kMergeBlocks);
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, tree_merge_kernel, (const int4*)a.meta, (const float*)a.part_lse,
                           (const float4*)a.part_o, out, lse);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace dsa
