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
// Behind shared prefixes (dsa_prefix_mla_fwd) a group's new rows are paired
// across its sequences, so an item walks the shared tiles once and then the own
// ones of its one or two sequences.  (Shared and own parts as items of their
// own, all joined in fp32: 242 instead of 180 us for 61 sequences of up to 15
// rows behind 3,774, and 263 KB of workspace a row and sequence.)  Cut, joined and merged as above.
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
#include <type_traits>

#include "internal.h"
#include "prompt.h"
#include "ptx.cuh"
#include "tree.h"

namespace dsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kTile = 128;                   // positions per tile
constexpr int kItemCost = 3;                 // an item's start and end, in tiles
constexpr int kApartUnits = 6;               // units a pair that are little work
constexpr int kFewRows = 64;                 // rows of a call up to which a merge goes by rows
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
    __device__ int32_t first_pos(int32_t t) const { return t * kTile; }
    __device__ bool begins() const { return true; }              // a segment is all that a pair has of an item
    __device__ bool ends() const { return true; }
    __device__ bool sees(uint32_t) const { return true; }
    __device__ bool from_start() const { return t0 == 0; }
};

// Behind shared prefixes an item is two new rows of a group, and its tiles lie in
// up to three sequences' caches: the shared ones, those of the first row's
// sequence, and those of the second row's if that is another.  A segment is what a
// pair has of one of them.
struct SharedSeg : Seg {
    int32_t shift;               // tiles of the item before the first of this cache, less those before it there
    int32_t from, to;            // the item's tiles that the pair has, of all three
    uint32_t live;               // bit r: CTA r's row sees this cache
    bool ahead;                  // no other item reads its rows
    __device__ bool whole() const { return from == 0 && to == tiles; }
    __device__ int32_t first_pos(int32_t t) const { return (t - shift) * kTile; }
    __device__ bool begins() const { return t0 == from; }
    __device__ bool ends() const { return t1 == to; }
    __device__ bool sees(uint32_t rank) const { return (live >> rank) & 1u; }
    __device__ bool from_start() const { return from == 0; }
};

// Behind shared prefixes the work is a list of runs, two a sequence: the items
// whose rows are both its own, and the one of its last row and the next
// sequence's first (or none), if a row is left.
struct alignas(16) Run {
    int32_t row, items;          // first new row, items
    int32_t lead, base;          // whose cache holds the shared rows, tiles of them
    int32_t b, len, n, i0;       // sequence, length of its cache, its new rows, which of them `row` is
    int32_t b2, len2, n2;        // of the second row's sequence (n2 = 0: none)
    int32_t rows;                // rows of an item
    int32_t lone, pad;           // whether the shared rows are this item's alone
    int64_t u;                   // units before it
    __device__ int32_t own() const { return (len + kTile - 1) / kTile - base; }
    __device__ int32_t tiles() const { return base + own() + (n2 > 0 ? (len2 + kTile - 1) / kTile - base : 0); }
};
static_assert(sizeof(Run) == 64, "four 16-byte loads");

struct RunPlan {
    int64_t all, chunk;          // units, and those of a pair
};

template <class S>
struct SmemOf {
    alignas(1024) uint8_t q[kQChunks * kChunkBytes];
    alignas(1024) uint8_t k[kKStages * kKBytes];
    alignas(1024) uint8_t v[kVStages * kVBytes];
    alignas(1024) uint8_t p[2 * kChunkBytes];
    alignas(8) uint64_t kfull[kKStages], kempty[kKStages], vfull[kVStages], vempty[kVStages], vloc[kVStages];
    uint64_t qfull, qempty, sfull[2], sempty[2], pfull, pvdone, ofree, segfull[kSegs], segempty[kSegs];
    Plan plan;
    S seg[kSegs];
    int64_t scan[kThreads / 32];
    int32_t longest[kThreads / 32];
    float xch[2][128];
    int32_t bad[4];
    uint32_t lost[4];            // softmax warps: 1 + the last segment with a score of -inf past the committed rows
    uint32_t tmem;
};
using Smem = SmemOf<Seg>;
static_assert(sizeof(SmemOf<SharedSeg>) <= 232448, "one CTA's shared memory");

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
    // behind shared prefixes only
    const RunPlan* rplan;
    const Run* runs;     // null: each pair's walker plans by itself (LocalRuns)
    GroupsDev groups;
    int32_t least_shared;
    int32_t runs_total;
    int2* cut_rows;      // [total_q] or null: of a row of a cut item, 2 * (first pair + 1) + which of its rows, last pair
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

__device__ int least_chunk(int tiles);

// prefix_plan_kernel's runs of at most 32 sequences and groups, by a warp: lane b
// holds sequence b's.
struct LocalRuns {
    int32_t q0 = 0, nq = 0, ctx = 0, base = 0, lead = 0, skip = 0, inner = 0, tail = 0, b2 = 0, len2 = 0, n2 = 0, lone = 0;
    int64_t u = 0, ut = 0;       // units before the first and the second run
    bool good = false;

    __device__ RunPlan make(const Args& a, int pairs) {
        constexpr uint32_t kAll = 0xffffffffu;
        const int lane = (int)lane_id(), G = a.groups.n;
        const bool seq = lane < a.bd.B, grp = lane < G;
        SeqInfo s{0, 0, 0};
        const int32_t off0 = grp ? __ldg(a.groups.off + lane) : 0, off1 = grp ? __ldg(a.groups.off + lane + 1) : 0;
        const int32_t shared = grp ? __ldg(a.groups.shared + lane) : 0;
        good = seq && load_seq(a.bd, lane, a.status, s);
        q0 = s.q0, nq = s.nq, ctx = s.ctx;
        const bool broken = __any_sync(kAll, seq && !good);
        const bool wrong = __any_sync(kAll, grp && (off0 < 0 || off0 > off1 || off1 > a.bd.B || (lane == 0 && off0 != 0) ||
                                                    (lane == G - 1 && off1 != a.bd.B) || shared < 0));
        int g = 0;
        for (int k = 1; k < G; ++k) g += __shfl_sync(kAll, off0, k) <= lane ? 1 : 0;
        const int32_t rows = __shfl_sync(kAll, shared, g);
        const bool bad = seq && !wrong && !(good && (nq == 0 || rows <= ctx - nq));
        if (bad || (wrong && lane == 0)) latch_status(a.status, DSA_ERR_BAD_BATCH);
        const uint32_t peers = __match_any_sync(kAll, seq ? g : 32 + lane), wrongs = __ballot_sync(kAll, bad);
        const uint32_t live = __ballot_sync(kAll, good && nq > 0) & peers, after = live & ~((2u << lane) - 1u);
        base = wrong || (wrongs & peers) ? 0 : rows / kTile;
        lead = live ? __ffs(live) - 1 : 0;
        const int32_t first = __shfl_sync(kAll, q0, __ffs(peers) - 1), end = __shfl_sync(kAll, q0 + nq, 31 - __clz(peers));
        const bool mixed = !broken && !wrong && base >= a.least_shared;
        const int32_t row1 = mixed ? end : q0 + nq;
        skip = mixed ? (q0 - first) & 1 : 0;
        lone = mixed && end - first <= 2;
        inner = good && nq > 0 ? (nq - skip) >> 1 : 0;
        tail = good && nq > 0 ? (nq - skip) & 1 : 0;
        b2 = after ? __ffs(after) - 1 : 0;
        len2 = __shfl_sync(kAll, ctx, b2);
        n2 = __shfl_sync(kAll, nq, b2);
        if (!tail || q0 + nq >= row1) n2 = 0;
        const Run x = run(false), y = run(true);
        const int64_t cost = (int64_t)inner * (x.tiles() + kItemCost), both = cost + (int64_t)tail * (y.tiles() + kItemCost);
        const int32_t longest =
            __reduce_max_sync(kAll, max(inner ? x.tiles() : 0, tail ? y.tiles() : 0));
        int64_t sum = both;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(kAll, sum, o);
            if (lane >= o) sum += v;
        }
        u = sum - both;
        ut = u + cost;
        const int64_t all = __shfl_sync(kAll, sum, 31), even = (all + pairs - 1) / pairs;
        return RunPlan{all, max(even, (int64_t)least_chunk(longest))};
    }
    // this lane's first or second run
    __device__ Run run(bool second) const {
        Run r{};
        r.row = second ? q0 + nq - 1 : q0 + skip;
        r.items = second ? tail : inner;
        r.lead = lead;
        r.base = base;
        r.b = (int32_t)lane_id();
        r.len = ctx;
        r.n = nq;
        r.i0 = second ? nq - 1 : skip;
        r.b2 = b2;
        r.len2 = len2;
        r.n2 = second ? n2 : 0;
        r.rows = second && n2 == 0 ? 1 : 2;
        r.lone = lone;
        r.u = second ? ut : u;
        return r;
    }
    // run i, to all lanes
    __device__ Run fetch(int32_t i) const {
        Run r = run(i & 1);
        int32_t* const w = reinterpret_cast<int32_t*>(&r);
#pragma unroll
        for (int k = 0; k < (int)(sizeof(Run) / 4); ++k) w[k] = __shfl_sync(0xffffffffu, w[k], i >> 1);
        return r;
    }
};

// The same over runs, by one warp: a pair has an equal share of their units.
struct RunIter {
    const Args& a;
    const int32_t pair;
    int64_t lo, hi, chunk, u0 = 0;
    int32_t r = 0, p = -1, at = 0, to = 0;       // run, its next item; the item's tiles that are left
    Run q{};
    LocalRuns local;
    __device__ RunIter(const Args& args, int32_t pair_, int32_t pairs) : a(args), pair(pair_) {
        const int lane = (int)lane_id();
        if (!a.runs) {
            share(local.make(a, pairs));
            if (lo >= hi) return;
            r = 2 * (__popc(__ballot_sync(0xffffffffu, lane < a.bd.B && local.u <= lo)) - 1);
            if (__shfl_sync(0xffffffffu, local.ut, r >> 1) <= lo) ++r;
            q = local.fetch(r);
            return;
        }
        // The last run that begins at or before lo: 32 probes at a time, the
        // first on their way with the plan itself.
        int32_t span = a.runs_total;             // it is one of runs r .. r + span - 1
        for (bool first = true; first || span > 1; first = false) {
            const int32_t step = (span + 31) / 32, i = r + lane * step;
            const int64_t u = lane * step < span ? a.runs[i].u : INT64_MAX;
            if (first) share(*a.rplan);
            const int last = __popc(__ballot_sync(0xffffffffu, u <= lo)) - 1;
            r += last * step;
            span = min(step, span - last * step);
        }
        if (lo < hi) q = a.runs[r];
    }
    __device__ void share(const RunPlan& pl) {
        chunk = pl.chunk;
        lo = min(pl.all, pair * chunk);
        hi = min(pl.all, lo + chunk);
    }
    __device__ int32_t holder(int64_t u) const { return (int32_t)(u / chunk); }

    // The next item of the pair's share, its tiles at .. to - 1.
    __device__ bool item(SharedSeg& s) {
        if (lo >= hi) return false;
        while (r < a.runs_total) {
            const int32_t tiles = q.tiles(), per = tiles + kItemCost;
            if (p < 0) p = (int32_t)min((int64_t)q.items, (lo - q.u) / per);
            while (p < q.items) {
                u0 = q.u + (int64_t)p * per + kItemCost;
                if (u0 - kItemCost >= hi) return false;
                at = (int32_t)max((int64_t)0, min((int64_t)tiles, lo - u0));
                to = (int32_t)max((int64_t)0, min((int64_t)tiles, hi - u0));
                const int32_t i = p++;
                if (to <= at) continue;
                s.row = q.row + 2 * i;
                s.rows = q.rows;
                s.tiles = tiles;
                s.u0 = u0;
                s.from = at;
                s.to = to;
                return true;
            }
            p = 0;
            if (++r < a.runs_total) q = a.runs ? a.runs[r] : local.fetch(r);
        }
        return false;
    }

    __device__ bool next(SharedSeg& s) {
        if (at >= to && !item(s)) return false;
        // (the item's run: an item is walked to its end before the next)
        const int32_t mid = q.base + q.own(), i = s.row - q.row;
        s.t0 = at;
        if (at < q.base) {
            s.t1 = min(to, q.base);
            s.b = q.lead;
            s.len = s.c = q.base * kTile;
            s.i0 = s.shift = 0;
            s.live = 3u;
            s.ahead = q.lone != 0;
        } else if (at < mid) {
            s.t1 = min(to, mid);
            s.b = q.b;
            s.len = q.len;
            s.c = q.len - q.n;
            s.i0 = q.i0 + i;
            s.shift = 0;
            s.live = q.n2 > 0 ? 1u : 3u;
            s.ahead = q.n <= 2;
        } else {
            s.t1 = to;
            s.b = q.b2;
            s.len = q.len2;
            s.c = q.len2 - q.n2;
            s.i0 = -1;                           // CTA 1's row is its first
            s.shift = mid - q.base;
            s.live = 2u;
            s.ahead = q.n2 <= 2;
        }
        at = s.t1;
        return true;
    }
};

// The least work worth a pair of its own, in units: a tile takes 1.2 us (2 us
// among the first) and a piece 0.17 us more in the merge, so an item of N
// tiles alone on the GPU is done soonest in pieces of about sqrt(N / 4)
// (1 x 8,000 rows: 18.9 us in pieces of 4 tiles, 23.6 of 1; 1 x 1,500: 14.7 in
// pieces of 1, 16.9 of 2 and of 4).
__device__ int least_chunk(int tiles) {
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
template <class S>
__device__ __forceinline__ int32_t box_row(const Args& a, const S& s, int32_t pos, bool& bad) {
    if (pos >= s.len) return a.rows_total;
    const int32_t r = cache_row(a.bd, a.pg, s.b, pos);
    if (r >= 0) return r;
    bad = true;
    return a.rows_total;
}

template <class S>
__device__ __forceinline__ bool past_committed(const S& s, int32_t t) { return s.first_pos(t + 1) > s.c; }

// Whether one of the new rows `rows` in the segment's tiles holds a NaN or an
// infinity; all lanes.  Called when a row past the committed ones scored -inf,
// which is seldom; a call, since the code of it inside the softmax role costs
// long calls 1-2 %, out of the way 0.5 % (16 trees of 64 over 8,192 rows).
template <class S>
__device__ __noinline__ bool any_not_finite(const Args& a, const S& s, uint64_t rows) {
#pragma unroll 1
    for (; rows; rows &= rows - 1u) {
        const int32_t pos = s.c + __ffsll((long long)rows) - 1;
        if (pos < s.first_pos(s.t0) || pos >= s.first_pos(s.t1)) continue;
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

// kRows: positions of a box of K (a stage's three chunks) and of V (two): 64 for
// pages of 64 rows and more and contiguous caches; pages of 32 and 16 take
// boxes of a page, K by 8-row groups x three chunks, which stay evenly spaced
// in a stage as a descriptor needs them (pages of 16: 12 K and 16 V boxes a
// tile; with K boxes of one group, 24 and 16, 155 instead of 141 us for 40
// rows in 5 groups of 6 behind 12,001).
//
// kShared: behind shared prefixes.  The work is runs: those that prefix_plan_kernel
// wrote, or, for at most 32 sequences, the walker's own (LocalRuns).  Over the own tiles of one of an item's two sequences the other CTA's
// lanes of O are left out of the product (0 * NaN is NaN).
template <int kRows, bool kShared>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    tree_mla_kernel(const Args a, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    using Segment = std::conditional_t<kShared, SharedSeg, Seg>;
    SmemOf<Segment>& S = *reinterpret_cast<SmemOf<Segment>*>(smem_raw);
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
    if constexpr (!kShared) {
        make_plan(a, S, pair, pairs);
        if (a.may_round) fence_proxy_async_smem();   // plan_rounds used the V ring
    }
    tc_fence_before();
    __syncthreads();
    cluster_wait();                              // .. and this CTA the peer's
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    Segment s;
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
    auto next_seg = [&](Segment& to) -> bool {
        const uint32_t slot = segs_read & (kSegs - 1);
        wait(S.segfull[slot], (segs_read / kSegs) & 1);
        ok = __all_sync(0xffffffffu, ok);
        to = S.seg[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&S.segempty[slot]));
        ++segs_read;
        return ok && to.t1 > to.t0;
    };
    constexpr int kboxes = 64 / kRows, vboxes = kTile / kRows;       // per stage's positions
    constexpr bool kGroups = kRows < 64;         // K boxes of 8-row groups x three chunks

    // MMAs are issued by one elected lane, which also waits: the tensor pipe
    // takes a K chunk's four MMAs in 150 cycles, less than a warp that waits
    // together, votes and branches to its issuing lane needs (4.5 us a tile
    // that way, of 1.3 us in the pipe).  Loads have that time: lane 0 waits,
    // then each lane issues a box.
    if (warp == 0) {
        // Q and K loads
        uint32_t g0 = 0, item = 0;               // tiles and items before this one
        for (; next_seg(s); g0 += s.t1 - s.t0, item += s.ends()) {
            // first rows of the segment's boxes, 32 at a time
            const int32_t n = (s.t1 - s.t0) * kboxes;
            for (int32_t x0 = 0; ok && x0 < n; x0 += 32) {
                bool bad = false;
                const int32_t x = x0 + lane;
                const int32_t row =
                    box_row(a, s, s.first_pos(s.t0 + x / kboxes) + 64 * (int)rank + (x % kboxes) * kRows, bad);
                for (int32_t y = 0; ok && y < 32 && x0 + y < n; y += kboxes) {
                    if (x0 + y == 0 && s.begins()) {
                        // No row for this CTA: zeros, from behind the queries.
                        // Whatever lay there would do as well, but its products
                        // cost power, which holds the clock (64 x 1 row over
                        // 32,768 in a long loop: 438 us, 407 with zeros).
                        const int32_t q_row = (int)rank < s.rows ? (s.row + (int)rank) * kH : a.bd.total_q * kH;
                        if (lane == 0 && (item == 0 || wait(S.qempty, (item - 1) & 1)))
                            mbar_arrive_expect_tx_pair(lead(S.qfull), (uint32_t)sizeof(S.q));
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                        if (ok && lane < kQChunks)
                            tma_load_2d_pair(smem_u32(S.q + lane * kChunkBytes), &tm_q, lead(S.qfull), 64 * lane, q_row);
                    }
                    const uint32_t g = g0 + (x0 + y) / kboxes;
                    const int32_t r = __shfl_sync(0xffffffffu, row, (y + lane) & 31);    // a box each
#pragma unroll 1
                    for (int gr = 0; ok && gr < kKStages; ++gr) {
                        const uint32_t bar = lead(S.kfull[gr]);
                        if (lane == 0 && (g == 0 || wait(S.kempty[gr], (g - 1) & 1)))
                            mbar_arrive_expect_tx_pair(bar, kKBytes);
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                        if (ok && lane < kboxes) {
                            const uint32_t dst = smem_u32(S.k + gr * kKBytes + lane * kRows * 128 * kGroup);
                            if constexpr (kGroups) tma_load_4d_pair(dst, &tm_k, bar, 0, 0, kGroup * gr, r >> 3);
                            else tma_load_3d_pair(dst, &tm_k, bar, 0, r, kGroup * gr);
                        }
                    }
                    // Rows that no other pair reads come from HBM: the next
                    // tile's are brought to L2 while this one's are loaded
                    // (64 x 1 row over 32,768: 416 -> 399 us; with rows that
                    // several pairs share the same costs 4-7 %).
                    bool ahead = a.ahead;
                    if constexpr (kShared) ahead = s.ahead;
                    if (ahead) {
                        const int32_t next = y + kboxes + lane;
                        const int32_t r2 = __shfl_sync(0xffffffffu, row, next & 31);
                        if (lane < kboxes && next < 32 && x0 + next < n && r2 < a.rows_total)
                            prefetch_l2_bulk(a.kv + (int64_t)r2 * kDQK, min(kRows, a.rows_total - r2) * 2 * kDQK);
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // MMA: S of tile g + 1, then PV of tile g
            constexpr uint32_t kIdS = idesc_bf16_f32(128, kTile), kIdO = idesc_bf16_f32(128, 256, false, true);
            // K stages: three chunks of 64 rows, or (smaller pages) eight
            // groups of 8 rows x three chunks; V stages: boxes of two 64-dim
            // blocks of vrows rows
            constexpr uint32_t ksbo = kGroups ? 1024 * kGroup : 1024;
            constexpr uint32_t kcstep = (kGroups ? 1024 : kChunkBytes) >> 4;
            // S of tile g; first / last of what the pair has of its item (number `item`)
            auto issue_s = [&](uint32_t g, bool first, bool last, uint32_t item) {
                if (first && !wait(S.qfull, item & 1)) return;
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
            // fresh: the first that its rows see; off0, off1: all ones where a CTA's row sees nothing of it
            auto issue_pv = [&](uint32_t g, bool first, bool fresh, uint32_t item, uint32_t off0, uint32_t off1) {
                if (first && item > 0 && !wait(S.ofree, (item - 1) & 1)) return;
                if (!wait(S.pfull, g & 1)) return;
                tc_fence_after();
                const uint64_t dp = sdesc_sw128(smem_u32(S.p), 0, 1024), dv = sdesc_sw128(smem_u32(S.v), kRows * 128, 1024);
#pragma unroll 1
                for (int j = 0; j < kVStages; ++j) {
                    if (!wait(S.vfull[j], g & 1)) return;
                    tc_fence_after();
                    const uint64_t db = dv + j * (kVBytes >> 4);
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k) {
                        const uint64_t da = dp + (k >> 2) * (kChunkBytes >> 4) + 2 * (k & 3);
                        const uint64_t dk = db + 128 * k + 128 * ((16 * k) & -kRows) / 16;
                        if constexpr (kShared)
                            mma_bf16_ss_pair_lanes(tmem + kOCol + 128 * j, da, dk, kIdO, !fresh || k != 0, off0, off1);
                        else
                            mma_bf16_ss_pair(tmem + kOCol + 128 * j, da, dk, kIdO, !fresh || k != 0);
                    }
                    mma_commit_pair(smem_u32(&S.vempty[j]));
                }
                mma_commit_pair(smem_u32(&S.pvdone));
            };
            Segment n;
            bool more = next_seg(n);
            uint32_t g = 0, item = 0, begun = 0; // begun: bit r, CTA r's row has seen a tile
            if (more && elect_one()) issue_s(0, true, n.t1 - n.t0 == 1 && n.ends(), 0);
            __syncwarp();
            ok = __all_sync(0xffffffffu, ok);
            while (ok && more) {
                s = n;
                more = next_seg(n);
                const int32_t tiles = s.t1 - s.t0;
                const uint32_t off0 = s.sees(0) ? 0u : ~0u, off1 = s.sees(1) ? 0u : ~0u;
                const uint32_t live = (off0 ? 0u : 1u) | (off1 ? 0u : 2u);
                if (s.begins()) begun = 0;
                const bool fresh = !(begun & live);
                begun |= live;
                if (elect_one()) {
                    for (int32_t t = 0; ok && t < tiles; ++t) {
                        if (t + 1 < tiles) issue_s(g + t + 1, false, t + 2 == tiles && s.ends(), item);
                        else if (more) issue_s(g + t + 1, n.begins(), n.t1 - n.t0 == 1 && n.ends(), item + s.ends());
                        if (ok) issue_pv(g + t, t == 0 && s.begins(), t == 0 && fresh, item, off0, off1);
                    }
                }
                __syncwarp();
                ok = __all_sync(0xffffffffu, ok);
                g += tiles;
                item += s.ends();
            }
        }
    } else if (warp == 2) {
        // V loads
        uint32_t g0 = 0, item = 0;
        bool any_bad = false;
        for (; next_seg(s); g0 += s.t1 - s.t0, item += s.ends()) {
            const int32_t n = (s.t1 - s.t0) * vboxes;
            if (s.begins()) any_bad = false;
            for (int32_t x0 = 0; ok && x0 < n; x0 += 32) {
                const int32_t x = x0 + lane;
                bool bad = false;
                const int32_t row = box_row(a, s, s.first_pos(s.t0) + x * kRows, bad);
                bad = __any_sync(0xffffffffu, bad);
                any_bad = any_bad || (bad && s.sees(rank));
                if (lane == 0) {
                    S.bad[item & 3] = any_bad;
                    if (bad) latch_status(a.status, DSA_ERR_BAD_INDEX);
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
                            tma_load_3d_pair(smem_u32(S.v + j * kVBytes + lane * kRows * 256), &tm_v, bar, 0, r,
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
                const int32_t pos0 = s.first_pos(t);
                for (int j = 0; j < kVStages; ++j) {
                    wait(S.vloc[j], fixed & 1);
                    __syncwarp();
                    // two rows at a time; boxes behind the last row are zero
                    const int32_t from = max(0, s.c - pos0) + (lane >> 4), live = min(kTile, s.len - pos0);
                    const int32_t end = (live + kRows - 1) & -kRows;
                    auto piece = [&](int32_t x) -> uint4* {
                        const int32_t in = x & (kRows - 1), blk = (lane >> 3) & 1;
                        return reinterpret_cast<uint4*>(S.v + j * kVBytes + (x - in) * 256 +
                                                        (blk * kRows + in) * 128 + (lane & 7) * 16);
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
        uint32_t g = 0, seg = 0, item = 0, xb = 0;
        float m = -INFINITY, l = 0.f;
        bool begun = false, lost = false;        // the row has seen a tile; an infinity that its scores do not show
        auto exchange = [&](float v) -> float {
            xb ^= 1;
            S.xch[xb][ln] = v;
            named_bar_sync(1, 128);
            return S.xch[xb][ln ^ 64];
        };
        // the four warps agree on each segment, since they meet at barriers
        while (!named_bar_or(1, 128, !next_seg(s))) {
            const bool mine = (int)rank < s.rows && s.sees(rank);
            const uint64_t bits =
                mine ? visible_bits(kShared && !a.mask
                                        ? ~0ull
                                        : __ldg(reinterpret_cast<const unsigned long long*>(a.mask) + s.row + rank),
                                    s.i0 + (int)rank)
                     : 0u;
            if ((int)rank >= s.rows && s.begins()) {
                // P of the last segment is read; zeros for this one
#pragma unroll
                for (int k = 0; k < 8; ++k) reinterpret_cast<uint4*>(S.p)[128 * k + ln] = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
            }
            if (s.begins()) {
                m = -INFINITY, l = 0.f;
                begun = lost = false;
            }
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
                    const int32_t d = s.c - (s.first_pos(t) + 64 * half);     // committed columns of this thread's 64
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
                if (begun && __any_sync(0xffffffffu, f != 1.f)) {
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
                begun = true;
            }
            if constexpr (kShared) {
                if (!s.ends()) {
                    __syncwarp();
                    if (mine && *reinterpret_cast<volatile uint32_t*>(&S.lost[warp - 4]) == seg + 1 &&
                        any_not_finite(a, s, bits))
                        lost = true;
                    ++seg;
                    continue;
                }
            }
            wait(S.pvdone, (g - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            const bool bad = *reinterpret_cast<volatile int32_t*>(&S.bad[item & 3]) != 0;
            if ((int)rank < s.rows) {
                __syncwarp();
                if (mine && *reinterpret_cast<volatile uint32_t*>(&S.lost[warp - 4]) == seg + 1 &&
                    any_not_finite(a, s, bits))
                    lost = true;
                if (lost) l = NAN;
                l += exchange(l);
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const float ls = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
                const int64_t head = (int64_t)(s.row + (int)rank) * kH;
                const bool whole = s.whole();
                const int64_t slot = 2 * (int64_t)pair + (s.from_start() ? 1 : 0);
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
                    // warp's 32 lanes side by side (zeros for a row that sees
                    // none of the pair's tiles: nothing wrote its lanes)
                    float4* part = reinterpret_cast<float4*>(a.part_o) +
                                   ((slot * 2 + (int)rank) * 4 + (warp - 4)) * 64 * 32 + lane;
#pragma unroll 2
                    for (uint32_t c = 0; c < 256; c += 32) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(tl + kOCol + c, o);
                        tmem_ld_wait();
                        if constexpr (kShared) {
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = begun ? o[k] : 0u;
                        }
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
            ++item;
        }
    } else {
        // the segments, and what tree_merge_kernel has to know of a cut item
        auto publish = [&](uint32_t n, bool more) {
            const uint32_t slot = n & (kSegs - 1);
            if (n >= kSegs) wait(S.segempty[slot], (n / kSegs - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!more) s.t0 = s.t1 = 0;
            if (lane == 0) {
                S.seg[slot] = s;
                mbar_arrive(smem_u32(&S.segfull[slot]));
            }
            __syncwarp();
        };
        bool more = true;
        int4 meta = make_int4(0, 0, 0, 0);
        if constexpr (kShared) {
            RunIter it(a, pair, pairs);
            if (!a.runs && a.cut_rows && pair == 0 && rank == 0) {
                // rows of no sequence: nothing to join
                for (int32_t row = lane; row < (a.bd.total_q + 31 & ~31); row += 32) {
                    bool any = false;
                    for (int b = 0; b < a.bd.B; ++b) {
                        const int32_t q0 = __shfl_sync(0xffffffffu, it.local.q0, b), nq = __shfl_sync(0xffffffffu, it.local.nq, b);
                        const int good = __shfl_sync(0xffffffffu, it.local.good ? 1 : 0, b);
                        any |= good && q0 <= row && row < q0 + nq;
                    }
                    if (!any && row < a.bd.total_q) a.cut_rows[row] = make_int2(0, 0);
                }
            }
            for (uint32_t n = 0; ok && more; ++n) {
                more = it.next(s);
                publish(n, more);
                if (more && s.ends()) {
                    const bool cut = !s.whole();
                    if (cut) meta = make_int4(s.row, s.rows, it.holder(s.u0 + s.tiles - 1), it.holder(s.u0));
                    if (a.cut_rows && s.from_start() && rank == 0 && lane < s.rows)
                        a.cut_rows[s.row + lane] = cut ? make_int2(2 * (pair + 1) + lane, meta.z) : make_int2(0, 0);
                }
            }
        } else {
            SegIter it(a, S.plan, pair, pairs);
            // the pair whose share holds unit u: the last with lo <= u
            auto holder = [&](int64_t u) -> int {
                int k = 0;
                for (int x = 0; x < pairs; x += 32)
                    k += __popc(__ballot_sync(0xffffffffu, x + lane < pairs && S.plan.lo[x + lane] <= u));
                return k - 1;
            };
            for (uint32_t n = 0; ok && more; ++n) {
                more = it.next(s);
                publish(n, more);
                if (more && !s.whole()) meta = make_int4(s.row, s.rows, holder(s.u0 + s.tiles - 1), holder(s.u0));
            }
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

constexpr int kMergeBlocks = 2, kMergeWarps = 8;      // blocks of an SM, warps of a block

// 16 joined columns of a lane's query row, `head` in out and lse.
__device__ __forceinline__ void store_joined(const float (&acc)[16], float sum, float top, int w, int c, int64_t head,
                                             uint16_t* __restrict__ out, float* __restrict__ lse) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint4* to = reinterpret_cast<uint4*>(out + head * kDV + 128 * (w >> 1) + (c & 127) + 2 * (c & 128));
#pragma unroll
    for (int k = 0; k < 2; ++k)
        to[k] = make_uint4(pack_bf16x2(acc[8 * k] * inv, acc[8 * k + 1] * inv),
                           pack_bf16x2(acc[8 * k + 2] * inv, acc[8 * k + 3] * inv),
                           pack_bf16x2(acc[8 * k + 4] * inv, acc[8 * k + 5] * inv),
                           pack_bf16x2(acc[8 * k + 6] * inv, acc[8 * k + 7] * inv));
    if (lse && (w >> 1) == 0 && c == 0) lse[head] = sum == 0.f ? -INFINITY : top + log2f(sum) * kLn2;
}

// Joins one unit's pieces: 16 TMEM columns (from c, of warp w's quarter) of 32
// lanes, a lane per query row, whose head is at row `head` of out.  at(e): twice
// the slot of piece e, and which of the item's two rows this is.  By a block, a
// warp every 8th piece.
template <class At>
__device__ __forceinline__ void join_unit(const At& at, int pieces, int w, int c, int64_t head,
                                          const float* __restrict__ part_lse, const float4* __restrict__ part_o,
                                          uint16_t* __restrict__ out, float* __restrict__ lse,
                                          float (*acc_s)[18][32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int step = kMergeWarps;
    const int x = 32 * (w & 1) + lane;           // the lane's head
    auto piece_lse = [&](int e) -> float { return part_lse[at(e) * 64 + x]; };
    // eight pieces' sums at a time, with a running maximum
    float acc[16], sum = 0.f, top = -INFINITY;
    bool bad = false, nan = false;
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] = 0.f;
#pragma unroll 1
    for (int e1 = warp; e1 < pieces; e1 += 8 * step) {
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
            const float4* o = part_o + ((at(e1 + q * step) * 4 + w) * 64 + c / 4) * 32 + lane;
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
    if (warp != 0) return;
    if (top == INFINITY) return;                 // a bad page in one of the pieces
    store_joined(acc, sum, top, w, c, head + x, out, lse);
}

// The same for at most 8 pieces, by a warp, with half of all loads on their way at
// once.
template <class At>
__device__ __forceinline__ void join_few(const At& at, int pieces, int w, int c, int64_t head,
                                         const float* __restrict__ part_lse, const float4* __restrict__ part_o,
                                         uint16_t* __restrict__ out, float* __restrict__ lse) {
    const int lane = threadIdx.x & 31, x = 32 * (w & 1) + lane;
    float ls[8], top = -INFINITY, acc[16], sum = 0.f;
    bool bad = false, nan = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) ls[e] = e < pieces ? part_lse[at(e) * 64 + x] : -INFINITY;
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] = 0.f;
#pragma unroll 1
    for (int e0 = 0; e0 < pieces; e0 += 4) {
        float4 v[4][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4* o = part_o + ((at(min(e0 + e, pieces - 1)) * 4 + w) * 64 + c / 4) * 32 + lane;
#pragma unroll
            for (int k = 0; k < 4; ++k) v[e][k] = o[32 * k];
        }
        if (e0 == 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                bad = bad || ls[e] == INFINITY;
                nan = nan || ls[e] != ls[e];
                top = fmaxf(top, ls[e]);
            }
        }
        const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (e0 + e >= pieces) break;
            const float f = ex2_approx(((e0 == 0 ? ls[e] : ls[e + 4]) - base) * kLog2e);
            sum += f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                acc[4 * k] += f * v[e][k].x;
                acc[4 * k + 1] += f * v[e][k].y;
                acc[4 * k + 2] += f * v[e][k].z;
                acc[4 * k + 3] += f * v[e][k].w;
            }
        }
    }
    if (bad) return;                             // a bad page in one of the pieces
    if (nan) top = NAN;
    store_joined(acc, sum, top, w, c, head + x, out, lse);
}

// Joins the partial results of the items that shares cut.  A unit is 16 TMEM
// columns of a CTA's 32 lanes, a lane per query row.  Items of at most 8 pieces
// take a warp for each unit; those of many (one long sequence over the whole
// GPU: 10 MB of pieces) a block, whose warps take every 8th piece (1 x 100,000
// rows: 83 -> 30 us, merge included).  The blocks that fit the GPU at once find the
// items themselves and share out the units of all.
__global__ void __launch_bounds__(32 * kMergeWarps, kMergeBlocks)
    tree_merge_kernel(const int4* __restrict__ meta, int pairs, const float* __restrict__ part_lse,
                      const float4* __restrict__ part_o, uint16_t* __restrict__ out, float* __restrict__ lse) {
    __shared__ float acc_s[kMergeWarps][18][32];
    __shared__ int4 item_s[kMaxPairs];
    __shared__ int32_t narrow_s[kMaxPairs + 1], wide_s[kMaxPairs + 1];   // units before each pair's item
    const int tid = threadIdx.x, warp = tid >> 5;
    pdl_launch_dependents();
    pdl_wait();
    if (tid < 32) {
        constexpr int kEach = kMaxPairs / 32;
        int32_t narrow[kEach], wide[kEach], n = 0, w = 0;
        int4 it[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) it[k] = kEach * tid + k < pairs ? meta[kEach * tid + k] : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            // rows, if the pair begins the item
            const int32_t units = it[k].w == kEach * tid + k ? 64 * it[k].y : 0;
            const bool many = it[k].z - it[k].w >= kMergeWarps;
            item_s[kEach * tid + k] = it[k];
            n += narrow[k] = many ? 0 : units;
            w += wide[k] = many ? units : 0;
        }
        n = warp_scan_i32(n);
        w = warp_scan_i32(w);
        if (tid == 31) narrow_s[kMaxPairs] = n, wide_s[kMaxPairs] = w;
#pragma unroll
        for (int k = kEach - 1; k >= 0; --k) {
            narrow_s[kEach * tid + k] = n -= narrow[k];
            wide_s[kEach * tid + k] = w -= wide[k];
        }
    }
    __syncthreads();
    // unit u of the items that `before` counts
    auto join = [&](const int32_t* before, int32_t u, bool many) {
        const int pair = last_at_or_below(before, kMaxPairs, u), unit = u - before[pair], rank = unit >> 6;
        const int4 it = item_s[pair];
        // its pieces: the first pair's slot 2 pair + 1, then slots 2 p of the pairs
        // behind it
        auto at = [&](int e) -> int64_t {
            return 2 * (e == 0 ? 2 * (int64_t)pair + 1 : 2 * ((int64_t)pair + e)) + rank;
        };
        const int pieces = it.z - pair + 1, w = (unit >> 4) & 3, c = 16 * (unit & 15);
        const int64_t head = (int64_t)(it.x + rank) * kH;
        if (many) join_unit(at, pieces, w, c, head, part_lse, part_o, out, lse, acc_s);
        else join_few(at, pieces, w, c, head, part_lse, part_o, out, lse);
    };
    for (int32_t u = (int32_t)blockIdx.x; u < wide_s[kMaxPairs]; u += (int32_t)gridDim.x) join(wide_s, u, true);
    for (int32_t u = kMergeWarps * (int32_t)blockIdx.x + warp; u < narrow_s[kMaxPairs]; u += kMergeWarps * (int32_t)gridDim.x)
        join(narrow_s, u, false);
}

// The same by rows, without the search: for calls of few rows, where the code that
// a block meets for the first time is what counts (4 rows behind 2,000: 9.1 -> 6.0 us;
// whole calls of 49 behind 28 22.1 -> 20.5, 55 behind 1,931 34.9 -> 33.0).
__global__ void __launch_bounds__(32 * kMergeWarps)
    few_merge_kernel(const int2* __restrict__ rows, int pairs, const float* __restrict__ part_lse,
                     const float4* __restrict__ part_o, uint16_t* __restrict__ out, float* __restrict__ lse) {
    __shared__ float acc_s[kMergeWarps][18][32];
    const int warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    pdl_wait();
    const int2 it = rows[blockIdx.x];
    if (it.x == 0) return;                       // a row that one pair has done, or no row
    const int pair = (it.x >> 1) - 1, pieces = it.y - pair + 1;
    if (pair < 0 || pieces < 2 || it.y >= pairs) return;     // (left by a call that timed out)
    auto at = [&](int e) -> int64_t { return 2 * (2 * ((int64_t)pair + e) + (e == 0 ? 1 : 0)) + (it.x & 1); };
    const int64_t head = (int64_t)blockIdx.x * kH;
    if (pieces > kMergeWarps) {
        for (int u = (int)blockIdx.y; u < 64; u += (int)gridDim.y)
            join_unit(at, pieces, u >> 4, 16 * (u & 15), head, part_lse, part_o, out, lse, acc_s);
    } else {
        for (int u = kMergeWarps * (int)blockIdx.y + warp; u < 64; u += kMergeWarps * (int)gridDim.y)
            join_few(at, pieces, u >> 4, 16 * (u & 15), head, part_lse, part_o, out, lse);
    }
}

// Blocks of a merge: those of one wave, or as many as have a unit at most.
int merge_blocks(int pairs) { return std::min(kMergeBlocks * num_sms(), 128 * pairs); }

// The runs of a call behind shared prefixes, by one block.  A group counts if all
// groups together are the batch in order and each of its sequences with new rows
// keeps the shared ones; else its sequences are computed each by itself.  Two rows of
// different sequences make an item only where every sequence is within its bounds, so
// that a group's rows lie side by side.  kFew: a thread for each sequence and group
// at most, so that everything is loaded at once and the rest is shared memory's.
constexpr int kPlanThreads = 1024;

template <bool kFew>
__global__ void __launch_bounds__(kPlanThreads)
    prefix_plan_kernel(const BatchDev bd, const GroupsDev gr, RunPlan* plan, Run* runs, int32_t* tiles_all,
                       int32_t* lead_all, int pairs, int least_shared, int2* cut_rows, int32_t* status) {
    __shared__ int64_t s_units[kPlanThreads / 32];
    __shared__ int32_t s_longest[kPlanThreads / 32];
    __shared__ int32_t s_off[kFew ? kPlanThreads + 1 : 1], s_rows[kFew ? kPlanThreads : 1], s_q[kFew ? kPlanThreads + 1 : 1],
        s_ctx[kFew ? kPlanThreads : 1], s_tiles[kFew ? kPlanThreads : 1], s_lead[kFew ? kPlanThreads : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = (int)blockDim.x;
    pdl_launch_dependents();
    pdl_wait();
    // tiles that a group shares, and the sequence that they are read from
    int32_t* const tiles_of = kFew ? s_tiles : tiles_all;
    int32_t* const lead = kFew ? s_lead : lead_all;
    const int32_t* const off = kFew ? s_off : gr.off;
    const int32_t* const rows_of = kFew ? s_rows : gr.shared;
    const int32_t* const q_off = kFew ? s_q : bd.q_off;
    const int32_t* const ctx_len = kFew ? s_ctx : bd.ctx_len;
    SeqInfo mine{0, 0, 0};
    bool good = false, wrong = false, broken = false;
    if (cut_rows)
        for (int32_t i = tid; i < bd.total_q; i += threads) cut_rows[i] = make_int2(0, 0);
    if (kFew) {
        if (tid < bd.B) {
            good = load_seq(bd, tid, status, mine);
            s_q[tid] = mine.q0;
            s_ctx[tid] = mine.ctx;
            if (tid == bd.B - 1) s_q[bd.B] = mine.q0 + mine.nq;
        }
        if (tid < gr.n) {
            s_off[tid] = __ldg(gr.off + tid);
            s_rows[tid] = __ldg(gr.shared + tid);
            if (tid == gr.n - 1) s_off[gr.n] = __ldg(gr.off + gr.n);
        }
        __syncthreads();
    }
    for (int g = tid; g < gr.n; g += threads) {
        const int32_t lo = off[g], hi = off[g + 1];
        wrong = wrong || lo < 0 || lo > hi || hi > bd.B || (g == 0 && lo != 0) || (g == gr.n - 1 && hi != bd.B) ||
                rows_of[g] < 0;
        tiles_of[g] = max(rows_of[g], 0) / kTile;
        lead[g] = bd.B;
    }
    if (wrong) latch_status(status, DSA_ERR_BAD_BATCH);
    wrong = __syncthreads_or(wrong);
    for (int32_t i = tid; i < bd.B; i += threads) {
        if (!kFew) good = load_seq(bd, i, status, mine);
        broken = broken || !good;
        if (wrong || (good && mine.nq == 0)) continue;
        const int g = last_at_or_below(off, gr.n, i);
        if (good && rows_of[g] <= mine.ctx - mine.nq) {
            atomicMin(lead + g, i);
        } else {
            latch_status(status, DSA_ERR_BAD_BATCH);
            tiles_of[g] = 0;
        }
    }
    const bool alone = __syncthreads_or(broken) || wrong;
    int64_t units = 0;
    int32_t longest = 0;
    for (int32_t i0 = 0; i0 < bd.B; i0 += threads) {
        const int32_t i = i0 + tid;
        Run inner{}, tail{};
        if (i < bd.B) {
            if (!kFew) good = load_seq(bd, i, status, mine);
            if (good && mine.nq > 0) {
                const int g = wrong ? 0 : last_at_or_below(off, gr.n, i);
                inner.base = wrong ? 0 : tiles_of[g];
                // the rows that may make items with this sequence's
                const bool mixed = !alone && inner.base >= least_shared;
                const int32_t row0 = mixed ? q_off[off[g]] : mine.q0, row1 = mixed ? q_off[off[g + 1]] : mine.q0 + mine.nq;
                const int32_t skip = (mine.q0 - row0) & 1, rest = mine.nq - skip;
                inner.row = mine.q0 + skip;
                inner.items = rest >> 1;
                inner.rows = 2;
                inner.lead = inner.base > 0 ? lead[g] : 0;
                inner.b = i;
                inner.len = mine.ctx;
                inner.n = mine.nq;
                inner.i0 = skip;
                inner.lone = mixed && row1 - row0 <= 2;
                tail = inner;
                tail.row = mine.q0 + mine.nq - 1;
                tail.items = rest & 1;
                tail.rows = 1;
                tail.i0 = mine.nq - 1;
                if (tail.items && tail.row + 1 < row1) {
                    tail.rows = 2;
                    tail.b2 = last_at_or_below(q_off, bd.B, tail.row + 1);
                    tail.len2 = ctx_len[tail.b2];
                    tail.n2 = q_off[tail.b2 + 1] - q_off[tail.b2];
                }
            }
        }
        const int64_t cost = (int64_t)inner.items * (inner.tiles() + kItemCost);
        const int64_t both = cost + (int64_t)tail.items * (tail.tiles() + kItemCost);
        longest = max(longest, max(inner.items ? inner.tiles() : 0, tail.items ? tail.tiles() : 0));
        int64_t iu = both;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, iu, o);
            if (lane >= o) iu += u;
        }
        if (lane == 31) s_units[warp] = iu;
        __syncthreads();
        int64_t bu = units;
        for (int w = 0; w < threads / 32; ++w) {
            if (w < warp) bu += s_units[w];
            units += s_units[w];
        }
        if (i < bd.B) {
            inner.u = bu + iu - both;
            tail.u = inner.u + cost;
            runs[2 * i] = inner;
            runs[2 * i + 1] = tail;
        }
        if (!kFew) __syncthreads();
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) s_longest[warp] = longest;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < threads / 32; ++w) longest = max(longest, s_longest[w]);
        const int64_t even = (units + pairs - 1) / pairs;
        *plan = RunPlan{units, max(even, (int64_t)least_chunk(longest))};
    }
}

// Tiles that a group has to share for items of two sequences.  Such an item
// spares the second its walk over the shared tiles, but takes the own tiles of both
// in turn, with the end of each (see the fix-up).  Where there is little work for
// every pair, only if the shared tiles are half of the longest cache.  Apart and
// together, one call after another: 15 rows in 4 groups behind up to 188, up to 586 of their
// own, 16.6 and 17.0 us; 8 in 2 groups behind 1,000, 1,000 of their own, 17.5 and 18.8; 4 behind
// 2,000, 40 or 1,500 of their own, 18.9 and 18.0, 17.3 and 16.3.  It is a rule of thumb: 24
// behind 400, 300 of their own, would be faster together (17.8 and 17.1), 3 x 5 behind
// 1,500 and 6 x 3 behind 700 apart (15.4 and 16.6, 16.0 and 16.9).
int least_shared(const BatchDev& bd, int pairs) {
    const int64_t items = ((int64_t)bd.total_q + std::min(bd.total_q, bd.B)) / 2;
    const int tiles = (bd.max_ctx + kTile - 1) / kTile;
    return items * (tiles + kItemCost) <= (int64_t)kApartUnits * pairs ? std::max(1, (tiles + 1) / 2) : 1;
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
    if (cudaFuncSetAttribute(tree_mla_kernel<64, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem)) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, tree_mla_kernel<64, false>, &cfg) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        return num_sms() / 2;
    }
    n = std::min(n, std::min(num_sms() / 2, kMaxPairs));
    cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Tensor maps of the queries and of the cache, whose boxes go by its pages.
struct TreeMaps {
    CUtensorMap q, k, v;
    uint32_t rows;
    bool ok;
    TreeMaps(const Args& a, const uint16_t* queries) {
        const int page = a.pg.table ? 1 << a.pg.shift : kTile;
        rows = (uint32_t)std::min(page, 64);
        ok = make_tmap_bf16_2d(&q, queries, kDQK, (uint64_t)a.bd.total_q * kH, 64, 64) &&
             (rows == 64 ? make_tmap_bf16_chunks(&k, a.kv, kQChunks, (uint64_t)a.rows_total, rows, kGroup)
                          : make_tmap_bf16_groups(&k, a.kv, kQChunks, (uint64_t)a.rows_total, rows, kGroup)) &&
             make_tmap_bf16_chunks(&v, a.kv, kQChunks, (uint64_t)a.rows_total, rows, 2);
    }
};

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
    const TreeMaps maps(a, q);
    if (!maps.ok) return cudaErrorInvalidValue;
    auto kernel = maps.rows == 64   ? tree_mla_kernel<64, false>
                  : maps.rows == 32 ? tree_mla_kernel<32, false>
                                     : tree_mla_kernel<16, false>;
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
    if ((e = cudaLaunchKernelEx(&cfg, kernel, a, maps.q, maps.k, maps.v)) != cudaSuccess) return e;
    count_launches(1);
    cfg.gridDim = dim3((unsigned)merge_blocks(pairs));
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, tree_merge_kernel, (const int4*)a.meta, pairs, (const float*)a.part_lse,
                           (const float4*)a.part_o, out, lse);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

namespace {

struct PrefixScratch {
    size_t plan, tiles, lead, runs, meta, cut, lse, o, bytes;
    PrefixScratch(const BatchDev& bd, int32_t groups) {
        const size_t slots = 2 * (size_t)std::min(num_sms() / 2, kMaxPairs);
        size_t at = 0;
        auto take = [&](size_t n) {
            const size_t mine = at;
            at += (n + 255) / 256 * 256;
            return mine;
        };
        plan = take(sizeof(RunPlan));
        tiles = take(sizeof(int32_t) * (size_t)groups);
        lead = take(sizeof(int32_t) * (size_t)groups);
        runs = take(sizeof(Run) * 2 * (size_t)bd.B);
        meta = take(sizeof(int4) * slots / 2);
        cut = take(sizeof(int2) * std::min(bd.total_q, kFewRows));
        lse = take(sizeof(float) * 128 * slots);
        o = take(sizeof(float) * 128 * kDV * slots);
        bytes = at;
    }
};

}  // namespace

size_t prefix_mla_scratch_bytes(const BatchDev& bd, int32_t groups) {
    return PrefixScratch(bd, groups).bytes;
}

cudaError_t launch_prefix_mla(const BatchDev& bd, const GroupsDev& gr, const PagesDev& pg, const uint16_t* q,
                              const uint16_t* kv, const uint64_t* mask, float sm_scale, uint16_t* out, float* lse,
                              void* scratch, int32_t* status, cudaStream_t stream) {
    const int pairs = max_pairs();
    const PrefixScratch at(bd, gr.n);
    uint8_t* const mem = static_cast<uint8_t*>(scratch);
    Args a{};
    a.bd = bd;
    a.pg = pg;
    a.mask = mask;
    a.kv = kv;
    a.scale_log2 = sm_scale * kLog2e;
    a.out = out;
    a.lse = lse;
    a.status = status;
    a.part_o = reinterpret_cast<float*>(mem + at.o);
    a.part_lse = reinterpret_cast<float*>(mem + at.lse);
    a.groups = gr;
    a.least_shared = least_shared(bd, pairs);
    a.runs_total = 2 * bd.B;
    a.meta = reinterpret_cast<int4*>(mem + at.meta);
    const bool few_rows = bd.total_q <= kFewRows;
    a.cut_rows = few_rows ? reinterpret_cast<int2*>(mem + at.cut) : nullptr;
    a.rows_total = pg.table ? pg.pool_pages << pg.shift : (int32_t)(bd.B * bd.stride);
    const TreeMaps maps(a, q);
    if (!maps.ok) return cudaErrorInvalidValue;
    auto kernel = maps.rows == 64   ? tree_mla_kernel<64, true>
                  : maps.rows == 32 ? tree_mla_kernel<32, true>
                                     : tree_mla_kernel<16, true>;
    constexpr size_t kSmem = sizeof(SmemOf<SharedSeg>);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int32_t n = std::max(gr.n, bd.B);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // (a launch of its own costs 2-4 us: 4 rows behind 2,000 20.5 -> 18.5, 2 behind 300 18.5 -> 16.6)
    if (n > 32) {
        RunPlan* plan = reinterpret_cast<RunPlan*>(mem + at.plan);
        Run* runs = reinterpret_cast<Run*>(mem + at.runs);
        a.rplan = plan;
        a.runs = runs;
        const bool few = n <= kPlanThreads;
        cfg.gridDim = dim3(1);
        cfg.blockDim = dim3(few ? (n + 31) / 32 * 32 : kPlanThreads);
        e = cudaLaunchKernelEx(&cfg, few ? prefix_plan_kernel<true> : prefix_plan_kernel<false>, bd, gr, plan, runs,
                               reinterpret_cast<int32_t*>(mem + at.tiles), reinterpret_cast<int32_t*>(mem + at.lead), pairs,
                               a.least_shared, a.cut_rows, status);
        if (e != cudaSuccess) return e;
        count_launches(1);
    }
    cfg.gridDim = dim3(2 * (unsigned)pairs);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    if ((e = cudaLaunchKernelEx(&cfg, kernel, a, maps.q, maps.k, maps.v)) != cudaSuccess) return e;
    count_launches(1);
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.dynamicSmemBytes = 0;
    if (few_rows) {
        // (a wave of blocks)
        const int units = (kMergeBlocks * num_sms() / bd.total_q + kMergeWarps - 1) / kMergeWarps * kMergeWarps;
        cfg.gridDim = dim3((unsigned)bd.total_q, std::clamp(units, kMergeWarps, 64));
        e = cudaLaunchKernelEx(&cfg, few_merge_kernel, (const int2*)a.cut_rows, pairs, (const float*)a.part_lse,
                               (const float4*)a.part_o, out, lse);
    } else {
        cfg.gridDim = dim3((unsigned)merge_blocks(pairs));
        e = cudaLaunchKernelEx(&cfg, tree_merge_kernel, (const int4*)a.meta, pairs, (const float*)a.part_lse,
                               (const float4*)a.part_o, out, lse);
    }
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace dsa
