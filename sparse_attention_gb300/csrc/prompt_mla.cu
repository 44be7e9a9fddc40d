// prompt_mla.cu -- causal attention of prompts over expanded rows: 64 heads,
// keys of 192 + 64 columns (the 64 shared by all heads), values of 256.
//
// A CTA pair takes an item: a head, and 256 consecutive new rows of a sequence
// (128 of them each CTA).  It walks the rows' keys in tiles of 128 positions:
//   S[256 q, 128 pos] = Q K^T     each CTA stages its 128 query rows (64 KiB,
//                                 resident) and 64 of the tile's keys
//   P = 2^(S c - m)               the running maximum m of a row moves only when
//                                 a score exceeds it by 2^8 (then O is
//                                 rescaled); P is rounded to bf16 for the
//                                 product, the MMA's type, its sum taken before
//                                 in fp32: an error of half a bf16 step of a
//                                 weight, like the result's own rounding
//   O[256 q, 256] += P V          each CTA stages 128 of the value columns of
//                                 all 128 positions
// O (256 TMEM columns) and two S tiles (128 each) fill a CTA's TMEM, a lane per
// query row; nothing but barriers and item numbers crosses between the CTAs.  P
// takes the place of its S, half the columns of each of the two threads of a
// row: from shared memory it would cost 64 KB a tile of a bandwidth that Q, K
// and V already use for 192 (128 bytes a cycle; a tile took 2,680 cycles, 2,090
// so).
// S of tile g + 1 is issued before PV of tile g, so the softmax of a tile runs
// under the tensor work of the next.
//
// What is masked cannot leak: expanded values are finite (a row that is not
// carries NaN in its key instead), rows behind a sequence up to the next multiple
// of 16 are zero, and the product with the values ends at such a multiple
// behind the last position that a row of the item sees.  A masked score is
// replaced by -inf before anything is formed of it, its weight is 0, and 0 times a
// finite value is 0.  (Tiles of keys go on to multiples of 128, which a
// sequence's room holds.)
//
// The new rows of a sequence are cut into 256s from their end, so that a
// remainder has the fewest keys (12 prompts of 839 to 2,012 rows: 420 tiles a pair
// cut from the front, 401 from the end).
//
// Items are taken from a counter, all query tiles of a head before the next
// head's, longest first: pairs that run together then read the same keys (a
// pair alone reads 128 KB a tile, 9 TB/s over the GPU; in step they come from
// L2), and short items fill the end.  The order decides which pair computes an item,
// never what it computes.
//
// Where sequences have at most 128 new rows an item is those, at M = 128 (kFew
// below).
//
// Roles of a CTA's 16 warps: K loads, MMA (rank 0 only), Q and V loads, items,
// eight softmax warps (two threads share a query row, 64 positions each),
// four that write results (an item's O is read out under the first S and softmax of
// the next).
//
// Bounds.  A tile is 16 MMAs of N = 128 and 8 of N = 256: 2,048 cycles for
// 33.6 MFLOP at M = 256.  An item costs 3,000 cycles more: its first S waits for its
// queries, which take the place of those of the item before, and its first PV for the
// softmax of that.  Measured, in single calls and in a loop that the power cap
// slows: 16,384 tokens 4.35-4.40 ms = 2,000-2,020 TFLOP/s (cuBLAS 1,921) and
// 5.0-5.05 ms = 1,740-1,760 (1,730 sustained); 12 prompts of 839 to 2,012 tokens
// 0.59-0.60 ms and 0.68-0.72, 401 tiles a pair for the 319 that the mask leaves.
#include <algorithm>
#include <atomic>

#include "internal.h"
#include "prompt.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kTile = 128;                   // positions per tile
constexpr int kMmaRows = 256;                // rows of an item and M of a pair's MMA, but where all have at most ..
constexpr int kFewRows = 128;                // .. these
constexpr int kThreads = 512;
constexpr int kSoftWarps = 8, kOutWarps = 4;
constexpr int kQBytes = 128 * 128;           // 128 rows x 64 columns
constexpr int kKBytes = 64 * 128;            // 64 rows x 64 columns
constexpr int kQChunks = kHeadQK / 64;       // 4
constexpr int kStages = 2;                   // whole tiles of K and of V
constexpr uint32_t kOCol = 0, kSCol = 256;   // TMEM columns
constexpr int kMaxSlots = 8;                 // items published ahead, at most
constexpr int kMaxPairs = 96;
constexpr float kRescale = 8.f;              // log2
static_assert(kTile == kExpRoom, "a sequence's room holds whole tiles");

struct Item {
    int32_t row;                 // packed row of the first of its query rows
    int32_t rows;                // how many there are
    int32_t pos;                 // position of the first
    int32_t at;                  // expanded row of position 0
    int32_t head, tiles;         // no tiles: nothing left
};

struct Smem {
    alignas(1024) uint8_t q[kQChunks * kQBytes];
    alignas(1024) uint8_t k[kStages * kQChunks * kKBytes];
    alignas(1024) uint8_t v[kStages * 2 * kQBytes];      // two blocks of 64 columns x 128 positions
    alignas(1024) uint8_t out[kOutWarps * 4096];         // results on their way out; kFew: P, two blocks of 64 rows x 64 positions
    alignas(8) uint64_t kfull[kStages], kempty[kStages], vfull[kStages], vempty[kStages];
    uint64_t qfull[kQChunks], qempty[kQChunks], sfull[2], pfull[2], pvdone[2], odone[2], lfull[2], invfree[2], ofree[2], followed[2], itemfull[kMaxSlots], itemempty[kMaxSlots];
    uint64_t numfull[kMaxSlots], numempty[kMaxSlots];          // item numbers on their way to rank 1
    Item item[kMaxSlots];
    uint32_t number[kMaxSlots];
    float xch[2][32 * kSoftWarps];
    alignas(16) int4 seq[kThreads];                      // the plan of a batch of few sequences: first new row, how many,
    int32_t start[kThreads + 1], sums[kThreads / 32];    // .. length, first expanded row; query tiles before it
    float inv[128];                                      // 1 / the sum of a finished item's row
    uint32_t tmem;
};
static_assert(sizeof(Smem) <= 232448, "one CTA's shared memory");

struct Args {
    BatchDev bd;
    ExpandedDev x;
    float scale_log2;
    uint16_t* out;
    float* lse;
    const int32_t* start;        // [B + 1] query tiles before a sequence; nullptr: each CTA sums them up itself
    uint32_t* next;              // items that pairs have taken behind their first ones, and pairs that are done; 0 between launches
    int32_t* status;
};

// Sequence b: its first new row, how many there are, its length, and where its
// expanded rows begin; no new rows for one that breaks the bounds.
__device__ __forceinline__ int4 sequence(const BatchDev& bd, const ExpandedDev& x, int b, int32_t* status) {
    if (b >= bd.B) return make_int4(0, 0, 0, 0);
    SeqInfo s;
    const int32_t lo = __ldg(x.off + b), hi = __ldg(x.off + b + 1);      // with the lengths, not behind them
    if (!load_seq(bd, b, status, s) || s.nq == 0) return make_int4(0, 0, 0, 0);
    const int32_t at = expanded_at(x, lo, hi, s.ctx, status);
    return at < 0 ? make_int4(0, 0, 0, 0) : make_int4(s.q0, s.nq, s.ctx, at);
}
template <int R>
__device__ __forceinline__ int32_t tiles_of(int32_t rows) {
    return (rows + R - 1) / R;
}

// Query tiles before each sequence, for batches of more than kThreads (a launch
// more: 4 us).
template <int R>
__global__ void __launch_bounds__(1024)
    prompt_plan_kernel(const BatchDev bd, const ExpandedDev x, int32_t* start, int32_t* status) {
    __shared__ int32_t sums[32];
    const int tid = threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    if (tid == 0) start[0] = 0;
    int32_t carry = 0;
    for (int b0 = 0; b0 < bd.B; b0 += 1024) {
        const int32_t n = tiles_of<R>(sequence(bd, x, b0 + tid, status).y);
        int32_t all;
        const int32_t before = block_sum_before(n, 32, sums, all);
        if (b0 + tid < bd.B) start[b0 + tid + 1] = carry + before + n;
        carry += all;
        __syncthreads();
    }
}

template <int R>
__device__ __forceinline__ Item item_of(const Args& a, const Smem& S, uint32_t number) {
    Item it{0, 0, 0, 0, 0, 0};
    const int32_t* const start = a.start ? a.start : S.start;
    if (number >= (uint32_t)start[a.bd.B] * kH) return it;
    const int b = last_at_or_below(start, a.bd.B, (int32_t)(number / kH));
    const uint32_t tiles = (uint32_t)(start[b + 1] - start[b]), in = number - (uint32_t)start[b] * kH;
    const int4 s = a.start ? sequence(a.bd, a.x, b, nullptr) : S.seq[b];
    const int32_t end = s.y - R * (int32_t)(in % tiles), i0 = max(0, end - R);
    if (end <= 0) return it;                     // lengths that change under the call
    it.head = (int32_t)(in / tiles);
    it.row = s.x + i0;
    it.rows = end - i0;
    it.pos = s.z - s.y + i0;
    it.at = s.w;
    it.tiles = (it.pos + it.rows - 1) / kTile + 1;
    return it;
}

// kFew: items of 128 rows at most, 64 each CTA's, and M = 128: half the tensor work
// of a tile, and a row's S and O in two lanes and half the columns, so that two O
// and two S fit TMEM beside each other and an item's results are read out under the
// next one's products.  What a short item waits for is latency, so its parts overlap those of
// its neighbours: queries in two buffers, items published eight ahead, four softmax
// warps an item in turn.  P goes through shared memory (as A in TMEM it would
// need its rows once in each half of the lanes).  Pairs take every pairs-th item instead of asking
// (an answer takes 2 us, a short item 1.4).  Taken where the bound on new rows is 128 and below (28
// prompts of 20 to 49 tokens 41-43 us, 75 without; 32 of 32 45, 83 without; 8 of 8 behind
// 445 31, 38 without; 32 of 128 94-96, 101 without; one of 100 10.3, 12.4; 32 of 33 to 100 behind up
// to 1,000 224-227, 242 without: HBM).
template <bool kFew>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prompt_mla_kernel(const Args a, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_pe,
                      const __grid_constant__ CUtensorMap tm_q16, const __grid_constant__ CUtensorMap tm_kv16,
                      const __grid_constant__ CUtensorMap tm_pe16) {
    constexpr int R = kFew ? kFewRows : kMmaRows, kMine = R / 2;     // rows of an item, and of a CTA
    constexpr int kQRows = kMine * 128;                              // bytes of a chunk of them
    constexpr int kQBufs = kFew ? 2 : 1, kOBufs = kFew ? 2 : 1;
    // items published ahead: of short ones the warps that write results are two
    // behind the loads (32 prompts of 32 tokens 61 us with two, 46 with eight);
    // a pair that asks for its items takes none too early
    constexpr int kSlots = kFew ? kMaxSlots : 2;
    // columns of an S and of an O: with M = 128 a row's are in two lanes
    constexpr uint32_t kSCols = kFew ? kTile / 2 : kTile, kOCols = kFew ? kHeadV / 2 : kHeadV;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem& S = *reinterpret_cast<Smem*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    pdl_launch_dependents();
    if (smem_u32(smem_raw) & 1023u) {            // the swizzle goes by address bits
        if (tid == 0) latch_status(a.status, DSA_ERR_INTERNAL);
        return;                                  // both CTAs: the same launch, the same offset
    }
    if (tid == 128) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&S.kfull[i]), 2);
            mbar_init(smem_u32(&S.kempty[i]), 1);
            mbar_init(smem_u32(&S.vfull[i]), 2);
            mbar_init(smem_u32(&S.vempty[i]), 1);
        }
        for (int i = 0; i < kQChunks; ++i) {
            mbar_init(smem_u32(&S.qfull[i]), 2);
            mbar_init(smem_u32(&S.qempty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&S.sfull[i]), 1);
            mbar_init(smem_u32(&S.pfull[i]), 2 * kSoftWarps / kOBufs);
            mbar_init(smem_u32(&S.pvdone[i]), 1);
        }
        for (int i = 0; i < kOBufs; ++i) {
            mbar_init(smem_u32(&S.lfull[i]), kSoftWarps / (kFew ? 4 : 2));
            mbar_init(smem_u32(&S.invfree[i]), kOutWarps);
            mbar_init(smem_u32(&S.odone[i]), 1);
            mbar_init(smem_u32(&S.ofree[i]), 2 * kOutWarps);
            if (kFew) mbar_init(smem_u32(&S.followed[i]), kSoftWarps / 2);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(smem_u32(&S.itemfull[i]), 1);
            mbar_init(smem_u32(&S.itemempty[i]), kSoftWarps + kOutWarps + (rank == 0 ? 3 : 2));   // the warps that read items
            mbar_init(smem_u32(&S.numfull[i]), 1);
            mbar_init(smem_u32(&S.numempty[i]), 1);
        }
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc_pair(smem_u32(&S.tmem), 512);
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        prefetch_tmap(&tm_pe);
        prefetch_tmap(&tm_q16);
        prefetch_tmap(&tm_kv16);
        prefetch_tmap(&tm_pe16);
    }
    __syncwarp();
    cluster_arrive();                            // the peer may use this CTA's barriers and TMEM ..
    pdl_wait();                                  // inputs, and the scratch of an earlier call
    if (!a.start) {
        S.seq[tid] = sequence(a.bd, a.x, tid, a.status);
        const int32_t n = tiles_of<R>(S.seq[tid].y);
        int32_t all;
        S.start[tid + 1] = block_sum_before(n, kThreads / 32, S.sums, all) + n;
        if (tid == 0) S.start[0] = 0;
    }
    tc_fence_before();
    __syncthreads();
    cluster_wait();                              // .. and this CTA the peer's
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    Item it;
    bool ok = true;
    // the barrier at `b`'s offset in the CTA of rank 0
    auto lead = [&](uint64_t& b) -> uint32_t { return map_to_cluster_rank(smem_u32(&b), 0); };
    // bounded; a thread whose wait expired waits for nothing any more
    auto wait = [&](uint64_t& b, uint32_t parity) -> bool {
        ok = ok && mbar_wait_small(smem_u32(&b), parity, a.status);
        return ok;
    };
    // the next item that warp 3 published; false behind the last
    uint32_t items_read = 0;
    auto next_item = [&](Item& to) -> bool {
        const uint32_t slot = items_read % kSlots;
        wait(S.itemfull[slot], (items_read / kSlots) & 1);
        ok = __all_sync(0xffffffffu, ok);
        to = S.item[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&S.itemempty[slot]));
        ++items_read;
        return ok && to.tiles > 0;
    };

    if (warp == 0 || warp == 2) {
        // K or V loads: lane 0 waits, then each lane issues a box.  Before an
        // item's V its Q, a chunk as soon as the last S of the item before (kFew:
        // of the one before that) is through with it: not before its K, which
        // need not wait for that.  kFew: a tile that the item's keys do not fill
        // comes in boxes of 16 rows, and so do fewer than a CTA's 64 queries, since
        // the rest of a sequence's room would be read from HBM for nothing (16
        // prompts of 16 tokens behind 48 37 -> 31 us; in long items it is not
        // worth the code).  What then lies in the other rows is masked or not multiplied, or
        // becomes nobody's lanes.
        const bool k = warp == 0;
        uint64_t* const full = k ? S.kfull : S.vfull;
        uint64_t* const empty = k ? S.kempty : S.vempty;
        // K: the head's three chunks, and by lane 1 the shared one; V: two
        const int boxes = k ? 2 : 1;
        const bool pe = k && lane == 1;
        constexpr uint32_t kBytes = kQChunks * kKBytes;          // of a stage of K, and of V
        static_assert(kBytes == 2 * kQBytes, "");
        const uint32_t stages = smem_u32(k ? S.k : S.v), to = stages + (pe ? (kQChunks - 1) * kKBytes : 0);
        const int32_t chunk = k ? 0 : kNope / 64 + 2 * (int)rank, row = k ? 64 * (int)rank : 0;
        // boxes of 16 rows: the lane's chunk and place in it
        const int wide = k ? 4 : 8, c16 = lane / wide, r16 = 16 * (lane % wide);
        const uint32_t to16 = stages + c16 * (k ? kKBytes : kQBytes) + r16 * 128;
        const bool pe16 = k && c16 == kQChunks - 1;
        uint32_t g = 0, seg = 0;
        for (; next_item(it); ++seg) {
            if (!k && kFew) {
                const uint32_t b = seg % kQBufs, use = seg / kQBufs, bar = lead(S.qfull[b]);
                const int n16 = (min(kMine, max(0, it.rows - kMine * (int)rank)) + 15) / 16;
                if (lane == 0 && (use == 0 || wait(S.qempty[b], (use - 1) & 1)))
                    mbar_arrive_expect_tx_pair(bar, n16 * kQChunks * 16 * 128);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                const uint32_t at = smem_u32(S.q + b * kQChunks * kQRows);
                const int32_t col = it.head * kHeadQK, first = it.row + kMine * (int)rank;
                if (ok && n16 == kMine / 16 && lane < kQChunks)
                    tma_load_2d_pair(at + lane * kQRows, &tm_q, bar, col + 64 * lane, first);
                if (ok && n16 < kMine / 16 && lane < 4 * kQChunks && (lane & 3) < n16)
                    tma_load_2d_pair(at + (lane >> 2) * kQRows + (lane & 3) * 2048, &tm_q16, bar, col + 64 * (lane >> 2),
                                     first + 16 * (lane & 3));
            }
            if (!k && !kFew) {
                for (int q = 0; ok && q < kQChunks; ++q) {
                    if (lane == 0 && (seg == 0 || wait(S.qempty[q], (seg - 1) & 1))) {
                        mbar_arrive_expect_tx_pair(lead(S.qfull[q]), kQRows);
                        tma_load_2d_pair(smem_u32(S.q + q * kQRows), &tm_q, lead(S.qfull[q]), it.head * kHeadQK + 64 * q,
                                         it.row + kMine * (int)rank);
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                }
            }
            for (int32_t t = 0; ok && t < it.tiles; ++t, ++g) {
                const uint32_t st = g % kStages, bar = lead(full[st]);
                // 16s of the item's keys here
                const int n16 = kFew ? min(wide, (max(0, it.pos + it.rows - t * kTile - row) + 15) / 16) : wide;
                if (lane == 0 && (g < kStages || wait(empty[st], (g / kStages - 1) & 1)))
                    mbar_arrive_expect_tx_pair(bar, n16 * (kBytes / wide));
                ok = __shfl_sync(0xffffffffu, ok, 0);
                const int32_t r = it.at + t * kTile + row, c = it.head * (kExpRow / 64) + chunk;
                if (ok && n16 == wide) {
                    if (pe) tma_load_2d_pair(to + st * kBytes, &tm_pe, bar, 0, r);
                    else if (lane < boxes) tma_load_3d_pair(to + st * kBytes, k ? &tm_k : &tm_v, bar, 0, r, c);
                } else if (ok && lane < 16 && r16 < 16 * n16) {
                    if (pe16) tma_load_2d_pair(to16 + st * kBytes, &tm_pe16, bar, 0, r + r16);
                    else tma_load_3d_pair(to16 + st * kBytes, &tm_kv16, bar, 0, r + r16, c + c16);
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            // MMA, by one lane that also waits: S of a tile, then PV of the one
            // before; an item's first S behind the last PV before it, under which
            // its queries are loaded (but kFew).  One loop over all tiles of all
            // items, and the next item is read behind the last S of one: what is
            // met once an item is fetched as it goes (15 cycles an instruction),
            // and nothing else runs meanwhile.
            constexpr uint32_t kIdS = idesc_bf16_f32(R, kTile);
            constexpr uint32_t kIdO = idesc_bf16_f32(R, kHeadV, false, true);
            const uint64_t dq = sdesc_sw128(smem_u32(S.q), 0, 1024), dk = sdesc_sw128(smem_u32(S.k), 0, 1024);
            const uint64_t dv = sdesc_sw128(smem_u32(S.v), kQBytes, 1024), dp = sdesc_sw128(smem_u32(S.out), 0, 1024);
            int32_t tiles = 0, keys = 0;         // of item `seg`
            uint32_t seg = 0, n = 0;             // n: tiles whose S is issued
            auto read = [&]() {
                const uint32_t slot = seg % kSlots;
                tiles = 0;
                if (!wait(S.itemfull[slot], (seg / kSlots) & 1)) return;
                tiles = S.item[slot].tiles;
                keys = S.item[slot].pos + S.item[slot].rows;
                mbar_arrive(smem_u32(&S.itemempty[slot]));
            };
            read();
            // the tile whose PV is next: its number, steps of 16 positions that some row sees, place in its item
            uint32_t m = 0, m_seg = 0;
            int32_t steps = 0;
            bool pending = false, m_first = false, m_last = false;
#pragma unroll 1
            for (int32_t t = 0; ok;) {
                const bool s_now = tiles > 0 && (kFew || t > 0 || !pending);
                if (!s_now && !pending) break;
                const bool first = t == 0, last = t + 1 == tiles;
                const uint32_t mine = seg;
                int32_t seen = 0;
                if (s_now) {
                    const uint32_t buf = n & 1, st = n % kStages;
                    if (!wait(S.kfull[st], (n / kStages) & 1)) break;
                    if (kFew && first && !wait(S.qfull[seg % kQBufs], (seg / kQBufs) & 1)) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < kQChunks; ++c) {
                        if (!kFew && first) {
                            if (!wait(S.qfull[c], seg & 1)) break;
                            tc_fence_after();
                        }
                        const uint64_t da = dq + ((kFew ? seg % kQBufs * kQChunks + c : c) * kQRows >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16_ss_pair(tmem + kSCol + kSCols * buf, da + 2 * k,
                                             dk + (st * kQChunks + c) * (kKBytes >> 4) + 2 * k, kIdS, (c | k) != 0);
                        if (!kFew && last) mma_commit_pair(smem_u32(&S.qempty[c]));
                    }
                    if (!ok) break;
                    if (kFew && last) mma_commit_pair(smem_u32(&S.qempty[seg % kQBufs]));
                    mma_commit_pair(smem_u32(&S.kempty[st]));
                    mma_commit_pair(smem_u32(&S.sfull[buf]));
                    ++n;
                    seen = min(kTile, keys - t * kTile + 15) / 16;
                    ++t;
                }
                if (pending) {
                    const uint32_t st = m % kStages;
                    const uint32_t ob = m_seg % kOBufs, use = m_seg / kOBufs;
                    if (m_first && use > 0 && !wait(S.ofree[ob], (use - 1) & 1)) break;
                    if (!wait(S.vfull[st], (m / kStages) & 1)) break;
                    if (!wait(S.pfull[m & 1], (m >> 1) & 1)) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int k = 0; k < steps; ++k) {
                        const uint64_t db = dv + st * (2 * kQBytes >> 4) + 128 * k;
                        if (kFew)
                            mma_bf16_ss_pair(tmem + kOCol + kOCols * ob, dp + (k >> 2) * (kQRows >> 4) + 2 * (k & 3), db, kIdO,
                                             !m_first || k != 0);
                        else
                            mma_bf16_ts_pair(tmem + kOCol, tmem + kSCol + kSCols * (m & 1) + 64 * (k >> 2) + 8 * (k & 3), db,
                                             kIdO, !m_first || k != 0);
                    }
                    mma_commit_pair(smem_u32(&S.vempty[st]));
                    mma_commit_pair(smem_u32(&S.pvdone[m % kOBufs]));
                    if (m_last) mma_commit_pair(smem_u32(&S.odone[ob]));
                }
                if (s_now && last) {
                    t = 0;
                    ++seg;
                    read();
                }
                pending = s_now;
                m = n - 1;
                m_seg = mine;
                m_first = first;
                m_last = last;
                steps = seen;
            }
        }
        __syncwarp();
    } else if (warp == 3) {
        // items: rank 0 takes their numbers and passes them on; their queries
        // are brought to L2 ahead
        for (uint32_t n = 0; ok; ++n) {
            const uint32_t slot = n % kSlots, turn = n / kSlots;
            uint32_t number = 0;
            auto wait_peer = [&](uint64_t& b, uint32_t parity) {
                if (ok && !mbar_wait_peer(smem_u32(&b), parity)) {
                    ok = false;
                    latch_status(a.status, DSA_ERR_TIMEOUT);
                }
            };
            if (lane == 0) {
                if (n >= kSlots) wait(S.itemempty[slot], (turn - 1) & 1);
                if (kFew) {
                    number = (blockIdx.x >> 1) + n * (gridDim.x >> 1);
                } else if (ok && rank == 0) {
                    number = n == 0 ? blockIdx.x >> 1 : (gridDim.x >> 1) + atomicAdd(a.next, 1u);
                    if (n >= kSlots) wait_peer(S.numempty[slot], (turn - 1) & 1);
                    if (ok) {
                        st_peer_u32(map_to_cluster_rank(smem_u32(&S.number[slot]), 1), number);
                        mbar_arrive_peer(map_to_cluster_rank(smem_u32(&S.numfull[slot]), 1));
                    }
                } else if (ok) {
                    wait_peer(S.numfull[slot], turn & 1);
                    number = *reinterpret_cast<volatile uint32_t*>(&S.number[slot]);
                    if (ok) mbar_arrive_peer(lead(S.numempty[slot]));
                }
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            it = item_of<R>(a, S, __shfl_sync(0xffffffffu, number, 0));
            if (lane == 0) {
                S.item[slot] = it;
                mbar_arrive(smem_u32(&S.itemfull[slot]));
            }
            __syncwarp();
            if (kFew) {
                if (lane < 4 * kQChunks && kMine * (int)rank + 16 * (lane & 3) < it.rows)
                    tma_prefetch_2d(&tm_q16, it.head * kHeadQK + 64 * (lane >> 2), it.row + kMine * (int)rank + 16 * (lane & 3));
            } else if (it.tiles > 0 && lane < kQChunks) {
                tma_prefetch_2d(&tm_q, it.head * kHeadQK + 64 * lane, it.row + kMine * (int)rank);
            }
            __syncwarp();
            if (it.tiles == 0) break;
        }
    } else if (kFew && warp < 4 + kSoftWarps) {
        // softmax: four warps an item, in turn, so that an item's end and the next
        // one's first tile go on side by side.  TMEM lanes x and 64 + x have row
        // x's first and last 64 positions.
        const int mine = (tid - 128) >> 7, ln = tid & 127, x = ln & 63, half = ln >> 6;
        const uint32_t tl = tmem + ((uint32_t)(ln & 96) << 16);
        float* const xch = S.xch[mine];
        uint32_t g = 0, seg = 0, xb = 0;
        auto exchange = [&](float v) -> float {
            xb ^= 128;
            xch[xb + ln] = v;
            named_bar_sync(1 + mine, 128);
            return xch[xb + (ln ^ 64)];
        };
        for (; !named_bar_or(1 + mine, 128, !next_item(it)); ++seg) {
            if ((int)(seg & 1) != mine) {
                // The other group's item.  Nothing holds its S back for this group, and a
                // barrier's parity tells only two phases apart, so this group does not
                // watch them: the other one signals when its item's last S is done.  (Its next
                // signal comes behind this group's next item, so these phases cannot pass unseen.)
                wait(S.followed[mine ^ 1], (seg >> 1) & 1);
                g += it.tiles;
                continue;
            }
            const int32_t first = it.pos + kMine * (int)rank;    // position of the CTA's first row
            const int32_t live = min(kMine, it.rows - kMine * (int)rank);
            const bool idle = (x & ~31) >= live;                 // such a warp keeps in step with the others
            float m = -INFINITY, l = 0.f;
            for (int32_t t = 0; t < it.tiles; ++t, ++g) {
                const uint32_t buf = g & 1;
                wait(S.sfull[buf], (g >> 1) & 1);
                __syncwarp();
                tc_fence_after();
                if (t + 1 == it.tiles && lane == 0) mbar_arrive(smem_u32(&S.followed[mine]));
                if (idle) {
                    // (what P holds there becomes nobody's lanes of O)
                    exchange(0.f);
                    if (lane == 0) mbar_arrive_pair(lead(S.pfull[buf]));
                    continue;
                }
                uint32_t r[2][32];
                tmem_ld_32x32b_x32(tl + kSCol + kSCols * buf, r[0]);
                tmem_ld_32x32b_x32(tl + kSCol + kSCols * buf + 32, r[1]);
                tmem_ld_wait();
                if ((t + 1) * kTile - 1 > first) {
                    const int32_t d = first + x - (t * kTile + 64 * half);       // the last column that the row sees
#pragma unroll
                    for (int k = 0; k < 64; ++k)
                        if (k > d) r[k >> 5][k & 31] = 0xFF800000u;
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
                // P is read, O at rest (PV of tile g - 2 is done: S of tile g was issued behind it)
                if (g > 0) wait(S.pvdone[(g - 1) & 1], ((g - 1) >> 1) & 1);
                __syncwarp();
                tc_fence_after();
                if (t > 0 && __any_sync(0xffffffffu, f != 1.f)) {
                    const uint32_t at = tl + kOCol + kOCols * (seg % kOBufs);
#pragma unroll 1
                    for (uint32_t c = 0; c < kOCols; c += 16) {
                        uint32_t v[16];
                        tmem_ld_32x32b_x16(at + c, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * f);
                        tmem_st_32x32b_x16(at + c, v);
                    }
                    tmem_st_wait();
                }
                uint8_t* const to = S.out + half * kQRows + x * 128;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<uint4*>(to + ((k ^ (x & 7)) << 4)) =
                        make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(lead(S.pfull[buf]));
            }
            // Every row sees itself, so l > 0 but where every score is -inf: NaN, as of the formula.
            l += exchange(l);
            if (half == 0) {
                if (seg > 1) wait(S.invfree[mine], ((seg >> 1) - 1) & 1);
                S.inv[kMine * mine + x] = rcp_approx(l);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&S.lfull[mine]));
                if (a.lse && x < live)
                    a.lse[(int64_t)(it.row + kMine * (int)rank + x) * kH + it.head] = (m + lg2_approx(l)) * kLn2;
            }
        }
    } else if (warp < 4 + kSoftWarps) {
        // softmax: TMEM lane = query row of this CTA
        const int ln = tid - 128, x = ln & 127, half = ln >> 7;
        const uint32_t tl = tmem + ((uint32_t)(x & ~31) << 16);
        uint32_t g = 0, seg = 0, xb = 0;
        auto exchange = [&](float v) -> float {
            xb ^= 1;
            S.xch[xb][ln] = v;
            named_bar_sync(1, 32 * kSoftWarps);
            return S.xch[xb][ln ^ 128];
        };
        // the warps agree on each item, since they meet at barriers
        while (!named_bar_or(1, 32 * kSoftWarps, !next_item(it))) {
            const int32_t first = it.pos + kMine * (int)rank;    // position of the CTA's first row
            // rows of this CTA; a warp without one keeps in step with the others
            const int32_t live = min(kMine, it.rows - kMine * (int)rank);
            const bool idle = (x & ~31) >= live;
            float m = -INFINITY, l = 0.f;
            for (int32_t t = 0; t < it.tiles; ++t, ++g) {
                const uint32_t buf = g & 1;
                wait(S.sfull[buf], (g >> 1) & 1);
                __syncwarp();
                tc_fence_after();
                if (idle) {
                    exchange(0.f);
                    if (lane == 0) mbar_arrive_pair(lead(S.pfull[buf]));
                    continue;
                }
                uint32_t r[2][32];
                tmem_ld_32x32b_x32(tl + kSCol + kTile * buf + 64 * half, r[0]);
                tmem_ld_32x32b_x32(tl + kSCol + kTile * buf + 64 * half + 32, r[1]);
                tmem_ld_wait();
                if ((t + 1) * kTile - 1 > first) {
                    const int32_t d = first + x - (t * kTile + 64 * half);       // the last column that the row sees
#pragma unroll
                    for (int k = 0; k < 64; ++k)
                        if (k > d) r[k >> 5][k & 31] = 0xFF800000u;
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
                if (t > 0 && __any_sync(0xffffffffu, f != 1.f)) {
                    wait(S.pvdone[0], (g - 1) & 1);
                    __syncwarp();
                    tc_fence_after();
#pragma unroll 1
                    for (uint32_t c = 0; c < 128; c += 16) {
                        uint32_t o[16];
                        tmem_ld_32x32b_x16(tl + kOCol + 128 * half + c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        tmem_st_32x32b_x16(tl + kOCol + 128 * half + c, o);
                    }
                }
                // P over the first half of the columns that this warp's part of S had
                tmem_st_32x32b_x32(tl + kSCol + kTile * buf + 64 * half, pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(lead(S.pfull[buf]));
            }
            // Every row sees itself, so l > 0 but where every score is -inf: NaN, as of the formula.
            l += exchange(l);
            if (half == 0) {
                if (seg > 0) wait(S.invfree[0], (seg - 1) & 1);
                S.inv[x] = rcp_approx(l);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&S.lfull[0]));
                if (a.lse && x < live)
                    a.lse[(int64_t)(it.row + kMine * (int)rank + x) * kH + it.head] = (m + lg2_approx(l)) * kLn2;
            }
            ++seg;
        }
    } else if (kFew) {
        // results: TMEM lanes x and 64 + x have row x's first and last 128 columns
        const int r0 = 32 * (warp & 1), half = (warp >> 1) & 1;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const bool odd = lane & 1;
        uint32_t seg = 0;
        while (next_item(it)) {
            const uint32_t ob = seg % kOBufs;
            wait(S.lfull[ob], (seg / kOBufs) & 1);
            wait(S.odone[ob], (seg / kOBufs) & 1);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            const float inv = S.inv[kMine * ob + r0 + lane];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.invfree[ob]));
            const int32_t mine = it.row + kMine * (int)rank + r0, live = min(kMine, it.rows - kMine * (int)rank) - r0;
            if (ok && live > 0) {
                // two lanes write their two rows in turn, 32 bytes of a row at a time
                const int32_t even = lane & ~1;
                uint16_t* const to = a.out + ((int64_t)(mine + even) * kH + it.head) * kHeadV + 128 * half + (odd ? 8 : 0);
#pragma unroll 1
                for (uint32_t c = 0; c < kOCols; c += 32) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(tl + kOCol + kOCols * ob + c, o);
                    tmem_ld_wait();
                    if (c == kOCols - 32) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_pair(lead(S.ofree[ob]));
                    }
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        uint32_t w[8], in[4];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            w[k] = pack_bf16x2(__uint_as_float(o[16 * v + 2 * k]) * inv,
                                               __uint_as_float(o[16 * v + 2 * k + 1]) * inv);
#pragma unroll
                        for (int k = 0; k < 4; ++k) in[k] = __shfl_xor_sync(0xffffffffu, odd ? w[k] : w[4 + k], 1);
                        if (even < live)
                            *reinterpret_cast<uint4*>(to + c + 16 * v) =
                                odd ? make_uint4(in[0], in[1], in[2], in[3]) : make_uint4(w[0], w[1], w[2], w[3]);
                        if (even + 1 < live)
                            *reinterpret_cast<uint4*>(to + (int64_t)kH * kHeadV + c + 16 * v) =
                                odd ? make_uint4(w[4], w[5], w[6], w[7]) : make_uint4(in[0], in[1], in[2], in[3]);
                    }
                }
            }
            if (!(ok && live > 0)) {
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(lead(S.ofree[ob]));
            }
            ++seg;
        }
    } else {
        // results: TMEM lane = query row of this CTA
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const int r0 = 32 * (warp & 3);
        // through shared memory, so that a store covers whole lines of 4 rows
        uint8_t* const stage = S.out + (warp & 3) * 4096;
        uint32_t seg = 0;
        while (next_item(it)) {
            wait(S.lfull[0], seg & 1);
            wait(S.odone[0], seg & 1);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            const float inv = S.inv[r0 + lane];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.invfree[0]));
            const int32_t mine = it.row + kMine * (int)rank + r0, live = min(kMine, it.rows - kMine * (int)rank) - r0;
            if (ok && live > 0) {
                uint16_t* const to = a.out + ((int64_t)mine * kH + it.head) * kHeadV + 8 * (lane & 7);
#pragma unroll 1
                for (uint32_t c = 0; c < 256; c += 64) {
                    uint32_t o[2][32];
                    tmem_ld_32x32b_x32(tl + kOCol + c, o[0]);
                    tmem_ld_32x32b_x32(tl + kOCol + c + 32, o[1]);
                    tmem_ld_wait();
                    if (c == 192) {              // O is free before its last columns are written
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_pair(lead(S.ofree[0]));
                    }
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = pack_bf16x2(__uint_as_float(o[v >> 2][8 * (v & 3) + 2 * k]) * inv,
                                               __uint_as_float(o[v >> 2][8 * (v & 3) + 2 * k + 1]) * inv);
                        *reinterpret_cast<uint4*>(stage + lane * 128 + ((v ^ (lane & 7)) << 4)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int row = 4 * k + (lane >> 3);
                        if (row < live)
                            *reinterpret_cast<uint4*>(to + (int64_t)row * kH * kHeadV + c) =
                                *reinterpret_cast<const uint4*>(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
                    }
                    __syncwarp();
                }
            }
            if (!(ok && live > 0)) {
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(lead(S.ofree[0]));
            }
            ++seg;
        }
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
    // the last pair leaves the counters as it found them
    if (tid == 0 && rank == 0) {
        const uint32_t last = (gridDim.x >> 1) - 1;
        __threadfence();
        if (atomicInc(a.next + 1, last) == last) *a.next = 0u;
    }
}

}  // namespace

int resident_pairs(const void* f, int threads, size_t smem, int most) {
    constexpr int kMaxDevices = 64, kMaxKernels = 8;
    static std::atomic<uintptr_t> key[kMaxKernels];
    static std::atomic<int> cache[kMaxKernels][kMaxDevices];
    int dev = 0, n = 0, slot = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return std::min(kDefaultSMs / 2, most);
    }
    for (; slot < kMaxKernels; ++slot) {
        uintptr_t none = 0, mine = reinterpret_cast<uintptr_t>(f);
        if (key[slot].compare_exchange_strong(none, mine) || none == mine) break;
    }
    if (slot < kMaxKernels && (n = cache[slot][dev].load(std::memory_order_relaxed)) > 0) return std::min(n, most);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * num_sms());
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, f, &cfg) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        return std::min(num_sms() / 2, most);
    }
    n = std::min(n, num_sms() / 2);
    if (slot < kMaxKernels) cache[slot][dev].store(n, std::memory_order_relaxed);
    return std::min(n, most);
}

size_t prompt_mla_scratch_bytes(const BatchDev& bd) { return ((size_t)bd.B + 1) * sizeof(int32_t); }

namespace {

template <bool kFew>
cudaError_t launch(const BatchDev& bd, const uint16_t* q, const ExpandedDev& x, float sm_scale, uint16_t* out,
                   float* lse, void* scratch, int32_t* status, cudaStream_t stream) {
    constexpr int R = kFew ? kFewRows : kMmaRows;
    const auto kernel = prompt_mla_kernel<kFew>;
    // no more pairs than the batch's bounds allow items
    const int64_t items = ((int64_t)bd.total_q / R + std::min<int64_t>(bd.B, bd.total_q)) * kH;
    const int pairs = (int)std::min<int64_t>(
        resident_pairs(reinterpret_cast<const void*>(kernel), kThreads, sizeof(Smem), kMaxPairs), items);
    Args a{};
    a.bd = bd;
    a.x = x;
    a.scale_log2 = sm_scale * kLog2e;
    a.out = out;
    a.lse = lse;
    a.next = reinterpret_cast<uint32_t*>(status) + kCounterWord;
    a.status = status;
    CUtensorMap tm_q, tm_k, tm_v, tm_pe, tm_q16, tm_kv16, tm_pe16;
    if (!make_tmap_bf16_2d(&tm_q, q, (uint64_t)kH * kHeadQK, (uint64_t)bd.total_q, 64, R / 2) ||
        !make_tmap_bf16_chunks(&tm_k, x.kv, (uint64_t)kH * kExpRow / 64, (uint64_t)x.rows, 64, kNope / 64) ||
        !make_tmap_bf16_chunks(&tm_v, x.kv, (uint64_t)kH * kExpRow / 64, (uint64_t)x.rows, kTile, 2) ||
        !make_tmap_bf16_2d(&tm_pe, x.k_pe, DSA_ROPE_DIM, (uint64_t)x.rows, 64, 64) ||
        !make_tmap_bf16_2d(&tm_q16, q, (uint64_t)kH * kHeadQK, (uint64_t)bd.total_q, 64, 16) ||
        !make_tmap_bf16_chunks(&tm_kv16, x.kv, (uint64_t)kH * kExpRow / 64, (uint64_t)x.rows, 16, 1) ||
        !make_tmap_bf16_2d(&tm_pe16, x.k_pe, DSA_ROPE_DIM, (uint64_t)x.rows, 64, 16))
        return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    if (bd.B > kThreads) {
        int32_t* start = static_cast<int32_t*>(scratch);
        a.start = start;
        cfg.gridDim = dim3(1);
        cfg.blockDim = dim3(1024);
        if ((e = cudaLaunchKernelEx(&cfg, prompt_plan_kernel<R>, bd, x, start, status)) != cudaSuccess) return e;
        count_launches(1);
    }
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem))) != cudaSuccess)
        return e;
    cfg.gridDim = dim3(2 * (unsigned)pairs);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Smem);
    e = cudaLaunchKernelEx(&cfg, kernel, a, tm_q, tm_k, tm_v, tm_pe, tm_q16, tm_kv16, tm_pe16);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace

// By the bounds on new rows and lengths alone, so that a captured call serves others.
cudaError_t launch_prompt_mla(const BatchDev& bd, const uint16_t* q, const ExpandedDev& x, float sm_scale,
                              uint16_t* out, float* lse, void* scratch, int32_t* status, cudaStream_t stream) {
    // no expanded rows: no room holds a sequence, which that kernel's first blocks latch
    if (x.rows == 0 || prompt_rows_suit(bd)) return launch_prompt_rows(bd, q, x, sm_scale, out, lse, status, stream);
    return bd.max_q <= kFewRows ? launch<true>(bd, q, x, sm_scale, out, lse, scratch, status, stream)
                                : launch<false>(bd, q, x, sm_scale, out, lse, scratch, status, stream);
}

}  // namespace dsa
