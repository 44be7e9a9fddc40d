// topk.cu -- deterministic causal top-k of indexer score rows.
//
// ("GLM-5.1 架构深度拆解", section 3.6 Steps 6-7: positions s > t are masked
// and min(index_topk, length) positions are kept; section 3.4: the
// selection must be deterministic; the GLM-5 explainer page: a query that
// sees fewer than 2048 positions keeps all of them.)
//
// One thread-block cluster of C CTAs per query row (C = 1 unless rows are
// long and few); CTA r owns the r-th contiguous slice of the row.  Scores
// map to order-preserving 32-bit keys (-0.0 folded onto +0.0).
//   1. A lower bound L for the k-th largest key: the lower edge of the
//      11-bit digit bin (the digit just below the bits all sampled keys
//      share) holding the (r+1)-th largest of 1024 evenly spaced keys of the
//      whole row, r sized so that well over k keys lie at or above it.
//      Every CTA of the cluster derives the same L.
//   2. One pass over the slice (16-byte loads, several in flight): warp w of
//      a CTA owns a contiguous segment and appends its keys >= L, in
//      position order, to a shared-memory region of its own (keys are
//      tested as floats against L; one warp scan per step places them).
//   3. The exact k-th largest key tau among the candidates of the cluster:
//      a radix select over the bits below those that L and the largest
//      candidate share (digits of up to 11 bits); each CTA counts
//      its candidates and every CTA sums the cluster's histograms through
//      distributed shared memory, so all derive the same digits.
//   4. The output in position order: candidates above tau and the first
//      `need` candidates equal to tau (ties go to the lower position), each
//      written at its rank; ranks add the counts of lower warps and lower
//      CTAs.  Positions come out ascending.
// Every key that is not a candidate lies below L <= tau, so the result is
// exactly the top-k of the row.  If the sample misjudges (fewer than k
// candidates in the cluster, or a full region) steps 3-4 run over the whole
// slices instead.  Atomics only count; the result is the same bit for bit
// on every run.
//
// Under a visibility mask (a tree of drafted tokens) a row's candidates are
// its committed positions, then the new positions whose bit is set, taken as
// one row without gaps: the at most 64 visible new scores are packed in
// shared memory and stand in for the row's end wherever it is read, and
// positions are mapped back as they are written.  The selection itself is the
// same code, so -inf scores and ties come out as they would on such a row.
// Masked rows that fit shared memory take a kernel of their own (below).
#include <cooperative_groups.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"
#include "tree.h"

namespace cg = cooperative_groups;

namespace dsa {
namespace {

// Threads per CTA: 1024 when a launch has fewer rows than SMs (one CTA per
// SM, more warps to hide latency), else 512 (two CTAs per SM).
constexpr int kBins = 2048;
constexpr int kSample = 512;
constexpr int kRegion = 512;                 // candidate slots per warp
constexpr int kPrefetch = 8;                 // 16-byte loads in flight per lane (32 keys)
static_assert(kPrefetch <= 8, "a lane's candidate flags fill one 32-bit word, its counts one 64-bit word");
constexpr int kMaxCluster = 8;
constexpr int kLongRow = 65536;              // rows above this may be split over a cluster
constexpr int kKeysPerCta = 32768;
constexpr int kShortRow = 49152;             // masked rows up to this stay in shared memory (192 KB)
constexpr int kRowOf256 = 10240;             // and take a CTA of 256 threads up to this (four or five per SM),
constexpr int kRowOf512 = 24576;             // of 512 up to this (two or three per SM),
constexpr int kFewRowOf512 = 16384;          // or this when there are few (one per SM);
constexpr int kAloneRow = 24576;             // few rows above this are split over a cluster
constexpr int kSlice = 12288;                // into slices of at most this

__device__ __forceinline__ uint32_t order_key(float f) {
    uint32_t u = __float_as_uint(f);
    if (u == 0x80000000u) u = 0u;     // -0.0 compares equal to +0.0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The float whose key is `key` (inverse of order_key; +0.0 for the key of
// zero).  For non-NaN x: x >= key_float(key) exactly when order_key(x) >= key,
// provided key_float(key) is not a NaN.
__device__ __forceinline__ float key_float(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

__device__ __forceinline__ uint32_t warp_inclusive_scan(uint32_t v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t n = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += n;
    }
    return v;
}

template <int NT, int REGION = kRegion>
struct alignas(16) TopkSmem {
    static constexpr int kMaxCand = NT / 32 * REGION;
    uint32_t hist[kBins];                 // zero between selects
    uint32_t sample[REGION > 1 ? kSample : 1];
    uint32_t cand_key[kMaxCand];          // warp w: [w * kRegion, w * kRegion + count)
    int32_t cand_pos[kMaxCand];
    uint32_t warp_sums[32];
    uint32_t wcnt[32], wgt[32], weq[32], wmax[32];
    uint32_t group[kBins / 32];           // this CTA's counts of 64 groups of 32 bins (cluster selects)
    uint32_t small[64];                   // this CTA's keys of a small boundary bin
    uint32_t small_all[64];               // the bin's keys of the whole cluster
    uint32_t total, sel_digit, sel_above, sel_count, chunk_total;
    uint32_t small_n, small_all_n, small_tau, small_need;
    uint32_t cta_cand, cta_overflow, cta_gt, cta_eq, cta_max;   // read by the rest of the cluster
    uint32_t all_cand, all_overflow, all_max, pre_gt, pre_eq;    // the cluster's, combined by warp 0
};

// The k-th largest of the keys that `visit` hands to this thread's callback,
// over this CTA (nranks == 1) or over the whole cluster (nranks == cluster
// size).  Every such key agrees with `prefix0` above its low `hi` bits;
// those bits are resolved from the top in digits of up to 11 bits, at most
// `passes` of them (enough passes = exact).  Returns tau (the bits found,
// zero below) and sets need = how many keys matching tau belong to the top
// k.  Starting below the bits the keys share keeps them spread over many
// bins (few atomic collisions).  Once at most 64 keys (over the cluster)
// remain in the boundary bin, they are gathered and ranked directly.  S.hist must
// be zero on entry; zero on return.
template <int NT, int REGION, typename Visit>
__device__ uint32_t radix_select(cg::cluster_group& cluster, int nranks, TopkSmem<NT, REGION>& S, uint32_t k, int hi,
                                 uint32_t prefix0, int passes, Visit visit, uint32_t& need_out) {
    constexpr int kWarps = NT / 32, kBinsPerThread = kBins / NT;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t pmask = hi >= 32 ? 0u : ~((1u << hi) - 1u);
    uint32_t prefix = prefix0 & pmask, need = k;
    int top = hi;
#pragma unroll 1
    for (int p = 0; p < passes && top > 0; ++p) {
        const int sh = max(0, top - 11);
        const uint32_t dmask = (1u << (top - sh)) - 1u;
        top = sh;
        visit([&](uint32_t key) {
            if ((key & pmask) == prefix) atomicAdd(&S.hist[(key >> sh) & dmask], 1u);
        });
        if (nranks > 1) {
            // Over a cluster: the group of 32 bins that holds the need-th
            // largest key, from every rank's 64 group counts, then its bin
            // from every rank's 32 counts of that group (the bin the flat
            // scan below would find, from 3 % of the remote reads).
            constexpr int kGroups = kBins / 32;
            __syncthreads();                           // this rank's histogram is complete
            if (tid < kGroups) {
                uint32_t g = 0u;
#pragma unroll 8
                for (int b2 = 0; b2 < 32; ++b2) g += S.hist[32 * tid + b2];
                S.group[tid] = g;
            }
            cluster.sync();                            // every rank's group counts are ready
            if (warp == 0) {
                // lane l: groups 2l and 2l + 1, summed over the ranks in rank order
                uint32_t g0 = 0u, g1 = 0u;
                {
                    uint32_t r0[kMaxCluster], r1[kMaxCluster];
#pragma unroll
                    for (int r = 0; r < kMaxCluster; ++r) {
                        const uint32_t* h = cluster.map_shared_rank(S.group, (unsigned)min(r, nranks - 1));
                        r0[r] = r < nranks ? h[2 * lane] : 0u;
                        r1[r] = r < nranks ? h[2 * lane + 1] : 0u;
                    }
#pragma unroll
                    for (int r = 0; r < kMaxCluster; ++r) {
                        g0 += r0[r];
                        g1 += r1[r];
                    }
                }
                const uint32_t incl = warp_inclusive_scan(g0 + g1);
                const uint32_t total = __shfl_sync(0xffffffffu, incl, 31);
                const uint32_t above1 = total - incl;  // keys in groups above 2l + 1
                const uint32_t above0 = above1 + g1;   // keys in groups above 2l
                int grp = -1;
                uint32_t gabove = 0u;
                if (above1 < need && need <= above1 + g1) {
                    grp = 2 * (int)lane + 1;
                    gabove = above1;
                } else if (above0 < need && need <= above0 + g0) {
                    grp = 2 * (int)lane;
                    gabove = above0;
                }
                const uint32_t has = __ballot_sync(0xffffffffu, grp >= 0);
                const int src = has ? __ffs(has) - 1 : 0;
                grp = __shfl_sync(0xffffffffu, grp, src);
                gabove = __shfl_sync(0xffffffffu, gabove, src);
                if (has) {
                    // lane l: bin 32 grp + l, summed over the ranks in rank order
                    uint32_t rb[kMaxCluster];
#pragma unroll
                    for (int r = 0; r < kMaxCluster; ++r) {
                        const uint32_t* h = cluster.map_shared_rank(S.hist, (unsigned)min(r, nranks - 1));
                        rb[r] = r < nranks ? h[32 * grp + lane] : 0u;
                    }
                    uint32_t cb = 0u;
#pragma unroll
                    for (int r = 0; r < kMaxCluster; ++r) cb += rb[r];
                    const uint32_t bincl = warp_inclusive_scan(cb);
                    const uint32_t gtot = __shfl_sync(0xffffffffu, bincl, 31);
                    const uint32_t above = gabove + (gtot - bincl);   // keys in higher bins
                    if (above < need && need <= above + cb) {
                        S.sel_digit = (uint32_t)(32 * grp + (int)lane);
                        S.sel_above = above;
                        S.sel_count = cb;
                    }
                }
                if (lane == 0) S.total = total;
            }
            cluster.sync();                            // every remote read done before any bin is cleared
#pragma unroll
            for (int x = 0; x < kBinsPerThread; ++x) S.hist[kBinsPerThread * tid + x] = 0u;
            __syncthreads();
        } else {
            // thread tid owns bins [kBinsPerThread tid, kBinsPerThread (tid + 1))
            uint32_t c[kBinsPerThread];
            uint32_t mine = 0u;
            __syncthreads();
#pragma unroll
            for (int x = 0; x < kBinsPerThread; ++x) c[x] = S.hist[kBinsPerThread * tid + x];
#pragma unroll
            for (int x = 0; x < kBinsPerThread; ++x) {
                S.hist[kBinsPerThread * tid + x] = 0u;
                mine += c[x];
            }
            // keys in higher bins = total - inclusive scan in bin order
            const uint32_t incl_w = warp_inclusive_scan(mine);
            if (lane == 31) S.warp_sums[warp] = incl_w;
            __syncthreads();
            if (warp == 0) {
                const uint32_t v = lane < kWarps ? S.warp_sums[lane] : 0u;
                const uint32_t sc = warp_inclusive_scan(v);
                if (lane < kWarps) S.warp_sums[lane] = sc;
                if (lane == kWarps - 1) S.total = sc;
            }
            __syncthreads();
            uint32_t above = S.total - (incl_w + (warp ? S.warp_sums[warp - 1] : 0u));
#pragma unroll
            for (int x = kBinsPerThread - 1; x >= 0; --x) {
                if (above < need && need <= above + c[x]) {
                    S.sel_digit = (uint32_t)(kBinsPerThread * tid + x);
                    S.sel_above = above;
                    S.sel_count = c[x];
                }
                above += c[x];
            }
            __syncthreads();
        }
        need -= S.sel_above;
        prefix |= S.sel_digit << sh;
        pmask |= dmask << sh;
        if (passes > 1 && top > 0 && S.sel_count <= 64u) {
            // at most 64 keys (in the cluster) share the digits found so far:
            // gather them and rank them exactly instead of more passes
            if (tid == 0) S.small_n = 0u;
            __syncthreads();
            visit([&](uint32_t key) {
                if ((key & pmask) == prefix) {
                    const uint32_t at = atomicAdd(&S.small_n, 1u);
                    if (at < 64u) S.small[at] = key;
                }
            });
            if (nranks == 1) __syncthreads();
            else cluster.sync();
            // every rank's list, concatenated in rank order
            auto rank_smem = [&](int r) -> const TopkSmem<NT, REGION>* {
                return nranks == 1 ? &S : cluster.map_shared_rank(&S, r);
            };
            if (tid < 64 * nranks) {
                const int r = tid >> 6, e = tid & 63;
                // every rank's list length, loaded at once (predicated)
                uint32_t len[kMaxCluster];
#pragma unroll
                for (int r2 = 0; r2 < kMaxCluster; ++r2)
                    len[r2] = r2 < nranks ? min(rank_smem(min(r2, nranks - 1))->small_n, 64u) : 0u;
                uint32_t off = 0u, mine = 0u, tot = 0u;
#pragma unroll
                for (int r2 = 0; r2 < kMaxCluster; ++r2) {
                    off += r2 < r ? len[r2] : 0u;
                    mine = r2 == r ? len[r2] : mine;
                    tot += len[r2];
                }
                if ((uint32_t)e < mine && off + (uint32_t)e < 64u) S.small_all[off + e] = rank_smem(r)->small[e];
                if (tid == 0) S.small_all_n = min(tot, 64u);
            }
            __syncthreads();
            // thread t ranks key t / 8 against keys 8 (t % 8) .. 8 (t % 8) + 7;
            // eight lanes sum their counts
            for (uint32_t ranker = (uint32_t)tid; ranker < 512u; ranker += NT) {
                const uint32_t nb = S.small_all_n;
                const uint32_t q = ranker >> 3, sub = ranker & 7u;
                const uint32_t x = q < nb ? S.small_all[q] : 0u;
                uint32_t gt = 0u, eq = 0u;
#pragma unroll
                for (uint32_t o = 0; o < 8u; ++o) {
                    const uint32_t qq = sub * 8u + o;
                    const uint32_t y = S.small_all[qq];
                    gt += (qq < nb && y > x) ? 1u : 0u;
                    eq += (qq < nb && y == x) ? 1u : 0u;
                }
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) {
                    gt += __shfl_xor_sync(0xffffffffu, gt, o);
                    eq += __shfl_xor_sync(0xffffffffu, eq, o);
                }
                // tau: the key with fewer than `need` larger keys and at least
                // `need` keys at or above it (every such thread agrees)
                if (sub == 0 && q < nb && gt < need && need <= gt + eq) {
                    S.small_tau = x;
                    S.small_need = need - gt;
                }
            }
            __syncthreads();
            prefix = S.small_tau;
            need = S.small_need;
            break;
        }
    }
    need_out = need;
    return prefix;
}

// Number of low bits in which keys of [lo, hi] may differ.
__device__ __forceinline__ int varying_bits(uint32_t lo, uint32_t hi) {
    return lo == hi ? 0 : 32 - __clz((int)(lo ^ hi));
}

// Exclusive prefix over the cluster's lower ranks of the CTA counts (gt, eq)
// stored in S.cta_gt / S.cta_eq; call after a cluster barrier.
template <int NT>
__device__ __forceinline__ void cluster_prefix(cg::cluster_group& cluster, int crank, TopkSmem<NT>& S,
                                               uint32_t& gt0, uint32_t& eq0) {
    // lane r of warp 0 loads lower rank r's counts (one remote read per
    // rank, not one per thread), the warp sums them, the CTA shares them
    if ((threadIdx.x >> 5) == 0) {
        const int r = (int)(threadIdx.x & 31);
        const TopkSmem<NT>* o = cluster.map_shared_rank(&S, (unsigned)min(r, max(crank - 1, 0)));
        uint32_t g = r < crank ? o->cta_gt : 0u, e = r < crank ? o->cta_eq : 0u;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            g += __shfl_xor_sync(0xffffffffu, g, off);
            e += __shfl_xor_sync(0xffffffffu, e, off);
        }
        if (r == 0) {
            S.pre_gt = g;
            S.pre_eq = e;
        }
    }
    __syncthreads();
    gt0 = S.pre_gt;
    eq0 = S.pre_eq;
}

// out[pos] = v for a rank pos < k; a rank outside the row would be a bug:
// it is skipped and latched instead of written.
__device__ __forceinline__ void put(int32_t* out, uint32_t pos, int k, int32_t v, int32_t* status) {
    if (pos < (uint32_t)k) out[pos] = v;
    else latch_status(status, DSA_ERR_INTERNAL);
}

// A masked row's end: packs its visible new scores and their positions
// (threads 0-63 write; the caller synchronises) and returns the row's length
// without gaps, c committed positions first.
__device__ __forceinline__ int32_t masked_end(const SeqInfo& sq, int32_t i, const float* row, const uint64_t* mask,
                                              float* end_score, int32_t* end_pos) {
    const int tid = threadIdx.x;
    const int32_t c = sq.ctx - sq.nq;
    const uint64_t bits = visible_bits(__ldg(reinterpret_cast<const unsigned long long*>(mask) + sq.q0 + i), i);
    if (tid < DSA_MAX_TREE && (bits >> tid) & 1u) {
        const int e = __popcll(bits & ((1ull << tid) - 1u));
        end_score[e] = __ldg(row + c + tid);
        end_pos[e] = c + tid;
    }
    return c + __popcll(bits);
}

template <int NT, bool MASKED>
__global__ void __launch_bounds__(NT, NT <= 512 ? 2 : 1)
    topk_kernel(const BatchDev bd, const RowRange rr, const float* __restrict__ scores, const int64_t ld,
                const int scores_local, const int k, int32_t* __restrict__ idx, const int idx_local,
                const int csize, int32_t* status, const uint64_t* __restrict__ mask) {
    constexpr int kThreads = NT, kWarps = NT / 32, kBinsPerThread = kBins / NT;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    TopkSmem<NT>& S = *reinterpret_cast<TopkSmem<NT>*>(smem_raw);
    cg::cluster_group cluster = cg::this_cluster();

    // every test below depends only on the row, so all CTAs of a cluster
    // take the same branch and reach the same cluster barriers
    pdl_launch_dependents();     // a dependent attention may start launching
    pdl_wait();                  // the scores of the previous launch are complete
    const int b = blockIdx.y;
    SeqInfo sq;
    if (!load_seq(bd, b, status, sq)) return;
    const int crank = (int)(blockIdx.x % (unsigned)csize);
    const int32_t i = rr.i0 + (int32_t)(blockIdx.x / (unsigned)csize);
    if (i >= min(rr.i1, sq.nq)) return;
    const int32_t t = sq.ctx - sq.nq + i;
    const float* row = scores + buf_row(scores_local, sq, b, i, rr) * ld;
    int32_t* out = idx + buf_row(idx_local, sq, b, i, rr) * (int64_t)k;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // the row's end under a mask: visible new scores and their positions
    __shared__ float end_score[MASKED ? DSA_MAX_TREE : 1];
    __shared__ int32_t end_pos[MASKED ? DSA_MAX_TREE : 1];
    const int32_t c = MASKED ? sq.ctx - sq.nq : 0;
    int32_t n = t + 1;
    if constexpr (MASKED) {
        n = masked_end(sq, i, row, mask, end_score, end_pos);
        __syncthreads();
    }
    auto position = [&](int32_t j) -> int32_t {
        if constexpr (MASKED) return j < c ? j : end_pos[j - c];
        else return j;
    };
    // a barrier over every thread that shares this row
    auto sync_row = [&]() {
        if (csize == 1) __syncthreads();
        else cluster.sync();
    };

    if (n <= k) {  // every causal position is selected
        if (crank == 0)
            for (int j = tid; j < k; j += kThreads) out[j] = j < n ? position(j) : -1;
        return;
    }
    auto row_key = [&](int32_t j) -> uint32_t {
        if constexpr (MASKED)
            if (j >= c) return order_key(end_score[j - c]);
        return order_key(__ldg(row + j));
    };

    // this CTA's slice [s_lo, s_hi) of the row (slices start on multiples of 128)
    const int32_t span = ((n + csize - 1) / csize + 127) & ~127;
    const int32_t s_lo = min(n, crank * span), s_hi = min(n, s_lo + span);

    // 1. the lower bound L (the same in every CTA): digits start below the
    // bits that all sample keys share
    const int32_t ns = min(n, kSample);
#pragma unroll
    for (int x = 0; x < kBinsPerThread; ++x) S.hist[kBinsPerThread * tid + x] = 0u;
    uint32_t smin = 0xFFFFFFFFu, smax = 0u;
    for (int q = tid; q < ns; q += kThreads) {
        const uint32_t key = row_key((int32_t)(((int64_t)q * n) / ns));
        S.sample[q] = key;
        smin = min(smin, key);
        smax = max(smax, key);
    }
    smin = __reduce_min_sync(0xffffffffu, smin);
    smax = __reduce_max_sync(0xffffffffu, smax);
    if (lane == 0) {
        S.wgt[warp] = smin;
        S.weq[warp] = smax;
    }
    __syncthreads();
    smin = __reduce_min_sync(0xffffffffu, lane < kWarps ? S.wgt[lane] : 0xFFFFFFFFu);
    smax = __reduce_max_sync(0xffffffffu, lane < kWarps ? S.weq[lane] : 0u);
    const float expect = (float)k * (float)ns / (float)n;
    const int32_t r = min(ns - 1, (int32_t)(1.25f * expect + 3.f * sqrtf(expect)) + 8);
    uint32_t unused;
    const uint32_t L = radix_select(cluster, 1, S, (uint32_t)(r + 1), varying_bits(smin, smax), smin, 1,
                                    [&](auto&& f) {
                                        for (int q = tid; q < ns; q += kThreads) f(S.sample[q]);
                                    },
                                    unused);

    // 2. one pass: warp w appends its keys >= L to its region, in position
    // order.  A step covers 128 x kPrefetch consecutive keys: lane l loads
    // the 16-byte groups l, l + 32, ... (coalesced, all in flight at once).
    // Keys are tested as floats against the float of L (the same order as
    // the keys, -0.0 == +0.0).  The per-group candidate counts of a lane
    // travel through one 64-bit warp scan (8-bit fields), which places every
    // candidate of the step in position order; their keys are read again
    // after the pass.
    const int32_t seg = ((s_hi - s_lo + kWarps - 1) / kWarps + 127) & ~127;
    const int32_t w_lo = min(s_hi, s_lo + warp * seg), w_hi = min(s_hi, w_lo + seg);
    uint32_t* rk = S.cand_key + warp * kRegion;
    int32_t* rp = S.cand_pos + warp * kRegion;
    const float Lf = key_float(L);
    uint32_t cnt = 0u;
    float fmx = -INFINITY;
    for (int32_t jb = w_lo; jb < w_hi; jb += 128 * kPrefetch) {
        float4 v[kPrefetch];
#pragma unroll
        for (int u = 0; u < kPrefetch; ++u) {
            const int32_t j = jb + 128 * u + 4 * (int32_t)lane;   // a multiple of 4 inside the padded row
            v[u] = j < w_hi ? __ldg(reinterpret_cast<const float4*>(row + j)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const bool tail = jb + 128 * kPrefetch > w_hi;    // warp-uniform
        uint32_t bits = 0u;                               // bit 4u + e: key jb + 128u + 4 lane + e
        uint64_t packed = 0u;
#pragma unroll
        for (int u = 0; u < kPrefetch; ++u) {
            float x[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
            if constexpr (MASKED) {
                const int32_t j = jb + 128 * u + 4 * (int32_t)lane;
                if (j + 3 >= c && j < w_hi)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (j + e >= c && j + e < w_hi) x[e] = end_score[j + e - c];
            }
            uint32_t bu = 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                bool c = x[e] >= Lf;
                if (tail) {
                    const bool in = jb + 128 * u + 4 * (int32_t)lane + e < w_hi;
                    c = c && in;
                    x[e] = in ? x[e] : -INFINITY;        // for the max only
                }
                bu |= (c ? 1u : 0u) << e;
                fmx = fmaxf(fmx, x[e]);
            }
            bits |= bu << (4 * u);
            packed |= (uint64_t)__popc(bu) << (8 * u);
        }
        uint64_t incl = packed;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t nb = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += nb;
        }
        const uint64_t tot = __shfl_sync(0xffffffffu, incl, 31);
        uint32_t base = cnt;
#pragma unroll
        for (int u = 0; u < kPrefetch; ++u) {
            uint32_t at = base + ((uint32_t)((incl - packed) >> (8 * u)) & 0xFFu);
            for (uint32_t bb = (bits >> (4 * u)) & 0xFu; bb; bb &= bb - 1u) {
                const int32_t j = jb + 128 * u + 4 * (int32_t)lane + (int32_t)(__ffs(bb) - 1);
                if (at < (uint32_t)kRegion) rp[at] = j;
                ++at;
            }
            base += (uint32_t)(tot >> (8 * u)) & 0xFFu;
        }
        cnt = base;
    }
    // the candidates' keys, re-read (L1 or L2 hits) once the pass is done:
    // independent loads, many in flight (reading each as it was appended put
    // one round trip per candidate on the pass: 7 K of its ~12 K cycles in a
    // decode row)
    __syncwarp();
    {
        const uint32_t n = min(cnt, (uint32_t)kRegion);
#pragma unroll 4
        for (uint32_t s = lane; s < n; s += 32) rk[s] = row_key(rp[s]);
    }
    // an upper bound of the candidates (keys of the slice, -inf when empty)
    uint32_t cmax = fmx >= Lf ? order_key(fmx) : 0u;
    cmax = __reduce_max_sync(0xffffffffu, cmax);
    if (lane == 0) {
        S.wcnt[warp] = cnt;
        S.wmax[warp] = cmax;
    }
    __syncthreads();
    if (warp == 0) {
        const uint32_t c = lane < kWarps ? S.wcnt[lane] : 0u;
        const uint32_t tot = warp_inclusive_scan(c);
        const bool overflow = __any_sync(0xffffffffu, c > (uint32_t)kRegion);
        const uint32_t mx = __reduce_max_sync(0xffffffffu, lane < kWarps ? S.wmax[lane] : 0u);
        if (lane == 31) {
            S.cta_cand = tot;
            S.cta_overflow = overflow ? 1u : 0u;
            S.cta_max = mx;
        }
    }
    sync_row();
    uint32_t all_cand = 0u, any_overflow = 0u, all_max = 0u;
    if (csize == 1) {
        all_cand = S.cta_cand;
        any_overflow = S.cta_overflow;
        all_max = S.cta_max;
    } else {
        // lane q of warp 0 loads rank q's counts (one remote read per rank,
        // not one per thread), the warp combines them, the CTA shares them
        if (warp == 0) {
            const int q = lane;
            const TopkSmem<NT>* o = cluster.map_shared_rank(&S, (unsigned)min(q, csize - 1));
            uint32_t cc = q < csize ? o->cta_cand : 0u, co = q < csize ? o->cta_overflow : 0u,
                     cm = q < csize ? o->cta_max : 0u;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                cc += __shfl_xor_sync(0xffffffffu, cc, off);
                co |= __shfl_xor_sync(0xffffffffu, co, off);
                cm = max(cm, __shfl_xor_sync(0xffffffffu, cm, off));
            }
            if (lane == 0) {
                S.all_cand = cc;
                S.all_overflow = co;
                S.all_max = cm;
            }
        }
        __syncthreads();
        all_cand = S.all_cand;
        any_overflow = S.all_overflow;
        all_max = S.all_max;
    }
    const bool use_candidates = !any_overflow && all_cand >= (uint32_t)k;

    uint32_t need;
    if (use_candidates) {
        // 3. tau among the cluster's candidates; every candidate lies in
        // [L, all_max], so the bits the two share are known
        const uint32_t tau = radix_select(cluster, csize, S, (uint32_t)k, varying_bits(L, all_max), L, 3,
                                          [&](auto&& f) {
                                              const uint32_t c = S.wcnt[warp];
                                              for (uint32_t s = lane; s < c; s += 32) f(rk[s]);
                                          },
                                          need);
        // 4. ordered output: counts per warp, prefix over warps and lower CTAs
        const uint32_t c = S.wcnt[warp];
        uint32_t g = 0u, e = 0u;
        for (uint32_t s0 = 0; s0 < c; s0 += 32) {
            const uint32_t s = s0 + lane;
            const uint32_t key = s < c ? rk[s] : 0u;
            g += __popc(__ballot_sync(0xffffffffu, s < c && key > tau));
            e += __popc(__ballot_sync(0xffffffffu, s < c && key == tau));
        }
        if (lane == 0) {
            S.wgt[warp] = g;
            S.weq[warp] = e;
        }
        __syncthreads();
        if (warp == 0) {
            const uint32_t gv = lane < kWarps ? S.wgt[lane] : 0u, ev = lane < kWarps ? S.weq[lane] : 0u;
            const uint32_t gi = warp_inclusive_scan(gv);
            const uint32_t ei = warp_inclusive_scan(ev);
            if (lane < kWarps) {
                S.wgt[lane] = gi - gv;
                S.weq[lane] = ei - ev;
            }
            if (lane == 31) {
                S.cta_gt = gi;
                S.cta_eq = ei;
            }
        }
        sync_row();
        uint32_t gt0, eq0;
        cluster_prefix(cluster, crank, S, gt0, eq0);
        uint32_t gt_run = gt0 + S.wgt[warp], eq_run = eq0 + S.weq[warp];
        const uint32_t lower = (1u << lane) - 1u;
        for (uint32_t s0 = 0; s0 < c; s0 += 32) {
            const uint32_t s = s0 + lane;
            const uint32_t key = s < c ? rk[s] : 0u;
            const bool isg = s < c && key > tau, ise = s < c && key == tau;
            const uint32_t bg = __ballot_sync(0xffffffffu, isg), be = __ballot_sync(0xffffffffu, ise);
            const uint32_t gtb = gt_run + __popc(bg & lower), eqb = eq_run + __popc(be & lower);
            if (isg) put(out, gtb + min(eqb, need), k, position(rp[s]), status);
            else if (ise && eqb < need) put(out, gtb + eqb, k, position(rp[s]), status);
            gt_run += __popc(bg);
            eq_run += __popc(be);
        }
    } else {
        // the sample misjudged: select and write over the whole slices
        const int32_t len = s_hi - s_lo;
        auto slice_key = [&](int32_t j) -> uint32_t { return row_key(s_lo + j); };
        const uint32_t tau = radix_select(cluster, csize, S, (uint32_t)k, 32, 0u, 3,
                                          [&](auto&& f) {
                                              for (int32_t j = tid; j < len; j += kThreads) f(slice_key(j));
                                          },
                                          need);
        uint32_t g = 0u, e = 0u;
        for (int32_t j = tid; j < len; j += kThreads) {
            const uint32_t key = slice_key(j);
            g += key > tau;
            e += key == tau;
        }
        const uint32_t gw = warp_inclusive_scan(g), ew = warp_inclusive_scan(e);
        if (lane == 31) {
            S.wgt[warp] = gw;
            S.weq[warp] = ew;
        }
        __syncthreads();
        if (warp == 0) {
            const uint32_t gs = warp_inclusive_scan(lane < kWarps ? S.wgt[lane] : 0u);
            const uint32_t es = warp_inclusive_scan(lane < kWarps ? S.weq[lane] : 0u);
            if (lane == 31) {
                S.cta_gt = gs;
                S.cta_eq = es;
            }
        }
        sync_row();
        uint32_t gt_run, eq_run;
        cluster_prefix(cluster, crank, S, gt_run, eq_run);
        constexpr int kE = 4;
#pragma unroll 1
        for (int32_t base = 0; base < len; base += kThreads * kE) {
            const int32_t j0 = base + tid * kE;
            uint32_t kk[kE];
            uint32_t gc = 0u, ec = 0u;
#pragma unroll
            for (int x = 0; x < kE; ++x) {
                kk[x] = j0 + x < len ? slice_key(j0 + x) : 0u;
                if (j0 + x < len) {
                    gc += kk[x] > tau;
                    ec += kk[x] == tau;
                }
            }
            const uint32_t wi = warp_inclusive_scan(gc | (ec << 16));
            if (lane == 31) S.warp_sums[warp] = wi;
            __syncthreads();
            if (warp == 0) {
                const uint32_t s = warp_inclusive_scan(lane < kWarps ? S.warp_sums[lane] : 0u);
                if (lane < kWarps) S.warp_sums[lane] = s;
                if (lane == kWarps - 1) S.chunk_total = s;
            }
            __syncthreads();
            const uint32_t packed = wi + (warp ? S.warp_sums[warp - 1] : 0u);
            uint32_t gtb = gt_run + (packed & 0xFFFFu) - gc;
            uint32_t eqb = eq_run + (packed >> 16) - ec;
#pragma unroll
            for (int x = 0; x < kE; ++x) {
                if (j0 + x < len) {
                    if (kk[x] > tau) {
                        put(out, gtb + min(eqb, need), k, position(s_lo + j0 + x), status);
                        ++gtb;
                    } else if (kk[x] == tau) {
                        if (eqb < need) put(out, gtb + eqb, k, position(s_lo + j0 + x), status);
                        ++eqb;
                    }
                }
            }
            gt_run += S.chunk_total & 0xFFFFu;
            eq_run += S.chunk_total >> 16;
            __syncthreads();
        }
    }
    if (csize > 1) cluster.sync();                 // the cluster may still read this CTA's counts
}

template <int NT, bool MASKED>
cudaError_t launch_nt(const BatchDev& bd, RowRange rr, const float* scores, int64_t ld, bool scores_local, int k,
                      int32_t* idx, bool idx_local, int csize, int32_t rows_per_seq, int32_t* status,
                      cudaStream_t stream, bool after_previous, const uint64_t* mask) {
    const size_t smem = sizeof(TopkSmem<NT>);
    cudaError_t e = cudaFuncSetAttribute(topk_kernel<NT, MASKED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows_per_seq * csize), (unsigned)bd.B);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)csize;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = after_previous ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, topk_kernel<NT, MASKED>, bd, rr, scores, ld, scores_local ? 1 : 0, k, idx,
                           idx_local ? 1 : 0, csize, status, mask);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

// Masked rows that fit a CTA's shared memory (committed scores, then the visible
// new ones without a gap, -inf behind them): one read of the row, no sampled
// bound, no candidate region.
//   1. min and max as the row arrives (BATCH 16-byte loads in flight per thread).
//   2. One histogram over about 2040 equal intervals of [min, max]: scores of a
//      row spread over it, so few atomics meet and few scores share the k-th's
//      interval.  The interval is read off the low bits of f * per + off, a
//      float in [2^21, 2^22) whose steps are quarters.
//   3. In position order, a segment per warp: scores above a window a little
//      wider than that interval are counted, those in it gathered and ranked.
//      Whatever the rounding, the counts prove the k-th to be in the window; if
//      they do not, or it holds more than 64 (ties, outliers that stretch the
//      range, infinities): radix_select over all scores and a count.
//   4. The selected indices, in order from packed warp scans, into shared
//      memory, and from there to idx; ties at the k-th are told apart only if
//      not all of them are taken.
// CLUSTER: the CTAs of a cluster take a slice of the row each and exchange the
// range, the sums of the intervals, the window's scores and the counts.
// Limited by instructions (34 per 32 scores and 4.5 K a row of 256 threads) and
// by the barriers between the passes (a scheduler issues in 59-67 % of the
// cycles).  Scores that an even division does not fit take the fallback of
// step 3, about three times as long: with one score of 50 standard deviations in a
// row, or many equal ones, 8 x 8 over 32,768 27-29 us (9.7), 64 full trees of 32
// over 9,001 125 (38), 1 x 8 over 32,768 19-20 (8.0); from about 20 standard
// deviations some rows do.  k = 2048, 64 trees of up to 32 rows
// over up to 9,001 positions: 17-19 us (topk_kernel 72, the row in registers
// instead of shared memory 23-29); 64 x 32 over 2,500: 17 us; 8 x 8 over
// 32,768: 9.6 us (CTA pairs); 1 x 8: 8.0 us (fours).
template <int NT, int BATCH, int MINB, bool CLUSTER>
__global__ void __launch_bounds__(NT, MINB)
    topk_short_kernel(const BatchDev bd, const float* __restrict__ scores, const int64_t ld, const int k,
                      int32_t* __restrict__ idx, int32_t* status, const uint64_t* __restrict__ mask) {
    constexpr int kWarps = NT / 32, kBinsPerThread = kBins / NT, kBlock = 4;   // 128-score groups per scan
    constexpr int kBinGroups = kWarps, kBinsPerGroup = kBins / kWarps;
    static_assert(kMaxTopk <= kBins, "the selected indices take the histogram's place");
    static_assert(kShortRow <= 32 * 128 * 32 && kRowOf512 <= 16 * 128 * 32 && kRowOf256 <= 8 * 128 * 32,
                  "a warp's segment has at most 32 groups");
    static_assert(kWarps <= 32 && NT >= DSA_MAX_TREE * 2, "one lane per warp's sum; new scores and padding by one thread each");
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ TopkSmem<NT, 1> S;
    __shared__ int32_t end_pos[DSA_MAX_TREE];
    __shared__ uint32_t list[CLUSTER ? 64 : 1], owner[CLUSTER ? 64 : 1];
    float* row_s = reinterpret_cast<float*>(smem_raw);
    float4* row4 = reinterpret_cast<float4*>(smem_raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int csize = CLUSTER ? (int)cluster.num_blocks() : 1, crank = CLUSTER ? (int)(blockIdx.x % (unsigned)csize) : 0;
    const int b = blockIdx.y, i = blockIdx.x / (unsigned)csize;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();                  // the scores of the previous launch are complete
    SeqInfo sq;
    if (!load_seq(bd, b, status, sq) || i >= sq.nq) return;
    const float* row = scores + ((int64_t)sq.q0 + i) * ld;
    int32_t* out = idx + ((int64_t)sq.q0 + i) * k;
    const int32_t c = sq.ctx - sq.nq;
    // this CTA's slice of the row: positions [s_lo, s_lo + span), the first `cl`
    // of them committed
    const int32_t span = CLUSTER ? ((sq.ctx + csize - 1) / csize + 127) & ~127 : sq.ctx;
    const int32_t s_lo = CLUSTER ? crank * span : 0;
    const int32_t cl = CLUSTER ? min(max(c - s_lo, 0), span) : c, old4 = (cl + 3) >> 2;
    row += s_lo;
    const unsigned long long word = __ldg(reinterpret_cast<const unsigned long long*>(mask) + sq.q0 + i);
    auto load = [&](int32_t g) -> float4 {
        return sq.ctx > k && g < old4 ? __ldg(reinterpret_cast<const float4*>(row) + g) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    float4 v[BATCH];
#pragma unroll
    for (int u = 0; u < BATCH; ++u) v[u] = load(NT * u + tid);
    const uint64_t bits = visible_bits(word, i);
    const int32_t n = c + __popcll(bits);
    // the new position of a visible bit, its place in the row, and its score
    const bool seen = tid < DSA_MAX_TREE && (bits >> (tid & 63)) & 1u;
    const int32_t place = c + __popcll(bits & ((1ull << (tid & 63)) - 1u));
    if (n <= k) {
        if (crank != 0) return;
        for (int j = tid; j < k; j += NT)
            if (j < c || j >= n) out[j] = j < c ? j : -1;
        if (seen) out[place] = c + tid;
        return;
    }
    float low = INFINITY, high = -INFINITY;
    if (seen) {
        end_pos[place - c] = c + tid;
        if (!CLUSTER || (place >= s_lo && place < s_lo + span)) {
            low = high = __ldg(row - s_lo + c + tid);
            row_s[place - s_lo] = low;
        }
    }
    const int32_t len = CLUSTER ? min(max(n - s_lo, 0), span) : n;   // the slice's scores
    if (len + tid < ((len + 127) & ~127)) row_s[len + tid] = -INFINITY;
#pragma unroll
    for (int x = 0; x < kBinsPerThread; ++x) S.hist[NT * x + tid] = 0u;
    if (tid < 32) S.weq[tid] = 0u;
    if (tid == 0) {
        S.small_n = 0u;
        S.sel_count = 0xFFFFFFFFu;
        S.pre_gt = 0u;
        S.pre_eq = 0u;
    }
    for (int32_t g0 = 0;;) {
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int32_t g = g0 + NT * u + tid;
            if (4 * g + 4 <= cl) {
                row4[g] = v[u];
                low = fminf(fminf(low, fminf(v[u].x, v[u].y)), fminf(v[u].z, v[u].w));
                high = fmaxf(fmaxf(high, fmaxf(v[u].x, v[u].y)), fmaxf(v[u].z, v[u].w));
            } else if (4 * g < cl) {                  // the group that the new scores follow in
                const float y[3] = {v[u].x, v[u].y, v[u].z};
                for (int x = 0; x < 3 && 4 * g + x < cl; ++x) {
                    row_s[4 * g + x] = y[x];
                    low = fminf(low, y[x]);
                    high = fmaxf(high, y[x]);
                }
            }
        }
        g0 += NT * BATCH;
        if (g0 >= old4) break;
#pragma unroll
        for (int u = 0; u < BATCH; ++u) v[u] = load(g0 + NT * u + tid);
    }
    low = -warp_max_f32(-low);
    high = warp_max_f32(high);
    if (lane == 0) {
        S.wgt[warp] = __float_as_uint(low);
        S.wmax[warp] = __float_as_uint(high);
    }
    __syncthreads();
    low = -warp_max_f32(lane < kWarps ? -__uint_as_float(S.wgt[lane]) : -INFINITY);
    high = warp_max_f32(lane < kWarps ? __uint_as_float(S.wmax[lane]) : -INFINITY);
    if constexpr (CLUSTER) {
        if (tid == 0) {
            S.cta_cand = __float_as_uint(low);
            S.cta_max = __float_as_uint(high);
        }
        cluster.sync();
        const auto* o = cluster.map_shared_rank(&S, (unsigned)min(lane, csize - 1));
        low = -warp_max_f32(-__uint_as_float(o->cta_cand));
        high = warp_max_f32(__uint_as_float(o->cta_max));
    }

    // interval of f: t = 4 + (f - low) * per, rounded to quarters, its floor;
    // four spare ones at each end for the rounding of `off`
    const float range = high - low, per = ((float)kBins - 8.f) / range, off = fmaf(-low, per, 2097152.f + 4.f);
    const bool linear = range > 0.f && range < INFINITY && per < INFINITY;   // false for NaN too
    const int32_t seg = ((len + kWarps - 1) / kWarps + 127) & ~127;
    const int32_t w_lo = min(len, warp * seg), w_hi = min(len, w_lo + seg);
    float tf = 0.f;
    uint32_t need = 0u, gt_pre = 0u;                  // gt_pre: in the lower ranks' slices
    bool ties = true, ranked = false;
    if (linear) {
#pragma unroll 2
        for (int32_t g = tid; 4 * g < len; g += NT) {
            const float4 x = row4[g];                 // at most 3 of -inf here: they add to interval 0
            const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
                atomicAdd(&S.hist[(__float_as_uint(fmaf(y[q], per, off)) >> 2) & (uint32_t)(kBins - 1)], 1u);
        }
        __syncthreads();
        uint32_t cnt[kBinsPerThread], mine = 0u;
#pragma unroll
        for (int q = 0; q < kBinsPerThread; q += 2) {
            const uint2 two = *reinterpret_cast<const uint2*>(&S.hist[kBinsPerThread * tid + q]);
            cnt[q] = two.x;
            cnt[q + 1] = two.y;
            mine += two.x + two.y;
        }
        if constexpr (CLUSTER) {
            // the warp's bins that hold the k-th from every rank's sums of a
            // warp's bins, then its bin from every rank's bins of that warp
            mine = __reduce_add_sync(0xffffffffu, mine);
            if (lane == 0) S.group[warp] = mine;
            cluster.sync();
            if (warp == 0) {
                uint32_t sum = 0u;
#pragma unroll
                for (int q = 0; q < kMaxCluster; ++q)
                    if (q < csize && lane < kBinGroups) sum += cluster.map_shared_rank(S.group, (unsigned)q)[lane];
                uint32_t incl = warp_inclusive_scan(sum);
                uint32_t above = __shfl_sync(0xffffffffu, incl, 31) - incl;
                const uint32_t has = __ballot_sync(0xffffffffu, above < (uint32_t)k && (uint32_t)k <= above + sum);
                const int grp = has ? __ffs(has) - 1 : 0;
                const uint32_t gabove = __shfl_sync(0xffffffffu, above, grp);
                uint32_t bin[kBinsPerGroup / 32];
#pragma unroll
                for (int x = 0; x < kBinsPerGroup / 32; ++x) bin[x] = 0u;
#pragma unroll
                for (int q = 0; q < kMaxCluster; ++q)
                    if (q < csize) {
                        const uint32_t* from = cluster.map_shared_rank(S.hist, (unsigned)q) + kBinsPerGroup * grp;
#pragma unroll
                        for (int x = 0; x < kBinsPerGroup / 32; ++x) bin[x] += from[kBinsPerGroup / 32 * lane + x];
                    }
                sum = 0u;
#pragma unroll
                for (int x = 0; x < kBinsPerGroup / 32; ++x) sum += bin[x];
                incl = warp_inclusive_scan(sum);
                above = gabove + __shfl_sync(0xffffffffu, incl, 31) - incl;
#pragma unroll
                for (int x = kBinsPerGroup / 32 - 1; x >= 0; --x) {
                    if (has && above < (uint32_t)k && (uint32_t)k <= above + bin[x]) {
                        S.sel_digit = (uint32_t)(kBinsPerGroup * grp + kBinsPerGroup / 32 * lane + x);
                        S.sel_count = bin[x];
                    }
                    above += bin[x];
                }
            }
            __syncthreads();
        } else {
            const uint32_t incl = warp_inclusive_scan(mine);
            if (lane == 31) S.warp_sums[warp] = incl;
            __syncthreads();
            const uint32_t sums = lane < kWarps ? S.warp_sums[lane] : 0u;
            // scores in higher intervals
            uint32_t above = mine - incl + __reduce_add_sync(0xffffffffu, lane >= warp ? sums : 0u) - mine;
            if (above < (uint32_t)k && (uint32_t)k <= above + mine) {
    #pragma unroll
                for (int q = kBinsPerThread - 1; q >= 0; --q) {
                    if (above < (uint32_t)k && (uint32_t)k <= above + cnt[q]) {
                        S.sel_digit = (uint32_t)(kBinsPerThread * tid + q);
                        S.sel_count = cnt[q];
                    }
                    above += cnt[q];
                }
            }
            __syncthreads();
        }
        if (S.sel_count <= 64u) {
            const float at = (float)S.sel_digit, width = range / ((float)kBins - 8.f);
            const float from = fmaf(at - 4.375f, width, low), to = fmaf(at - 2.875f, width, low);
            // subtraction is monotone: a score in the window is within `half` of mid
            const float mid = 0.5f * from + 0.5f * to, half = fmaxf(to - mid, mid - from);
            uint32_t higher = 0u, hits = 0u;          // hits: the lane's groups with a score in the window
#pragma unroll 2
            for (int32_t j = w_lo, u = 0; j < w_hi; j += 128, ++u) {
                const float4 x = row4[(j >> 2) + lane];
                const float y[4] = {x.x, x.y, x.z, x.w};
                float d = INFINITY;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    higher += y[q] > to ? 1u : 0u;
                    d = fminf(d, fabsf(y[q] - mid));
                }
                hits |= (d <= half ? 1u : 0u) << u;
            }
            for (; hits; hits &= hits - 1u) {
                const float4 x = row4[(w_lo >> 2) + 32 * (__ffs(hits) - 1) + lane];
                const float y[4] = {x.x, x.y, x.z, x.w};
                uint32_t in = 0u;
#pragma unroll
                for (int q = 0; q < 4; ++q) in += y[q] >= from && y[q] <= to ? 1u : 0u;
                uint32_t s = atomicAdd(&S.small_n, in);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (y[q] >= from && y[q] <= to && s < 64u) {
                        S.small[s] = __float_as_uint(y[q]);
                        S.small_all[s++] = (uint32_t)warp;
                    }
            }
            higher = __reduce_add_sync(0xffffffffu, higher);
            if (lane == 0) S.wcnt[warp] = higher;
            __syncthreads();
            uint32_t m = S.small_n, all_higher = __reduce_add_sync(0xffffffffu, lane < kWarps ? S.wcnt[lane] : 0u);
            if constexpr (CLUSTER) {
                // every rank's list behind the lower ranks', with its owner
                if (tid == 0) S.cta_gt = all_higher;
                cluster.sync();
                const auto* o = cluster.map_shared_rank(&S, (unsigned)min(lane, csize - 1));
                const uint32_t n_of = lane < csize ? o->small_n : 0u, higher_of = lane < csize ? o->cta_gt : 0u;
                const uint32_t behind = warp_inclusive_scan(n_of);
                m = __shfl_sync(0xffffffffu, behind, 31);
                all_higher = __reduce_add_sync(0xffffffffu, higher_of);
                gt_pre = __reduce_add_sync(0xffffffffu, lane < crank ? higher_of : 0u);
                for (int q = warp; q < csize; q += kWarps) {
                    const uint32_t from_q = __shfl_sync(0xffffffffu, behind - n_of, q), n_q = __shfl_sync(0xffffffffu, n_of, q);
                    const auto* of = cluster.map_shared_rank(&S, (unsigned)q);
                    for (uint32_t x = lane; m <= 64u && x < n_q; x += 32u) {
                        list[from_q + x] = of->small[x];
                        owner[from_q + x] = of->small_all[x] + ((uint32_t)q << 8);
                    }
                }
                __syncthreads();
            }
            const uint32_t want = (uint32_t)k - all_higher;
            const uint32_t* values = CLUSTER ? list : S.small;
            ranked = m <= 64u && want - 1u < m;       // 0 < want <= m
            if (ranked) {
                // eight threads rank a score against eight each
                for (uint32_t ranker = (uint32_t)tid; ranker < 8u * m; ranker += NT) {
                    const uint32_t q = ranker >> 3, sub = ranker & 7u;
                    const float f = __uint_as_float(values[q]);
                    uint32_t gt = 0u, eq = 0u;
                    for (uint32_t o = sub; o < m; o += 8u) {
                        const float y = __uint_as_float(values[o]);
                        gt += y > f ? 1u : 0u;
                        eq += y == f ? 1u : 0u;
                    }
                    const uint32_t group = 0xFFu << (lane & 24);
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) {
                        gt += __shfl_xor_sync(group, gt, o);
                        eq += __shfl_xor_sync(group, eq, o);
                    }
                    if (sub == 0 && gt < want && want <= gt + eq) {
                        // equal scores (both zeros) write the same values but this one
                        S.small_tau = __float_as_uint(f);
                        S.small_need = want - gt;
                        S.total = eq;
                    }
                }
                __syncthreads();
                tf = __uint_as_float(S.small_tau);
                need = S.small_need;
                ties = S.total != need;
                if ((uint32_t)tid < m) {
                    const float f = __uint_as_float(values[tid]);
                    const uint32_t of = CLUSTER ? owner[tid] : S.small_all[tid];
                    const int rank = (int)(of >> 8);
                    const bool above = f > tf || (!ties && f == tf);
                    if (above || f == tf) {
                        if (rank == crank) atomicAdd(above ? &S.wcnt[of & 0xFFu] : &S.weq[of & 0xFFu], 1u);
                        else if (rank < crank) atomicAdd(above ? &S.pre_gt : &S.pre_eq, 1u);
                    }
                }
            }
        }
    }
    uint32_t tau = 0u;
    if (!ranked) {
        if constexpr (CLUSTER) cluster.sync();        // other ranks may still read this one's counts
        else __syncthreads();
#pragma unroll
        for (int x = 0; x < kBinsPerThread; ++x) S.hist[NT * x + tid] = 0u;
        uint32_t kmin = 0xFFFFFFFFu, kmax = 0u;
#pragma unroll 1
        for (int32_t j = tid; j < len; j += NT) {
            const uint32_t q = order_key(row_s[j]);
            kmin = min(kmin, q);
            kmax = max(kmax, q);
        }
        kmin = __reduce_min_sync(0xffffffffu, kmin);
        kmax = __reduce_max_sync(0xffffffffu, kmax);
        if (lane == 0) {
            S.wgt[warp] = kmin;
            S.wmax[warp] = kmax;
        }
        __syncthreads();
        kmin = __reduce_min_sync(0xffffffffu, lane < kWarps ? S.wgt[lane] : 0xFFFFFFFFu);
        kmax = __reduce_max_sync(0xffffffffu, lane < kWarps ? S.wmax[lane] : 0u);
        if constexpr (CLUSTER) {
            if (tid == 0) {
                S.cta_overflow = kmin;
                S.all_max = kmax;
            }
            cluster.sync();
            const auto* o = cluster.map_shared_rank(&S, (unsigned)min(lane, csize - 1));
            kmin = __reduce_min_sync(0xffffffffu, o->cta_overflow);
            kmax = __reduce_max_sync(0xffffffffu, o->all_max);
        }
        tau = radix_select(cluster, csize, S, (uint32_t)k, varying_bits(kmin, kmax), kmin, 3,
                           [&](auto&& f) {
#pragma unroll 1
                               for (int32_t j = tid; j < len; j += NT) f(order_key(row_s[j]));
                           },
                           need);
        uint32_t gt = 0u, eq = 0u;
#pragma unroll 1
        for (int32_t j = w_lo + lane; j < w_hi; j += 32) {
            const uint32_t q = order_key(row_s[j]);
            gt += q > tau ? 1u : 0u;
            eq += q == tau ? 1u : 0u;
        }
        gt = __reduce_add_sync(0xffffffffu, gt);
        eq = __reduce_add_sync(0xffffffffu, eq);
        if (lane == 0) {
            S.wcnt[warp] = gt;
            S.weq[warp] = eq;
        }
        if constexpr (CLUSTER) {
            __syncthreads();
            gt = __reduce_add_sync(0xffffffffu, lane < kWarps ? S.wcnt[lane] : 0u);
            eq = __reduce_add_sync(0xffffffffu, lane < kWarps ? S.weq[lane] : 0u);
            if (tid == 0) {
                S.cta_gt = gt;
                S.cta_eq = eq;
            }
            cluster.sync();
            const auto* o = cluster.map_shared_rank(&S, (unsigned)min(lane, csize - 1));
            gt = __reduce_add_sync(0xffffffffu, lane < crank ? o->cta_gt : 0u);
            eq = __reduce_add_sync(0xffffffffu, lane < crank ? o->cta_eq : 0u);
            if (tid == 0) {
                S.pre_gt = gt;
                S.pre_eq = eq;
            }
            gt_pre = 0u;
        }
    }
    if constexpr (CLUSTER) cluster.sync();            // the last remote read is done
    else __syncthreads();
    // the histogram's place takes the selected indices from here on
    uint32_t* sel = S.hist;
    const uint32_t sg = lane < kWarps ? S.wcnt[lane] : 0u, se = ties && lane < kWarps ? S.weq[lane] : 0u;
    uint32_t g0 = __reduce_add_sync(0xffffffffu, lane < warp ? sg : 0u);
    uint32_t e0 = __reduce_add_sync(0xffffffffu, lane < warp ? se : 0u);
    // taken in this slice, and where they go: scores above the k-th, and of the
    // equal ones the first `need` of the row
    const uint32_t e_pre = CLUSTER ? min(S.pre_eq, need) : 0u, first = CLUSTER ? gt_pre + S.pre_gt + e_pre : 0u;
    const uint32_t left = need - e_pre;
    const uint32_t taken = __reduce_add_sync(0xffffffffu, sg) + min(__reduce_add_sync(0xffffffffu, se), left);
    if (first + taken > (uint32_t)k || (!CLUSTER && taken != (uint32_t)k)) {   // would be a bug: no write past k
        latch_status(status, DSA_ERR_INTERNAL);
        return;
    }
    if (!ties) {
        for (int32_t j0 = w_lo; j0 < w_hi; j0 += 128 * kBlock) {
            // a byte per group for the warp's scan
            float4 x[kBlock];
            uint32_t own = 0u;
#pragma unroll
            for (int u = 0; u < kBlock; ++u) {
                if (j0 + 128 * u >= w_hi) break;
                x[u] = row4[(j0 >> 2) + 32 * u + lane];
                own += ((x[u].x >= tf ? 1u : 0u) + (x[u].y >= tf ? 1u : 0u) + (x[u].z >= tf ? 1u : 0u) +
                        (x[u].w >= tf ? 1u : 0u)) << (8 * u);
            }
            const uint32_t incl = warp_inclusive_scan(own), all = __shfl_sync(0xffffffffu, incl, 31);
            const uint32_t excl = incl - own;
#pragma unroll
            for (int u = 0; u < kBlock; ++u) {
                if (j0 + 128 * u >= w_hi) break;
                uint32_t* to = sel + g0 + ((excl >> (8 * u)) & 0xFFu);
                const uint32_t j = (uint32_t)(j0 + 128 * u + 4 * lane);
                if (x[u].x >= tf) *to++ = j;
                if (x[u].y >= tf) *to++ = j + 1u;
                if (x[u].z >= tf) *to++ = j + 2u;
                if (x[u].w >= tf) *to++ = j + 3u;
                g0 += (all >> (8 * u)) & 0xFFu;
            }
        }
    } else {
        const uint32_t lower = (1u << lane) - 1u;
#pragma unroll 1
        for (int32_t j0 = w_lo; j0 < w_hi; j0 += 32) {
            const int32_t j = j0 + lane;
            const float x = row_s[j];                 // at most 31 past w_hi, inside the padded row
            const uint32_t key = order_key(x);
            const bool gt = j < w_hi && (ranked ? x > tf : key > tau), eq = j < w_hi && (ranked ? x == tf : key == tau);
            const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
            const uint32_t g = g0 + __popc(bg & lower), e = e0 + __popc(be & lower);
            if (gt) sel[g + min(e, left)] = (uint32_t)j;
            else if (eq && e < left) sel[g + e] = (uint32_t)j;
            g0 += __popc(bg);
            e0 += __popc(be);
        }
    }
    __syncthreads();
    // late: a dependent's CTAs that come earlier take shared memory from rows
    // that wait for it (256 rows over 8,192 in a loop: 9.5 us instead of 7.9)
    pdl_launch_dependents();
    auto position = [&](uint32_t at) -> int32_t {
        const int32_t j = s_lo + (int32_t)at;
        return j < c ? j : end_pos[j - c];
    };
    if (!CLUSTER && k % 4 == 0) {
        for (int32_t g = tid; 4 * g < k; g += NT) {
            const uint4 w = reinterpret_cast<const uint4*>(sel)[g];
            reinterpret_cast<int4*>(out)[g] = make_int4(position(w.x), position(w.y), position(w.z), position(w.w));
        }
    } else {
        for (uint32_t g = tid; g < taken; g += NT) out[first + g] = position(sel[g]);
    }
}

template <int NT, int BATCH, int MINB, bool CLUSTER = false>
cudaError_t launch_short(const BatchDev& bd, const float* scores, int64_t ld, const uint64_t* mask, int k, int32_t* idx,
                         int32_t* status, cudaStream_t stream, int csize = 1) {
    const size_t smem = (((size_t)bd.max_ctx + csize - 1) / csize + 127) / 128 * 128 * sizeof(float);
    // the same limit in every call: another thread's may come between this and the launch
    cudaError_t e = cudaFuncSetAttribute(topk_short_kernel<NT, BATCH, MINB, CLUSTER>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kShortRow * (int)sizeof(float));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(bd.max_q * csize), (unsigned)bd.B);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)csize;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CLUSTER ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, topk_short_kernel<NT, BATCH, MINB, CLUSTER>, bd, scores, ld, k, idx, status, mask);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

template <bool MASKED>
cudaError_t launch_rows(const BatchDev& bd, RowRange rr, const float* scores, int64_t ld, bool scores_local, int k,
                        int32_t* idx, bool idx_local, int32_t* status, cudaStream_t stream, bool after_previous,
                        const uint64_t* mask) {
    const int32_t rows_per_seq = min(rr.i1, bd.max_q) - rr.i0;
    if (rows_per_seq <= 0) return cudaSuccess;
    // long rows, few of them: split each row over a cluster
    const int64_t rows = (int64_t)rows_per_seq * bd.B;
    int csize = 1;
    if (bd.max_ctx > kLongRow && rows < 2 * num_sms())
        csize = (int)std::min<int64_t>(kMaxCluster, ((int64_t)bd.max_ctx + kKeysPerCta - 1) / kKeysPerCta);
    return rows < num_sms() ? launch_nt<1024, MASKED>(bd, rr, scores, ld, scores_local, k, idx, idx_local, csize,
                                                      rows_per_seq, status, stream, after_previous, mask)
                            : launch_nt<512, MASKED>(bd, rr, scores, ld, scores_local, k, idx, idx_local, csize,
                                                     rows_per_seq, status, stream, after_previous, mask);
}

}  // namespace

cudaError_t launch_topk(const BatchDev& bd, RowRange rr, const float* scores, int64_t ld, bool scores_local,
                        int k, int32_t* idx, bool idx_local, int32_t* status, cudaStream_t stream,
                        bool after_previous) {
    return launch_rows<false>(bd, rr, scores, ld, scores_local, k, idx, idx_local, status, stream, after_previous,
                              nullptr);
}

cudaError_t launch_tree_topk(const BatchDev& bd, const float* scores, int64_t ld, const uint64_t* mask, int k,
                             int32_t* idx, int32_t* status, cudaStream_t stream) {
    // Rows that fit a CTA's shared memory.  Fewer rows than SMs: a CTA has an SM
    // to itself and takes as many threads as its row feeds (8,192 positions: 5.7
    // us with 512, 6.3 with 1024; 32,768: 11.8 and 10.9).  Else a smaller CTA
    // pays for fewer warps' sums, as long as an SM's shared memory holds rows
    // for enough of them (64 x 32 rows over 9,001: 41 us with 256 threads, 44
    // with 512, 80 with 1024; 16 x 64 over 20,000: 51, 43, 54; over 32,768:
    // 112, 91, 79).
    // With fewer than two rows per SM the smaller CTA gains nothing (256 rows over
    // 8,192: 8.7 us with 256 threads, 7.9 with 512).
    const int64_t rows = (int64_t)bd.B * bd.max_q;
    const bool few = rows < num_sms();
    // Long rows and SMs to spare: a cluster shares a row (8 rows over 32,768: 9.8
    // us with one CTA, 9.5, 8.0 and 8.5 with two, four and eight; over 100,000:
    // 18 (topk_kernel) and 10.4 with eight; 16 rows over 16,384: 7.0, and 7.4 with four).
    int csize = 1;
    while (bd.max_ctx > kAloneRow && csize < kMaxCluster && rows * 2 * csize <= num_sms() && bd.max_ctx > kSlice * csize)
        csize *= 2;
    // Rows that one CTA does not hold take as many as do, unless topk_kernel splits
    // them itself and there are two of them per SM or nearly (512 rows over 131,000:
    // 222 us, topk_kernel 904; 256 over 70,000: 55 and 71; 256 over 100,000: 105
    // and 89).
    int fit = 1;
    while (fit < kMaxCluster && bd.max_ctx > (int64_t)kShortRow * fit) fit *= 2;
    if (fit <= 2 || rows < num_sms() || rows >= 2 * num_sms()) csize = std::max(csize, fit);
    if (csize > 1 && bd.max_ctx <= (int64_t)kShortRow * csize)
        return launch_short<512, 4, 1, true>(bd, scores, ld, mask, k, idx, status, stream, csize);
    if (bd.max_ctx <= kShortRow) {
        if (rows >= 2 * num_sms() && bd.max_ctx <= kRowOf256)
            return launch_short<256, 4, 5>(bd, scores, ld, mask, k, idx, status, stream);
        return bd.max_ctx <= (few ? kFewRowOf512 : kRowOf512)
                   ? launch_short<512, 4, 3>(bd, scores, ld, mask, k, idx, status, stream)
                   : launch_short<1024, 8, 1>(bd, scores, ld, mask, k, idx, status, stream);
    }
    return launch_rows<true>(bd, RowRange{0, bd.max_q}, scores, ld, false, k, idx, false, status, stream, false, mask);
}

}  // namespace dsa
