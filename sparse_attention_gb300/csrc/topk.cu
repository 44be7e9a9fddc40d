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
    uint32_t sample[kSample];
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
            if (tid < 512) {
                const uint32_t nb = S.small_all_n;
                const uint32_t q = (uint32_t)tid >> 3, sub = (uint32_t)tid & 7u;
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

// Masked rows of up to NT * KPT positions: the whole row stays in registers
// (warp w owns a contiguous segment, read as coalesced 16-byte groups while
// the mask and the row's end are on their way), so there is no sampled bound,
// no candidate region and no second read.
//   1. One histogram over 2048 equal intervals of [min, max]: scores of a row
//      spread over it, so few atomics meet and few keys stay.  Subtraction, product and truncation are monotone, so the
//      interval of the k-th largest is exact whatever the rounding.
//   2. At most 64 keys in it: gathered and ranked.  More (ties, outliers that
//      stretch the range, infinities): radix_select over all keys.
//   3. Output in position order from packed warp scans; ties at tau are
//      counted only if not all of them are taken.
// Bound by instructions.  64 trees of up to 32 rows over up to 9,001
// positions, k = 2048: 29-35 us (topk_kernel 72); 8 trees of 8 over 32,768:
// 12-14 us (21.7).
template <int NT, int KPT>
__global__ void __launch_bounds__(NT, NT == 1024 ? 1 : KPT <= 8 ? 3 : 2)
    topk_short_kernel(const BatchDev bd, const float* __restrict__ scores, const int64_t ld, const int k,
                      int32_t* __restrict__ idx, int32_t* status, const uint64_t* __restrict__ mask) {
    constexpr int kWarps = NT / 32, kGroups = KPT / 4, kBinsPerThread = kBins / NT;
    static_assert(kGroups <= 8, "a lane's counts fill one 64-bit word");
    __shared__ TopkSmem<NT, 1> S;
    __shared__ float end_score[DSA_MAX_TREE];
    __shared__ int32_t end_pos[DSA_MAX_TREE];
    cg::cluster_group cluster = cg::this_cluster();
    const int b = blockIdx.y, i = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    SeqInfo sq;
    if (!load_seq(bd, b, status, sq) || i >= sq.nq) return;
    const float* row = scores + ((int64_t)sq.q0 + i) * ld;
    int32_t* out = idx + ((int64_t)sq.q0 + i) * k;
    const int32_t c = sq.ctx - sq.nq;
    const int32_t seg = ((sq.ctx + kWarps - 1) / kWarps + 127) & ~127;
    const int32_t w_lo = min(sq.ctx, warp * seg), w_end = min(sq.ctx, w_lo + seg);
    float4 v[kGroups];
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
        const int32_t j = w_lo + 128 * u + 4 * lane;
        v[u] = sq.ctx > k && j < w_end ? __ldg(reinterpret_cast<const float4*>(row + j))
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int32_t n = masked_end(sq, i, row, mask, end_score, end_pos);
#pragma unroll
    for (int x = 0; x < kBinsPerThread; ++x) S.hist[NT * x + tid] = 0u;
    if (tid == 0) {
        S.small_n = 0u;
        S.sel_count = 0xFFFFFFFFu;
    }
    __syncthreads();
    auto position = [&](int32_t j) -> int32_t { return j < c ? j : end_pos[j - c]; };
    if (n <= k) {
        for (int j = tid; j < k; j += NT) out[j] = j < n ? position(j) : -1;
        return;
    }
    const int32_t w_hi = min(n, w_end);
    // The lane's scores; NaN behind the row's end, which is above, below and
    // equal to nothing.  Groups past the segment's length are skipped
    // everywhere (the same branch for the whole CTA), and groups that lie
    // before the packed end take no test per score (the same for a warp): the
    // kernel is bound by its instructions.
    const int32_t plain = min(c, w_hi) - w_lo;   // this warp's scores before the packed end
    float x[KPT], low = INFINITY, high = -INFINITY;
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
        if (128 * u >= seg) break;
        float y[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        if (128 * u + 128 > plain) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int32_t j = w_lo + 128 * u + 4 * lane + e;
                y[e] = j < w_hi ? (j < c ? y[e] : end_score[j - c]) : NAN;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[4 * u + e] = y[e];
            low = fminf(low, y[e]);
            high = fmaxf(high, y[e]);
        }
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

    // a little less than kBins intervals, so that `high` falls into the last
    const float span = high - low, scale = ((float)kBins - 0.125f) / span;
    const bool linear = span > 0.f && span < INFINITY && scale < INFINITY;   // false for NaN too
    float tf = 0.f;
    uint32_t tau = 0u, need = 0u;
    bool ties = true, ranked = false;
    auto bin = [&](float f) -> uint32_t { return (uint32_t)(int)((f - low) * scale); };
    if (linear) {
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
            if (128 * u >= seg) break;
            const bool all = 128 * u + 128 <= plain;
#pragma unroll
            for (int q = 4 * u; q < 4 * u + 4; ++q)
                if (all || x[q] == x[q]) atomicAdd(&S.hist[min(bin(x[q]), (uint32_t)kBins - 1u)], 1u);
        }
        __syncthreads();
        uint32_t cnt[kBinsPerThread], mine = 0u;
#pragma unroll
        for (int q = 0; q < kBinsPerThread; ++q) {
            cnt[q] = S.hist[kBinsPerThread * tid + q];
            S.hist[kBinsPerThread * tid + q] = 0u;
            mine += cnt[q];
        }
        const uint32_t incl = warp_inclusive_scan(mine);
        if (lane == 31) S.warp_sums[warp] = incl;
        __syncthreads();
        const uint32_t sums = warp_inclusive_scan(lane < kWarps ? S.warp_sums[lane] : 0u);
        const uint32_t before = __shfl_sync(0xffffffffu, sums, (warp + 31) & 31);
        // keys in higher bins
        uint32_t above = __shfl_sync(0xffffffffu, sums, 31) - (incl + (warp ? before : 0u));
#pragma unroll
        for (int q = kBinsPerThread - 1; q >= 0; --q) {
            if (above < (uint32_t)k && (uint32_t)k <= above + cnt[q]) {
                S.sel_digit = (uint32_t)(kBinsPerThread * tid + q);
                S.sel_above = above;
                S.sel_count = cnt[q];
            }
            above += cnt[q];
        }
        __syncthreads();
        if (S.sel_count <= 64u) {
            const uint32_t digit = S.sel_digit;
#pragma unroll
            for (int u = 0; u < kGroups; ++u) {
                if (128 * u >= seg) break;
#pragma unroll
                for (int q = 4 * u; q < 4 * u + 4; ++q)
                    if (x[q] == x[q] && bin(x[q]) == digit)
                        S.small[atomicAdd(&S.small_n, 1u) & 63u] = __float_as_uint(x[q]);
            }
            __syncthreads();
            // eight threads rank a score against eight each
            const uint32_t m = min(S.small_n, 64u), want = (uint32_t)k - S.sel_above;
            if (tid < 512) {
                const uint32_t q = (uint32_t)tid >> 3, sub = (uint32_t)tid & 7u;
                const float f = q < m ? __uint_as_float(S.small[q]) : NAN;
                uint32_t gt = 0u, eq = 0u;
#pragma unroll
                for (uint32_t o = 0; o < 8u; ++o) {
                    const float y = sub * 8u + o < m ? __uint_as_float(S.small[sub * 8u + o]) : NAN;
                    gt += y > f ? 1u : 0u;
                    eq += y == f ? 1u : 0u;
                }
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) {
                    gt += __shfl_xor_sync(0xffffffffu, gt, o);
                    eq += __shfl_xor_sync(0xffffffffu, eq, o);
                }
                if (sub == 0 && q < m && gt < want && want <= gt + eq) {
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
            ranked = true;
        }
    }
    if (!ranked) {
        uint32_t kmin = 0xFFFFFFFFu, kmax = 0u;
#pragma unroll 1
        for (int32_t j = w_lo + lane; j < w_hi; j += 32) {
            const uint32_t q = order_key(j < c ? __ldg(row + j) : end_score[j - c]);
            kmin = min(kmin, q);
            kmax = max(kmax, q);
        }
        kmin = __reduce_min_sync(0xffffffffu, kmin);
        kmax = __reduce_max_sync(0xffffffffu, kmax);
        __syncthreads();
        if (lane == 0) {
            S.wgt[warp] = kmin;
            S.wmax[warp] = kmax;
        }
        __syncthreads();
        kmin = __reduce_min_sync(0xffffffffu, lane < kWarps ? S.wgt[lane] : 0xFFFFFFFFu);
        kmax = __reduce_max_sync(0xffffffffu, lane < kWarps ? S.wmax[lane] : 0u);
        tau = radix_select(cluster, 1, S, (uint32_t)k, varying_bits(kmin, kmax), kmin, 3,
                           [&](auto&& f) {
#pragma unroll 1
                               for (int32_t j = w_lo + lane; j < w_hi; j += 32)
                                   f(order_key(j < c ? __ldg(row + j) : end_score[j - c]));
                           },
                           need);
    }

    // scores above the k-th, and equal to it; without a cut among the equal
    // ones they count as above.  A byte per 128-key group for the warp's scan.
    uint32_t bg = 0u, be = 0u;
    if (ranked) {
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
            if (128 * u >= seg) break;
#pragma unroll
            for (int q = 4 * u; q < 4 * u + 4; ++q) {
                if (ties) {
                    bg |= (x[q] > tf ? 1u : 0u) << q;
                    be |= (x[q] == tf ? 1u : 0u) << q;
                } else {
                    bg |= (x[q] >= tf ? 1u : 0u) << q;
                }
            }
        }
    } else {
#pragma unroll
        for (int q = 0; q < KPT; ++q) {
            const bool in = w_lo + 128 * (q >> 2) + 4 * lane + (q & 3) < w_hi;
            const uint32_t key = in ? order_key(x[q]) : 0u;
            bg |= (in && key > tau ? 1u : 0u) << q;
            be |= (in && key == tau ? 1u : 0u) << q;
        }
    }
    auto scan = [&](uint32_t bits, uint64_t& excl, uint64_t& total) -> uint32_t {
        uint64_t p = 0u;
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
            if (128 * u >= seg) break;
            p |= (uint64_t)__popc((bits >> (4 * u)) & 0xFu) << (8 * u);
        }
        uint64_t incl = p;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        total = __shfl_sync(0xffffffffu, incl, 31);
        excl = incl - p;
        // the bytes' sum
        const uint64_t pairs = (total & 0x00FF00FF00FF00FFull) + ((total >> 8) & 0x00FF00FF00FF00FFull);
        return (uint32_t)((pairs * 0x0001000100010001ull) >> 48);
    };
    uint64_t xg, tg, xe = 0u, te = 0u;
    const uint32_t sg = scan(bg, xg, tg), se = ties ? scan(be, xe, te) : 0u;
    __syncthreads();
    if (lane == 0) {
        S.wcnt[warp] = sg;
        S.weq[warp] = se;
    }
    __syncthreads();
    const uint32_t all_g = warp_inclusive_scan(lane < kWarps ? S.wcnt[lane] : 0u);
    uint32_t g0 = __shfl_sync(0xffffffffu, all_g, warp) - sg;
    if (!ties) {
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
            if (128 * u >= seg) break;
            uint32_t g = g0 + ((uint32_t)(xg >> (8 * u)) & 0xFFu);
            const int32_t j = w_lo + 128 * u + 4 * lane;
            const bool all = 128 * u + 128 <= plain;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if ((bg >> (4 * u + e)) & 1u) put(out, g++, k, all ? j + e : position(j + e), status);
            g0 += (uint32_t)(tg >> (8 * u)) & 0xFFu;
        }
        return;
    }
    const uint32_t all_e = warp_inclusive_scan(lane < kWarps ? S.weq[lane] : 0u);
    uint32_t e0 = __shfl_sync(0xffffffffu, all_e, warp) - se;
#pragma unroll 1
    for (int u = 0; u < kGroups; ++u) {
        uint32_t g = g0 + ((uint32_t)(xg >> (8 * u)) & 0xFFu), e = e0 + ((uint32_t)(xe >> (8 * u)) & 0xFFu);
        for (uint32_t both = ((bg | be) >> (4 * u)) & 0xFu; both; both &= both - 1u) {
            const int q = __ffs(both) - 1;
            const int32_t j = w_lo + 128 * u + 4 * lane + q;
            if ((bg >> (4 * u + q)) & 1u) {
                put(out, g + min(e, need), k, position(j), status);
                ++g;
            } else {
                if (e < need) put(out, g + e, k, position(j), status);
                ++e;
            }
        }
        g0 += (uint32_t)(tg >> (8 * u)) & 0xFFu;
        e0 += (uint32_t)(te >> (8 * u)) & 0xFFu;
    }
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
    // Rows that fit a CTA's registers.  With fewer rows than SMs a CTA has an
    // SM to itself: 1024 threads; else 512 and two or three CTAs per SM.
    const bool few = (int64_t)bd.B * bd.max_q < num_sms();
    const int per = (bd.max_ctx + (few ? 1023 : 511)) / (few ? 1024 : 512);
    if (per <= 32) {
        auto kernel = few ? (per <= 8    ? topk_short_kernel<1024, 8>
                             : per <= 16 ? topk_short_kernel<1024, 16>
                                         : topk_short_kernel<1024, 32>)
                          : (per <= 8    ? topk_short_kernel<512, 8>
                             : per <= 16 ? topk_short_kernel<512, 16>
                                         : topk_short_kernel<512, 32>);
        kernel<<<dim3((unsigned)bd.max_q, (unsigned)bd.B), few ? 1024 : 512, 0, stream>>>(bd, scores, ld, k, idx, status,
                                                                                      mask);
        const cudaError_t e = cudaGetLastError();
        if (e == cudaSuccess) count_launches(1);
        return e;
    }
    return launch_rows<true>(bd, RowRange{0, bd.max_q}, scores, ld, false, k, idx, false, status, stream, false, mask);
}

}  // namespace dsa
