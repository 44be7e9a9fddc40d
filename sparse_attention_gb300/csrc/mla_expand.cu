// mla_expand.cu -- latent cache rows expanded to each head's keys and values:
// [192 | 256] x 64 heads = W_kvb c, a product of (rows x 512) by (512 x 28,672)
// whose rows are gathered from a paged or contiguous cache.
//
// Rows are taken in units of 16 consecutive positions of a sequence, aligned
// to 16 (a page holds whole units), and packed 16 units to a tile whatever
// sequences they are of, so that 64 sequences of one new token each fill 4
// tiles and not 64.  A tile is 256 rows x 128 columns on a CTA pair
// (cta_group::2, M = 256, N = 128).  The pair keeps its 256 rows, all 512 columns
// of them, in tensor memory (half of it) as the products' A and walks along
// W's rows, which come from L2 (29 MB, read by every tile, so evicted last)
// through a ring of 32 KB boxes.  (A in shared memory would be read at 32 bytes a
// cycle beside W's 32 + 32 and the results' 16 + 16, all of its bandwidth; boxes
// of 8 KB, a chunk of 64 columns each, cost the lane that issues them 480 cycles
// apiece and the call 198 instead of 143 us for 8,192 rows.)  Each pair has an
// equal share of the tiles, laid end to end, rows slowest.
//
// The epilogue rounds a thread's row to bf16, 64 columns a warp, through 4 KiB of
// its own shared memory and TMA stores of its two units: the result is the
// larger part of the traffic, and a warp needs no other to write its part.
// Values are kept finite (a masked weight of 0 times an infinity would be
// NaN); rows of a unit that are not to be written (before `first`, on a bad
// page) go out one by one.
//
// One more warp of every CTA copies the rotary keys, NaN for rows that hold a
// NaN or an infinity anywhere, beside all of this.
//
// Roles of a CTA's 12 warps: W loads, MMA (rank 0 only), rotary keys, row loads,
// eight for rows to tensor memory and for the epilogue.  Bounds: 32 MMAs of
// N = 128 a tile, 2,048 cycles for 34 MFLOP, and 57 KB of writes a row.  Measured:
// 8,192 rows behind 1,003 138-141 us in single calls and short loops (1,710-1,740
// TFLOP/s, 1,921 measured peak), 156 in long ones (1,540, 1,730 sustained); 8 prompts of
// 100 to 300 tokens 37 us.
#include <algorithm>

#include "internal.h"
#include "prompt.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 384;
constexpr int kUnit = 16;                        // positions
constexpr int kUnits = 16;                       // of a tile, half of them each CTA's
constexpr int kCols = 128;                       // of a tile
constexpr int kTilesN = kH * kExpRow / kCols;    // 224
constexpr int kChunks = kDV / 64;                // 8
constexpr int kGroup = 4;                        // chunks of W a stage
constexpr int kABytes = 128 * 128, kBBytes = kGroup * 64 * 128;   // 128 rows x 64 columns; 64 rows x a stage's
constexpr int kUnitBytes = kUnit * 128;
constexpr int kASlots = 4, kBStages = 4, kEpiWarps = 8;
constexpr uint32_t kDCol = kDV / 2;              // TMEM columns: A (two values each), then two accumulators
constexpr int kMaxPairs = 96;
static_assert(kH * kExpRow % kCols == 0 && kDV % 64 == 0, "whole tiles");

struct Smem {
    alignas(1024) uint8_t a[kASlots * kABytes];
    alignas(1024) uint8_t b[kBStages * kBBytes];
    alignas(1024) uint8_t stage[kEpiWarps * 2 * kUnitBytes];     // a warp's two units x 64 columns
    alignas(8) uint64_t afull[kASlots], aempty[kASlots], aready, bfull[kBStages], bempty[kBStages], tfull[2], tempty[2];
    int32_t start[kThreads + 1], sums[kThreads / 32];        // the plan of a batch of few sequences
    uint32_t tmem;
};
static_assert(sizeof(Smem) <= 232448, "one CTA's shared memory");

struct Args {
    BatchDev bd;
    PagesDev pg;
    ExpandedDev x;
    const uint16_t* kv;
    const int32_t* first;        // nullptr: 0 throughout
    const int32_t* start;        // [B + 1] units before a sequence; nullptr: each CTA sums them up itself
    int32_t rows_total;          // cache rows
    int32_t* status;
};

// A pair's tiles: its share of them laid end to end, rows slowest, the columns
// of a tile's rows in an order that has all pairs at W's same few rows at a
// time: step i of any pair takes, while it can, a column tile that is i
// modulo the shares' length (76 pairs otherwise read as many places of W: 143 us
// for 8,192 rows instead of 138).
struct Walk {
    int32_t t, hi, share;        // the next rows' first tile, the end, tiles of a share
    int32_t rows = 0, col = 0;   // the tile
    bool fresh = false;          // .. is the first of its rows
    int32_t step = 0, left = 0, begin = 0, end = 0;
    __device__ Walk(int32_t lo, int32_t hi_, int32_t share_) : t(lo), hi(hi_), share(share_) {}
    __device__ bool next() {
        fresh = left == 0;
        if (fresh) {
            if (t >= hi) return false;
            rows = t / kTilesN;
            begin = t - rows * kTilesN;
            end = min(kTilesN, begin + hi - t);
            left = end - begin;
            t += left;
            const int32_t off = (step - begin) % share;
            col = begin + (off < 0 ? off + share : off);
            if (col >= end) col = begin;
        } else if (++col == end) {
            col = begin;
        }
        --left;
        ++step;
        return true;
    }
};

__device__ __forceinline__ int32_t first_of(const Args& a, int b) { return a.first ? __ldg(a.first + b) : 0; }

// A unit: its sequence, first position, first position to write, and length of the sequence.
struct Unit {
    int32_t b, pos, first, ctx, at;
};

__device__ __forceinline__ bool unit_of(const Args& a, const int32_t* start, int32_t u, Unit& x) {
    if (u >= start[a.bd.B]) return false;
    x.b = last_at_or_below(start, a.bd.B, u);
    x.first = first_of(a, x.b);
    x.pos = (x.first & ~(kUnit - 1)) + kUnit * (u - start[x.b]);
    x.ctx = __ldg(a.bd.ctx_len + x.b);
    x.at = __ldg(a.x.off + x.b);
    return true;
}

// Two bf16 kept within the type's largest values; of NaN, one of those.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t v) {
    asm("{\n .reg .b32 t;\n max.bf16x2 t, %0, %1;\n min.bf16x2 %0, t, %2;\n}\n" : "+r"(v) : "r"(0xFF7FFF7Fu), "r"(0x7F7F7F7Fu));
    return v;
}

// Units of sequence b: none of one that breaks the bounds.
__device__ __forceinline__ int32_t units_of(const Args& a, int b) {
    if (b >= a.bd.B) return 0;
    SeqInfo s;
    // with the lengths, not behind them
    const int32_t lo = __ldg(a.x.off + b), hi = __ldg(a.x.off + b + 1), f = first_of(a, b);
    if (!load_seq(a.bd, b, a.status, s) || expanded_at(a.x, lo, hi, s.ctx, a.status) < 0) return 0;
    if (f < 0 || f > s.ctx) latch_status(a.status, DSA_ERR_BAD_BATCH);
    if (f < 0 || f >= s.ctx) return 0;
    // 64 bits: a context within 16 of 2^31
    return (int32_t)(((int64_t)s.ctx + kUnit - 1) / kUnit) - f / kUnit;
}

// Units before each sequence, for batches of more than kThreads (a launch more:
// 4 us).
__global__ void __launch_bounds__(1024) expand_plan_kernel(const Args a, int32_t* start) {
    __shared__ int32_t sums[32];
    const int tid = threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    if (tid == 0) start[0] = 0;
    int32_t carry = 0;
    for (int b0 = 0; b0 < a.bd.B; b0 += 1024) {
        const int32_t n = units_of(a, b0 + tid);
        int32_t all;
        const int32_t before = block_sum_before(n, 32, sums, all);
        if (b0 + tid < a.bd.B) start[b0 + tid + 1] = carry + before + n;
        carry += all;
        __syncthreads();
    }
}

// Rotary keys of the units u0, u0 + step, ..: a warp.
__device__ __forceinline__ void rotary_keys(const Args& a, const int32_t* start, int32_t u0, int32_t step) {
    const int lane = (int)lane_id();
    const int32_t units = start[a.bd.B];
    for (int32_t u = u0; u < units; u += step) {
        Unit x;
        unit_of(a, start, u, x);
        const int32_t row0 = x.pos < x.ctx ? cache_row(a.bd, a.pg, x.b, x.pos) : 0;
        if (row0 < 0) {
            // the unit's positions are not written, what lies behind the sequence is
            if (lane == 0) latch_status(a.status, DSA_ERR_BAD_INDEX);
            x.first = x.ctx;
            x.ctx = 0;
        }
#pragma unroll 1
        for (int i0 = 0; i0 < kUnit; i0 += 4) {
            uint4 v[4][3];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool live = x.pos + i0 + i < x.ctx;
                const uint4* row = reinterpret_cast<const uint4*>(a.kv + (int64_t)(row0 + i0 + i) * kDQK);
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    v[i][k] = live && 32 * k + lane < kDQK / 8 ? __ldg(row + 32 * k + lane) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                bool hit = false;
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    const uint32_t w[4] = {v[i][k].x, v[i][k].y, v[i][k].z, v[i][k].w};
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        hit = hit || (w[q] & 0x7F80u) == 0x7F80u || (w[q] & 0x7F800000u) == 0x7F800000u;
                }
                const uint32_t nan = __any_sync(0xffffffffu, hit) ? 0x7FFF7FFFu : 0u;
                if (lane < DSA_ROPE_DIM / 8 && x.pos + i0 + i >= x.first)
                    reinterpret_cast<uint4*>(a.x.k_pe + (int64_t)(x.at + x.pos + i0 + i) * DSA_ROPE_DIM)[lane] =
                        make_uint4(v[i][2].x | nan, v[i][2].y | nan, v[i][2].z | nan, v[i][2].w | nan);
            }
        }
    }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mla_expand_kernel(const Args a, const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                      const __grid_constant__ CUtensorMap tm_out) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem& S = *reinterpret_cast<Smem*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    pdl_launch_dependents();
    if (smem_u32(smem_raw) & 1023u) {            // the swizzle goes by address bits
        if (tid == 0) latch_status(a.status, DSA_ERR_INTERNAL);
        return;                                  // both CTAs: the same launch, the same offset
    }
    if (tid == kThreads - 32) {
        for (int i = 0; i < kASlots; ++i) {
            mbar_init(smem_u32(&S.afull[i]), 1);
            mbar_init(smem_u32(&S.aempty[i]), kEpiWarps / 2);
        }
        mbar_init(smem_u32(&S.aready), 2 * kEpiWarps);
        for (int i = 0; i < kBStages; ++i) {
            mbar_init(smem_u32(&S.bfull[i]), 2);
            mbar_init(smem_u32(&S.bempty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&S.tfull[i]), 1);
            mbar_init(smem_u32(&S.tempty[i]), 2 * kEpiWarps);
        }
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc_pair(smem_u32(&S.tmem), 512);
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tm_a);
        prefetch_tmap(&tm_b);
        prefetch_tmap(&tm_out);
    }
    __syncwarp();
    cluster_arrive();                            // the peer may use this CTA's barriers and TMEM ..
    pdl_wait();                                  // inputs, and the plan
    if (!a.start) {
        const int32_t n = units_of(a, tid);
        int32_t all;
        S.start[tid + 1] = block_sum_before(n, kThreads / 32, S.sums, all) + n;
        if (tid == 0) S.start[0] = 0;
    }
    const int32_t* const start = a.start ? a.start : S.start;
    tc_fence_before();
    __syncthreads();
    cluster_wait();                              // .. and this CTA the peer's
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    const int64_t tiles = (int64_t)((start[a.bd.B] + kUnits - 1) / kUnits) * kTilesN;
    const int32_t t_lo = (int32_t)(tiles * pair / pairs), t_hi = (int32_t)(tiles * (pair + 1) / pairs);
    Walk at(t_lo, t_hi, (int32_t)((tiles + pairs - 1) / pairs));
    bool ok = true;
    auto lead = [&](uint64_t& b) -> uint32_t { return map_to_cluster_rank(smem_u32(&b), 0); };
    // bounded; a thread whose wait expired waits for nothing any more
    auto wait = [&](uint64_t& b, uint32_t parity) -> bool {
        ok = ok && mbar_wait_small(smem_u32(&b), parity, a.status);
        return ok;
    };

    if (warp == 0) {
        // W, by one lane
        if (lane == 0) {
            const uint64_t keep = l2_evict_last_policy();
            uint32_t it = 0;
            while (ok && at.next()) {
#pragma unroll 1
                for (int c = 0; c < kChunks; c += kGroup, ++it) {
                    const uint32_t s = it % kBStages;
                    if (it >= kBStages && !wait(S.bempty[s], (it / kBStages - 1) & 1)) break;
                    mbar_arrive_expect_tx_pair(lead(S.bfull[s]), kBBytes);
                    tma_load_3d_pair_hint(smem_u32(S.b + s * kBBytes), &tm_b, lead(S.bfull[s]), 0,
                                          at.col * kCols + kCols / 2 * (int)rank, c, keep);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            // MMA, by one lane that also waits
            constexpr uint32_t kId = idesc_bf16_f32(256, kCols);
            const uint64_t db = sdesc_sw128(smem_u32(S.b), 0, 1024);
            uint32_t it = 0, turn = 0;
            for (uint32_t n = 0; ok && at.next(); ++n) {
                const uint32_t buf = n & 1;
                if (at.fresh) {
                    if (!wait(S.aready, turn & 1)) break;
                    ++turn;
                }
                if (n >= 2 && !wait(S.tempty[buf], ((n >> 1) - 1) & 1)) break;
#pragma unroll 1
                for (int c = 0; c < kChunks; c += kGroup, ++it) {
                    const uint32_t s = it % kBStages;
                    if (!wait(S.bfull[s], (it / kBStages) & 1)) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4 * kGroup; ++k)
                        mma_bf16_ts_pair(tmem + kDCol + kCols * buf, tmem + 32 * c + 8 * k,
                                         db + (s * kBBytes + (k >> 2) * 64 * 128 + 32 * (k & 3)) / 16, kId, (c | k) != 0);
                    mma_commit_pair(smem_u32(&S.bempty[s]));
                }
                if (!ok) break;
                mma_commit_pair(smem_u32(&S.tfull[buf]));
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        rotary_keys(a, start, (int)blockIdx.x, (int)gridDim.x);
    } else if (warp == 3) {
        // latent rows: a unit's 16 of each chunk a lane; zeros for rows that are none
        uint32_t it = 0;
        for (int32_t m = t_lo / kTilesN; ok && t_lo < t_hi && m <= (t_hi - 1) / kTilesN; ++m) {
            Unit x;
            int32_t row = a.rows_total;
            if (lane < kUnits / 2 && unit_of(a, start, kUnits * m + kUnits / 2 * (int)rank + lane, x) && x.pos < x.ctx) {
                const int32_t r = cache_row(a.bd, a.pg, x.b, x.pos);
                if (r >= 0) row = r;
            }
#pragma unroll 1
            for (int c = 0; ok && c < kChunks; ++c, ++it) {
                const uint32_t s = it % kASlots;
                if (lane == 0 && (it < kASlots || wait(S.aempty[s], (it / kASlots - 1) & 1)))
                    mbar_arrive_expect_tx(smem_u32(&S.afull[s]), kABytes);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (ok && lane < kUnits / 2)
                    tma_load_2d(smem_u32(S.a + s * kABytes + lane * kUnitBytes), &tm_a, smem_u32(&S.afull[s]), 64 * c, row);
            }
        }
    } else {
        // epilogue: TMEM lane = row of this CTA, half of the tile's columns a warp
        const int w = warp & 3, half = (warp - 4) >> 2, in = lane & (kUnit - 1);
        const uint32_t tl = tmem + ((uint32_t)(32 * w) << 16);
        uint8_t* const stage = S.stage + (warp - 4) * 2 * kUnitBytes;
        uint32_t chunks = 0;                     // of rows that went to tensor memory
        int32_t dst = -1;                        // the row's place, -1: not written
        bool zero = false, whole = false;        // .. past the sequence; all of its unit's rows are written
        for (uint32_t n = 0; at.next(); ++n) {
            if (at.fresh) {
                Unit x;
                dst = -1;
                if (unit_of(a, start, kUnits * at.rows + kUnits / 2 * (int)rank + 2 * w + (lane >> 4), x)) {
                    const int32_t pos = x.pos + in;
                    zero = pos >= x.ctx;
                    if (pos >= x.first && (zero || cache_row(a.bd, a.pg, x.b, pos) >= 0)) dst = x.at + pos;
                }
                const uint32_t writes = __ballot_sync(0xffffffffu, dst >= 0);
                whole = ((writes >> (lane & 16)) & 0xFFFFu) == 0xFFFFu;
                // The tile's rows to tensor memory, a chunk of every two each half of the
                // warps.  No product reads the last ones any more: their
                // last accumulator was full.
#pragma unroll 1
                for (int c = half; c < kChunks; c += 2) {
                    const uint32_t it = chunks + c, s = it % kASlots;
                    wait(S.afull[s], (it / kASlots) & 1);
                    __syncwarp();
                    const uint8_t* from = S.a + s * kABytes + (32 * w + lane) * 128;
                    uint32_t r[32];
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        const uint4 q = *reinterpret_cast<const uint4*>(from + ((v ^ (lane & 7)) << 4));
                        r[4 * v] = q.x, r[4 * v + 1] = q.y, r[4 * v + 2] = q.z, r[4 * v + 3] = q.w;
                    }
                    tmem_st_32x32b_x32(tl + 32 * c, r);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&S.aempty[s]));
                }
                chunks += kChunks;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(lead(S.aready));
            }
            const uint32_t buf = n & 1;
            wait(S.tfull[buf], (n >> 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            uint32_t r[2][32];
            tmem_ld_32x32b_x32(tl + kDCol + kCols * buf + 64 * half, r[0]);
            tmem_ld_32x32b_x32(tl + kDCol + kCols * buf + 64 * half + 32, r[1]);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(lead(S.tempty[buf]));
            bulk_wait_read<0>();                 // the stores of the tile before
            __syncwarp();
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                uint32_t p[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    p[k] = finite_bf16x2(pack_bf16x2(__uint_as_float(r[v >> 2][8 * (v & 3) + 2 * k]),
                                                     __uint_as_float(r[v >> 2][8 * (v & 3) + 2 * k + 1])));
                *reinterpret_cast<uint4*>(stage + lane * 128 + ((v ^ (lane & 7)) << 4)) =
                    zero ? make_uint4(0, 0, 0, 0) : make_uint4(p[0], p[1], p[2], p[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            const int32_t to = at.col * kCols + 64 * half;
            if (in == 0) {
                if (whole) tma_store_2d(&tm_out, smem_u32(stage + (lane >> 4) * kUnitBytes), to, dst);
                bulk_commit();
            }
            if (!__all_sync(0xffffffffu, whole)) {
#pragma unroll 1
                for (int k = 0; k < 8; ++k) {
                    const int row = 4 * k + (lane >> 3), piece = lane & 7;
                    const int32_t d = __shfl_sync(0xffffffffu, whole ? -1 : dst, row);
                    if (d >= 0)
                        *reinterpret_cast<uint4*>(a.x.kv + (int64_t)d * kH * kExpRow + to + 8 * piece) =
                            *reinterpret_cast<const uint4*>(stage + row * 128 + ((piece ^ (row & 7)) << 4));
                }
                __syncwarp();
            }
        }
        bulk_wait_all();
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

}  // namespace

size_t mla_expand_scratch_bytes(const BatchDev& bd) { return ((size_t)bd.B + 1) * sizeof(int32_t); }

cudaError_t launch_mla_expand(const BatchDev& bd, const PagesDev& pg, const uint16_t* kv, const uint16_t* w_kvb,
                              const int32_t* first, const ExpandedDev& x, void* scratch, int32_t* status,
                              cudaStream_t stream) {
    const int pairs = resident_pairs(reinterpret_cast<const void*>(mla_expand_kernel), kThreads, sizeof(Smem), kMaxPairs);
    Args a{};
    a.bd = bd;
    a.pg = pg;
    a.x = x;
    a.kv = kv;
    a.first = first;
    a.rows_total = pg.table ? pg.pool_pages << pg.shift : (int32_t)(bd.B * bd.stride);
    a.status = status;
    CUtensorMap tm_a, tm_b, tm_out;
    if (!make_tmap_bf16_2d(&tm_a, kv, kDQK, (uint64_t)a.rows_total, 64, kUnit) ||
        !make_tmap_bf16_chunks(&tm_b, w_kvb, kChunks, (uint64_t)kH * kExpRow, kCols / 2, kGroup) ||
        !make_tmap_bf16_2d(&tm_out, x.kv, (uint64_t)kH * kExpRow, (uint64_t)x.rows, 64, kUnit))
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
        cfg.gridDim = dim3(1);
        cfg.blockDim = dim3(1024);
        if ((e = cudaLaunchKernelEx(&cfg, expand_plan_kernel, a, start)) != cudaSuccess) return e;
        count_launches(1);
        a.start = start;
    }
    if ((e = cudaFuncSetAttribute(mla_expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem))) !=
        cudaSuccess)
        return e;
    cfg.gridDim = dim3(2 * (unsigned)pairs);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Smem);
    e = cudaLaunchKernelEx(&cfg, mla_expand_kernel, a, tm_a, tm_b, tm_out);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace dsa
