// mla_expand.cu -- latent cache rows expanded to each head's keys and values:
// [192 | 256] x 64 heads = W_kvb c, a product of (rows x 512) by (512 x 28,672)
// whose rows are gathered from a paged or contiguous cache.
//
// Rows are taken in units of 16 consecutive positions of a sequence, aligned
// to 16 (a page holds whole units), and packed 16 units to a tile whatever
// sequences they are of, so that 64 sequences of one new token each fill 4
// tiles and not 64.  A tile is 256 rows x 256 columns on a CTA pair
// (cta_group::2, M = 256, N = 256): the 512 columns of its latent rows stay in
// shared memory (128 KiB a CTA) while the pair walks along W's rows, which come
// through a ring of 64-column chunks from L2 (29 MB, read by every tile).  Each
// pair has an equal share of the tiles, laid end to end, rows slowest.
//
// The epilogue rounds a thread's row to bf16, 64 columns at a time, through 4
// KiB of a warp's own shared memory and TMA stores of its two units: the
// result is the larger part of the traffic, and a warp needs no other to
// write its part.  Values are kept finite (a masked weight of 0 times
// an infinity would be NaN); rows of a unit that are not to be written (before
// `first`, on a bad page) go out one by one.
//
// Two more warps of every CTA copy the rotary keys, NaN for rows that hold a
// NaN or an infinity anywhere, beside all of this.
//
// Roles of a CTA's 12 warps: loads, MMA (rank 0 only), two for rotary keys,
// eight for the epilogue (with four: 188 us for 8,192 rows instead of XX).  Bounds: 32 MMAs of N = 256 a tile, 4,096 cycles for
// 67 MFLOP, and 57 KB of writes a row.
#include <algorithm>

#include "internal.h"
#include "prompt.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 384;
constexpr int kUnit = 16;                        // positions
constexpr int kUnits = 16;                       // of a tile, half of them each CTA's
constexpr int kCols = 256;                       // of a tile
constexpr int kTilesN = kH * kExpRow / kCols;    // 112
constexpr int kChunks = kDV / 64;                // 8
constexpr int kChunkBytes = 128 * 128;           // 128 rows x 64 columns
constexpr int kUnitBytes = kUnit * 128;
constexpr int kBStages = 4, kEpiWarps = 8;
constexpr int kMaxPairs = 96;
static_assert(kH * kExpRow % kCols == 0 && kDV % 64 == 0, "whole tiles");

struct Smem {
    alignas(1024) uint8_t a[kChunks * kChunkBytes];
    alignas(1024) uint8_t b[kBStages * kChunkBytes];
    alignas(1024) uint8_t stage[kEpiWarps * 2 * kUnitBytes];     // a warp's two units x 64 columns
    alignas(8) uint64_t afull[kChunks], aempty, bfull[kBStages], bempty[kBStages], tfull[2], tempty[2];
    uint32_t tmem;
};
static_assert(sizeof(Smem) <= 232448, "one CTA's shared memory");

struct Args {
    BatchDev bd;
    PagesDev pg;
    ExpandedDev x;
    const uint16_t* kv;
    const int32_t* first;        // nullptr: 0 throughout
    const int32_t* start;        // [B + 1] units before a sequence
    int32_t rows_total;          // cache rows
    int32_t* status;
};

__device__ __forceinline__ int32_t first_of(const Args& a, int b) { return a.first ? __ldg(a.first + b) : 0; }

// A unit: its sequence, first position, first position to write, and length of the sequence.
struct Unit {
    int32_t b, pos, first, ctx, at;
};

__device__ __forceinline__ bool unit_of(const Args& a, int32_t u, Unit& x) {
    if (u >= a.start[a.bd.B]) return false;
    x.b = last_at_or_below(a.start, a.bd.B, u);
    x.first = first_of(a, x.b);
    x.pos = (x.first & ~(kUnit - 1)) + kUnit * (u - a.start[x.b]);
    x.ctx = __ldg(a.bd.ctx_len + x.b);
    x.at = __ldg(a.x.off + x.b);
    return true;
}

// Two bf16 kept within the type's largest values; of NaN, one of those.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t v) {
    asm("{\n .reg .b32 t;\n max.bf16x2 t, %0, %1;\n min.bf16x2 %0, t, %2;\n}\n" : "+r"(v) : "r"(0xFF7FFF7Fu), "r"(0x7F7F7F7Fu));
    return v;
}

// Units before each sequence.  One that breaks the bounds has none.
__global__ void __launch_bounds__(1024) expand_plan_kernel(const Args a, int32_t* start) {
    __shared__ int32_t sums[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();
    pdl_wait();
    if (tid == 0) start[0] = 0;
    int32_t carry = 0;
    for (int b0 = 0; b0 < a.bd.B; b0 += 1024) {
        const int b = b0 + tid;
        SeqInfo s{0, 0, 0};
        int32_t n = 0;
        if (b < a.bd.B && load_seq(a.bd, b, a.status, s) && expanded_at(a.x, b, s.ctx, a.status) >= 0) {
            const int32_t f = first_of(a, b);
            if (f < 0 || f > s.ctx) {
                latch_status(a.status, DSA_ERR_BAD_BATCH);
            } else if (f < s.ctx) {
                // 64 bits: a context within 128 of 2^31
                auto up = [](int64_t v, int64_t to) { return (v + to - 1) / to * to; };
                const int64_t end = up(f, kExpRoom) < up(s.ctx, kExpRoom) ? up(s.ctx, kExpRoom) : up(s.ctx, kUnit);
                n = (int32_t)((end - (f & ~(kUnit - 1))) / kUnit);
            }
        }
        int32_t incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        if (warp == 0) {
            int32_t v = sums[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            sums[lane] = v;
        }
        __syncthreads();
        if (b < a.bd.B) start[b + 1] = carry + incl + (warp > 0 ? sums[warp - 1] : 0);
        carry += sums[31];
        __syncthreads();
    }
}

// Rotary keys of the units u0, u0 + step, ..: a warp.
__device__ __forceinline__ void rotary_keys(const Args& a, int32_t u0, int32_t step) {
    const int lane = (int)lane_id();
    const int32_t units = a.start[a.bd.B];
    for (int32_t u = u0; u < units; u += step) {
        Unit x;
        unit_of(a, u, x);
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
        for (int i = 0; i < kChunks; ++i) mbar_init(smem_u32(&S.afull[i]), 2);
        mbar_init(smem_u32(&S.aempty), 1);
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
    tc_fence_before();
    __syncthreads();
    cluster_wait();                              // .. and this CTA the peer's
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    const int64_t tiles = (int64_t)((a.start[a.bd.B] + kUnits - 1) / kUnits) * kTilesN;
    const int32_t t_lo = (int32_t)(tiles * pair / pairs), t_hi = (int32_t)(tiles * (pair + 1) / pairs);
    bool ok = true;
    auto lead = [&](uint64_t& b) -> uint32_t { return map_to_cluster_rank(smem_u32(&b), 0); };
    // bounded; a thread whose wait expired waits for nothing any more
    auto wait = [&](uint64_t& b, uint32_t parity) -> bool {
        if (ok && !mbar_wait_rolled(smem_u32(&b), parity)) {
            ok = false;
            latch_status(a.status, DSA_ERR_TIMEOUT);
        }
        return ok;
    };

    if (warp == 0) {
        // loads
        int32_t m = -1;                          // the tile's rows
        uint32_t it = 0, turn = 0;
        for (int32_t t = t_lo; ok && t < t_hi; ++t) {
            if (t / kTilesN != m) {
                m = t / kTilesN;
                if (turn > 0) wait(S.aempty, (turn - 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ++turn;
                // a unit's 16 rows of each chunk; zeros for rows that are none
                Unit x;
                int32_t row = a.rows_total;
                if (lane < kUnits / 2 && unit_of(a, kUnits * m + kUnits / 2 * (int)rank + lane, x) && x.pos < x.ctx) {
                    const int32_t r = cache_row(a.bd, a.pg, x.b, x.pos);
                    if (r >= 0) row = r;
                }
#pragma unroll 1
                for (int c = 0; c < kChunks; ++c) {
                    if (lane == 0) mbar_arrive_expect_tx_pair(lead(S.afull[c]), kChunkBytes);
                    __syncwarp();
                    if (lane < kUnits / 2)
                        tma_load_2d_pair(smem_u32(S.a + c * kChunkBytes + lane * kUnitBytes), &tm_a, lead(S.afull[c]),
                                         64 * c, row);
                }
            }
            if (lane == 0) {
                for (int c = 0; ok && c < kChunks; ++c, ++it) {
                    const uint32_t s = it % kBStages;
                    if (it >= kBStages && !wait(S.bempty[s], (it / kBStages - 1) & 1)) break;
                    mbar_arrive_expect_tx_pair(lead(S.bfull[s]), kChunkBytes);
                    tma_load_2d_pair(smem_u32(S.b + s * kChunkBytes), &tm_b, lead(S.bfull[s]), 64 * c,
                                     (t % kTilesN) * kCols + 128 * (int)rank);
                }
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, ok);
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            // MMA, by one lane that also waits
            constexpr uint32_t kId = idesc_bf16_f32(256, kCols);
            const uint64_t da = sdesc_sw128(smem_u32(S.a), 0, 1024), db = sdesc_sw128(smem_u32(S.b), 0, 1024);
            uint32_t it = 0, turn = 0;
            for (int32_t t = t_lo; ok && t < t_hi; ++t) {
                const uint32_t n = (uint32_t)(t - t_lo), buf = n & 1;
                if (t == t_lo || t % kTilesN == 0) ++turn;
                if (n >= 2 && !wait(S.tempty[buf], ((n >> 1) - 1) & 1)) break;
#pragma unroll 1
                for (int c = 0; c < kChunks; ++c, ++it) {
                    const uint32_t s = it % kBStages;
                    if (!wait(S.afull[c], (turn - 1) & 1)) break;
                    if (!wait(S.bfull[s], (it / kBStages) & 1)) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16_ss_pair(tmem + kCols * buf, da + c * (kChunkBytes >> 4) + 2 * k,
                                         db + s * (kChunkBytes >> 4) + 2 * k, kId, (c | k) != 0);
                    mma_commit_pair(smem_u32(&S.bempty[s]));
                }
                if (!ok) break;
                mma_commit_pair(smem_u32(&S.tfull[buf]));
                if (t + 1 < t_hi && (t + 1) % kTilesN == 0) mma_commit_pair(smem_u32(&S.aempty));
            }
        }
        __syncwarp();
    } else if (warp < 4) {
        rotary_keys(a, 2 * (int)blockIdx.x + warp - 2, 2 * (int)gridDim.x);
    } else {
        // epilogue: TMEM lane = row of this CTA, half of the tile's columns a warp
        const int w = warp & 3, half = (warp - 4) >> 2, in = lane & (kUnit - 1);
        const uint32_t tl = tmem + ((uint32_t)(32 * w) << 16);
        uint8_t* const stage = S.stage + (warp - 4) * 2 * kUnitBytes;
        int32_t m = -1, dst = -1;                // the row's place, -1: not written
        bool zero = false, whole = false;        // .. past the sequence; all of its unit's rows are written
        for (int32_t t = t_lo; t < t_hi; ++t) {
            if (t / kTilesN != m) {
                m = t / kTilesN;
                Unit x;
                dst = -1;
                if (unit_of(a, kUnits * m + kUnits / 2 * (int)rank + 2 * w + (lane >> 4), x)) {
                    const int32_t pos = x.pos + in;
                    zero = pos >= x.ctx;
                    if (pos >= x.first && (zero || cache_row(a.bd, a.pg, x.b, pos) >= 0)) dst = x.at + pos;
                }
                const uint32_t writes = __ballot_sync(0xffffffffu, dst >= 0);
                whole = ((writes >> (lane & 16)) & 0xFFFFu) == 0xFFFFu;
            }
            const uint32_t n = (uint32_t)(t - t_lo), buf = n & 1;
            wait(S.tfull[buf], (n >> 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < kCols / 2; c += 64) {
                const int32_t col = kCols / 2 * half + c;
                uint32_t r[2][32];
                tmem_ld_32x32b_x32(tl + kCols * buf + col, r[0]);
                tmem_ld_32x32b_x32(tl + kCols * buf + col + 32, r[1]);
                tmem_ld_wait();
                if (c == kCols / 2 - 64) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_pair(lead(S.tempty[buf]));
                }
                bulk_wait_read<0>();             // the stores of 64 columns ago
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
                const int32_t to = (t % kTilesN) * kCols + col;
                if (in == 0) {
                    if (whole) tma_store_2d(&tm_out, smem_u32(stage + (lane >> 4) * kUnitBytes), to, dst);
                    bulk_commit();
                }
                if (!__all_sync(0xffffffffu, whole)) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int row = 4 * k + (lane >> 3), at = lane & 7;
                        const int32_t d = __shfl_sync(0xffffffffu, whole ? -1 : dst, row);
                        if (d >= 0)
                            *reinterpret_cast<uint4*>(a.x.kv + (int64_t)d * kH * kExpRow + to + 8 * at) =
                                *reinterpret_cast<const uint4*>(stage + row * 128 + ((at ^ (row & 7)) << 4));
                    }
                    __syncwarp();
                }
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
    int32_t* start = static_cast<int32_t*>(scratch);
    Args a{};
    a.bd = bd;
    a.pg = pg;
    a.x = x;
    a.kv = kv;
    a.first = first;
    a.start = start;
    a.rows_total = pg.table ? pg.pool_pages << pg.shift : (int32_t)(bd.B * bd.stride);
    a.status = status;
    CUtensorMap tm_a, tm_b, tm_out;
    if (!make_tmap_bf16_2d(&tm_a, kv, kDQK, (uint64_t)a.rows_total, 64, kUnit) ||
        !make_tmap_bf16_2d(&tm_b, w_kvb, kDV, (uint64_t)kH * kExpRow, 64, 128) ||
        !make_tmap_bf16_2d(&tm_out, x.kv, (uint64_t)kH * kExpRow, (uint64_t)x.rows, 64, kUnit))
        return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(1024);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, expand_plan_kernel, a, start);
    if (e != cudaSuccess) return e;
    count_launches(1);
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
