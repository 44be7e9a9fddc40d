// tree_mla.cu -- latent attention of a step's new rows over everything they
// see in a (paged or contiguous) cache: the committed rows and, by a bit mask,
// the drafted rows of the same sequence.
//
// A warp per (row, head) walks the visible positions with a running maximum
// and sum (fp32), 18 query and 16 value dims per lane.
#include <cfloat>

#include "internal.h"
#include "ptx.cuh"
#include "tree.h"

namespace dsa {
namespace {

constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

__global__ void __launch_bounds__(32 * kWarps)
    tree_mla_kernel(const BatchDev bd, const PagesDev pg, const uint16_t* __restrict__ q,
                    const uint16_t* __restrict__ kv, const uint64_t* __restrict__ mask, float scale_log2,
                    uint16_t* __restrict__ out, float* __restrict__ lse, int32_t* status) {
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    SeqInfo sq;
    if (!load_seq(bd, b, status, sq)) return;
    if (sq.nq > DSA_MAX_TREE) {
        latch_status(status, DSA_ERR_BAD_BATCH);
        return;
    }
    const int i = blockIdx.x >> 3;
    if (i >= sq.nq) return;
    const int h = (blockIdx.x & 7) * kWarps + (threadIdx.x >> 5);
    const int64_t r = sq.q0 + i;
    const int32_t c = sq.ctx - sq.nq;
    const uint64_t bits = visible_bits(mask[r], i);
    const uint16_t* qr = q + (r * kH + h) * kDQK;
    float qv[18], o[16];
#pragma unroll
    for (int k = 0; k < 18; ++k) qv[k] = bf(qr[lane + 32 * k]);
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = 0.f;
    float m = -INFINITY, l = 0.f;
    for (int32_t s = 0; s < sq.ctx; ++s) {
        if (s >= c && !((bits >> (s - c)) & 1u)) continue;
        const int32_t row = cache_row(bd, pg, b, s);
        if (row < 0) {
            latch_status(status, DSA_ERR_BAD_INDEX);
            return;
        }
        const uint16_t* kr = kv + (int64_t)row * kDQK;
        float kvv[18], dot = 0.f;
#pragma unroll
        for (int k = 0; k < 18; ++k) {
            kvv[k] = bf(kr[lane + 32 * k]);
            dot += qv[k] * kvv[k];
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
        dot *= scale_log2;
        const float mn = fmaxf(m, dot), f = exp2f(m - mn), p = exp2f(dot - mn);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = o[k] * f + p * kvv[k];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int k = 0; k < 16; ++k)
        out[(r * kH + h) * kDV + lane + 32 * k] = (uint16_t)(pack_bf16x2(o[k] * inv, 0.f) & 0xFFFFu);
    if (lse && lane == 0) lse[r * kH + h] = (m + log2f(l)) * kLn2;
}

}  // namespace

size_t tree_mla_scratch_bytes(const BatchDev&) { return 0; }

cudaError_t launch_tree_mla(const BatchDev& bd, const PagesDev& pg, const uint16_t* q, const uint16_t* kv,
                            const uint64_t* mask, float sm_scale, uint16_t* out, float* lse, void*, int32_t* status,
                            cudaStream_t stream) {
    tree_mla_kernel<<<dim3((unsigned)bd.max_q * 8, (unsigned)bd.B), 32 * kWarps, 0, stream>>>(
        bd, pg, q, kv, mask, sm_scale * kLog2e, out, lse, status);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace dsa
