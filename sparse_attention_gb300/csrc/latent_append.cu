// latent_append.cu -- latent cache rows of new tokens: RMSNorm of the 512
// compressed values, rotate-half RoPE of the 64 rotary ones, and the write
// into the token's cache slot, in one pass ("GLM-5.1 架构深度拆解", section
// 4.5 Step 2).
//
// A warp per token holds the whole row in registers (two 16-byte pieces of
// the latent part per lane; lanes 0-3 also both halves of 8 rotary pairs), so
// it is read and written once: 2,304 bytes plus 512 of its rotary rows.
// Bound by HBM with many tokens (8,192: 5.3 us = 4.4 TB/s with the launch's
// ramp), by one round trip with few (64: 2.1 us).
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"
#include "tree.h"

namespace dsa {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(w[k] << 16);
        f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

__global__ void __launch_bounds__(32 * kWarps)
    latent_append_kernel(int32_t total_q, const uint16_t* __restrict__ x, int64_t x_stride,
                         const float* __restrict__ gamma, float eps, const float* __restrict__ cos_t,
                         const float* __restrict__ sin_t, int32_t table_rows, const int32_t* __restrict__ positions,
                         const int32_t* __restrict__ slots, int64_t cache_rows, uint16_t* __restrict__ kv,
                         int32_t* status) {
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (r >= total_q) return;
    const uint4* row = reinterpret_cast<const uint4*>(x + r * x_stride);
    // everything is loaded before the slot is looked at: one round trip
    const uint4 a = __ldg(row + lane), b = __ldg(row + 32 + lane);
    uint4 p0 = make_uint4(0, 0, 0, 0), p1 = p0;
    if (lane < 4) {
        p0 = __ldg(row + 64 + lane);
        p1 = __ldg(row + 68 + lane);
    }
    const int32_t slot = __ldg(slots + r), pos = __ldg(positions + r);
    if (slot == -1) return;
    if (slot < 0 || slot >= cache_rows || pos < 0 || pos >= table_rows) {
        if (lane == 0) latch_status(status, DSA_ERR_BAD_INDEX);
        return;
    }
    float v0[8], v1[8], g[8];
    unpack8(a, v0);
    unpack8(b, v1);
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += v0[k] * v0[k] + v1[k] * v1[k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float scale = rsqrtf(sum * (1.f / kDV) + eps);
    uint4* dst = reinterpret_cast<uint4*>(kv + (int64_t)slot * kDQK);
    load8(gamma + 8 * lane, g);
#pragma unroll
    for (int k = 0; k < 8; ++k) v0[k] = v0[k] * scale * g[k];
    dst[lane] = pack8(v0);
    load8(gamma + 256 + 8 * lane, g);
#pragma unroll
    for (int k = 0; k < 8; ++k) v1[k] = v1[k] * scale * g[k];
    dst[32 + lane] = pack8(v1);
    if (lane < 4) {
        float c0[8], s0[8], c1[8], s1[8];
        const float* cr = cos_t + (int64_t)pos * DSA_ROPE_DIM + 8 * lane;
        const float* sr = sin_t + (int64_t)pos * DSA_ROPE_DIM + 8 * lane;
        load8(cr, c0);
        load8(cr + 32, c1);
        load8(sr, s0);
        load8(sr + 32, s1);
        unpack8(p0, v0);
        unpack8(p1, v1);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float lo = v0[k], hi = v1[k];
            v0[k] = lo * c0[k] - hi * s0[k];
            v1[k] = hi * c1[k] + lo * s1[k];
        }
        dst[64 + lane] = pack8(v0);
        dst[68 + lane] = pack8(v1);
    }
}

}  // namespace

cudaError_t launch_latent_append(int32_t total_q, const uint16_t* x, int64_t x_stride, const float* gamma, float eps,
                                 const float* cos_t, const float* sin_t, int32_t table_rows,
                                 const int32_t* positions, const int32_t* slots, int64_t cache_rows, uint16_t* kv,
                                 int32_t* status, cudaStream_t stream) {
    latent_append_kernel<<<(unsigned)((total_q + kWarps - 1) / kWarps), 32 * kWarps, 0, stream>>>(
        total_q, x, x_stride, gamma, eps, cos_t, sin_t, table_rows, positions, slots, cache_rows, kv, status);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace dsa
