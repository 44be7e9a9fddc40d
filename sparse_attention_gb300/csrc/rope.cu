// rope.cu -- rotary positions: tables of cosines and sines for any range of
// positions, plain or scaled for long contexts, and the rotation of a part of
// every head ("GLM-5.1 架构深度拆解", section 4.5 Steps 1-3 and section 3.6
// Step 1: 64 of a query's 256 columns, 64 of an index query's 128).
//
// Tables.  Pair i of position p turns by p f_i, f_i = base^(-2i/dim).  In 64-bit
// fixed point an angle is a fraction of a turn: F_i = 2^64 f_i / (2 pi) is formed
// on the host, p F_i mod 2^64 drops whole turns for nothing, its upper bits are
// the nearest quarter turn, and the signed rest is rounded to a float (relative
// to its own size, so small angles lose nothing).  Far positions are as exact
// as near ones (error of the angle p 2^-56 turns, from F_i's 53 bits) without
// 64-bit floating point, which this GPU has little of.  Bound by the writes and the
// launch: 202,752 x 64 x 2 floats are 104 MB.
//
// Rotation.  A thread holds 8 pairs of up to 4 heads of a token, so that a
// token's table row is read once for them, all loads in flight before the
// first store.  Bound by HBM with many tokens, by one round trip with few.
#include <algorithm>
#include <cmath>

#include "internal.h"
#include "prompt.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = DSA_MAX_ROPE_DIM / 2;

struct Turns {
    uint64_t f[kMaxPairs];       // 2^64 turns per position
};

// cos and sin of phase / 2^64 turns: within an eighth of a turn of a quarter,
// so the Taylor series' first five terms leave 1.8e-9 of a sine, its first six 1.2e-10
// of a cosine.  With the fp32 roundings (three in x, one at the end, the inner
// ones weighed by what their terms add) either is off by at most 4.4 x 2^-24 of its
// size; mscale's own rounding and its product add a 2^-24 each.
__device__ __forceinline__ void turn(uint64_t phase, float& c, float& s) {
    const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
    const int64_t rest = (int64_t)(phase - ((uint64_t)quarter << 62));
    const float x = __ll2float_rn(rest) * (float)(2 * M_PI * 0x1p-64), z = x * x;
    float c1 = -1.f / 3628800, s1 = 1.f / 362880;
    c1 = fmaf(c1, z, 1.f / 40320);
    s1 = fmaf(s1, z, -1.f / 5040);
    c1 = fmaf(c1, z, -1.f / 720);
    s1 = fmaf(s1, z, 1.f / 120);
    c1 = fmaf(c1, z, 1.f / 24);
    s1 = fmaf(s1, z, -1.f / 6);
    c1 = fmaf(c1, z, -0.5f);
    s1 = fmaf(s1 * z, x, x);
    c1 = fmaf(c1, z, 1.f);
    const bool odd = quarter & 1;
    c = odd ? s1 : c1;
    s = odd ? c1 : s1;
    if ((quarter + 1) & 2) c = -c;
    if (quarter & 2) s = -s;
}

__global__ void __launch_bounds__(kThreads)
    rope_table_kernel(const __grid_constant__ Turns t, int32_t rows, int32_t first, int32_t pairs, float mscale,
                      float* __restrict__ cos_t, float* __restrict__ sin_t) {
    pdl_launch_dependents();
    const int quads = pairs / 4;                 // a thread's four pairs
    const int64_t n = (int64_t)rows * quads;
    const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    pdl_wait();
    if (e >= n) return;
    const int32_t r = (int32_t)(e / quads), i = 4 * (int32_t)(e - (int64_t)r * quads);
    const uint64_t p = (uint64_t)first + (uint64_t)r;
    float4 c, s;
    float* cp = &c.x;
    float* sp = &s.x;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        turn(p * t.f[i + k], cp[k], sp[k]);
        cp[k] *= mscale;
        sp[k] *= mscale;
    }
    float* cr = cos_t + (int64_t)r * 2 * pairs + i;
    float* sr = sin_t + (int64_t)r * 2 * pairs + i;
    *reinterpret_cast<float4*>(cr) = c;
    *reinterpret_cast<float4*>(cr + pairs) = c;
    *reinterpret_cast<float4*>(sr) = s;
    *reinterpret_cast<float4*>(sr + pairs) = s;
}

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

struct RopeArgs {
    int32_t total, heads, dim, table_rows;
    const uint16_t* x;           // not __restrict__: may be out
    int64_t x_token, x_head;
    const float *cos_t, *sin_t;
    const int32_t* positions;
    uint16_t* out;
    int64_t out_token, out_head;
    int32_t pieces;              // dim / 16: threads of a head, 8 pairs each
    int32_t groups;              // ceil(heads / U): a thread takes heads g, g + groups, ..
    int32_t tokens;              // of a CTA
    float sign;                  // of the sines
    int32_t* status;
};

// kNeighbour: pairs (2i, 2i + 1), else (i, i + dim / 2).  U heads a thread.
template <bool kNeighbour, int U>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int32_t per = a.groups * a.pieces;
    const int32_t t0 = blockIdx.x * a.tokens, units = min(a.tokens, a.total - t0) * per;
    const int32_t second = kNeighbour ? 8 : a.dim / 2;       // where the other 8 of a thread's 16 values are
    for (int32_t u = threadIdx.x; u < units; u += kThreads) {
        const int32_t t = t0 + u / per, v = u % per, g = v / a.pieces, p = v % a.pieces;
        const int32_t at = (kNeighbour ? 16 : 8) * p;
        const uint16_t* x = a.x + t * a.x_token + at;
        uint4 lo[U], hi[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int32_t h = g + k * a.groups;
            if (h >= a.heads) break;
            lo[k] = *reinterpret_cast<const uint4*>(x + h * a.x_head);
            hi[k] = *reinterpret_cast<const uint4*>(x + h * a.x_head + second);
        }
        const int32_t pos = __ldg(a.positions + t);
        if (pos < 0 || pos >= a.table_rows) {
            if (pos != -1 && v == 0) latch_status(a.status, DSA_ERR_BAD_INDEX);
            continue;
        }
        float c[8], s[8];
        load8(a.cos_t + (int64_t)pos * a.dim + 8 * p, c);
        load8(a.sin_t + (int64_t)pos * a.dim + 8 * p, s);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k] *= a.sign;
        uint16_t* out = a.out + t * a.out_token + at;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int32_t h = g + k * a.groups;
            if (h >= a.heads) break;
            float f0[8], f1[8];
            unpack8(lo[k], f0);
            unpack8(hi[k], f1);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (kNeighbour) {
                    float(&f)[8] = q < 4 ? f0 : f1;
                    const float x0 = f[2 * q & 7], x1 = f[(2 * q & 7) + 1];
                    f[2 * q & 7] = x0 * c[q] - x1 * s[q];
                    f[(2 * q & 7) + 1] = x1 * c[q] + x0 * s[q];
                } else {
                    const float x0 = f0[q], x1 = f1[q];
                    f0[q] = x0 * c[q] - x1 * s[q];
                    f1[q] = x1 * c[q] + x0 * s[q];
                }
            }
            *reinterpret_cast<uint4*>(out + h * a.out_head) = pack8(f0);
            *reinterpret_cast<uint4*>(out + h * a.out_head + second) = pack8(f1);
        }
    }
}

template <bool kNeighbour, int U>
cudaError_t launch(RopeArgs a, cudaStream_t stream) {
    a.groups = (a.heads + U - 1) / U;
    const int32_t per = a.groups * a.pieces;
    a.tokens = std::max(1, kThreads / per);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.total + a.tokens - 1) / a.tokens));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, rope_kernel<kNeighbour, U>, a);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace

cudaError_t launch_rope_table(int32_t rows, int32_t first, int32_t dim, double base, const dsa_rope_scaling* scaling,
                              float* cos_t, float* sin_t, cudaStream_t stream) {
    Turns t{};
    const int32_t pairs = dim / 2;
    const double pi = 3.14159265358979323846;
    double lo = 0, hi = 0;
    const bool yarn = scaling && scaling->original_ctx > 0;
    if (yarn) {
        // the pair that turns n times in the original context
        auto edge = [&](double n) { return dim * std::log(scaling->original_ctx / (n * 2 * pi)) / (2 * std::log(base)); };
        lo = std::max(std::floor(edge(scaling->beta_fast)), 0.0);
        hi = std::min(std::ceil(edge(scaling->beta_slow)), dim - 1.0);
    }
    for (int32_t i = 0; i < pairs; ++i) {
        double f = std::pow(base, -2.0 * i / dim);
        if (yarn) {
            const double part = std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
            f = f / scaling->factor * part + f * (1 - part);
        } else if (scaling) {
            f /= scaling->factor;
        }
        t.f[i] = (uint64_t)std::ldexp(f / (2 * pi), 64);     // f <= 1
    }
    const int64_t n = (int64_t)rows * (pairs / 4);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((n + kThreads - 1) / kThreads));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, rope_table_kernel, t, rows, first, pairs,
                                             scaling ? scaling->mscale : 1.f, cos_t, sin_t);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

cudaError_t launch_rope(int32_t total_q, int32_t heads, int32_t dim, const uint16_t* x, int64_t x_token, int64_t x_head,
                        const float* cos_t, const float* sin_t, int32_t table_rows, const int32_t* positions,
                        bool neighbour, bool inverse, uint16_t* out, int64_t out_token, int64_t out_head,
                        int32_t* status, cudaStream_t stream) {
    RopeArgs a{};
    a.total = total_q;
    a.heads = heads;
    a.dim = dim;
    a.table_rows = table_rows;
    a.x = x;
    a.x_token = x_token;
    a.x_head = x_head;
    a.cos_t = cos_t;
    a.sin_t = sin_t;
    a.positions = positions;
    a.out = out;
    a.out_token = out_token;
    a.out_head = out_head;
    a.pieces = dim / 16;
    a.sign = inverse ? -1.f : 1.f;
    a.status = status;
    // Few tokens: more threads in flight; many: fewer reads of the table.  Rows of 64
    // heads x 64 columns, one and four heads a thread: 64 tokens 1.5 and 2.2 us, 2,048 6.9
    // and 7.7, 4,864 (the border) 14.4 and 14.7, 9,728 28.7 and 27.7, 32,768 89.3 and 82.0.
    const bool few = (int64_t)total_q * heads * a.pieces < (int64_t)4 * 2048 * num_sms();
    if (neighbour) return few ? launch<true, 1>(a, stream) : launch<true, 4>(a, stream);
    return few ? launch<false, 1>(a, stream) : launch<false, 4>(a, stream);
}

}  // namespace dsa
