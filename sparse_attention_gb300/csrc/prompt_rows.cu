// prompt_rows.cu -- causal attention over expanded rows for calls of few new
// rows over short contexts (a few tokens appended to each of many short
// sequences), on the FMA pipes.
//
// There the tensor kernel's time is an item's way through its pipeline, 1.4 us for
// each 76 of the 64 heads x sequences, whatever the rows are, and 9 us for the first.  Here a warp takes a
// head and four new rows of a sequence: a lane holds 8 of a key's 256 columns
// (512 bytes a key, one load), and 8 of the value's; four keys at a time are
// loaded, their 16 dot products summed over the warp, and folded into the four
// rows' running maxima, sums and results.  Everything is fp32 but the inputs and the
// rounding of the result.  Some 30 instructions a (row, key) pair and warp, and
// keys in turn: taken while the bounds leave at most 64 keys and 512 pairs (rows x
// length) a sequence.  There it is the faster one (32 sequences of 1 to 4 new
// rows behind 2 38 -> 8 us, 25 x 8 behind 5 33 -> 16, 15 x 20 25 -> 19; one of 7 10 ->
// 6); beyond, at 1,024 pairs, it is not (32 x 32 45 -> 72, 16 x 16 behind 48 27 ->
// 55, 32 x 1 behind 1,000 288 -> 513).  The bounds decide, not the lengths: under a captured
// call's 128 new rows of 4,096 the 32 x 1-4 take 39 us, under 512 of 4,096 78.
#include "internal.h"
#include "prompt.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kWarps = 4, kRows = 4, kKeys = 4;

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(w[k] << 16);
        f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
}

// Blocks (four heads, sequence, four rows).
__global__ void __launch_bounds__(32 * kWarps)
    prompt_rows_kernel(const BatchDev bd, const ExpandedDev x, const uint16_t* __restrict__ q, float scale_log2,
                       uint16_t* __restrict__ out, float* __restrict__ lse, int32_t* status) {
    const int lane = threadIdx.x & 31, head = (int)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int b = (int)blockIdx.y, i0 = (int)blockIdx.z * kRows;
    pdl_launch_dependents();
    pdl_wait();
    SeqInfo s;
    const int32_t lo = __ldg(x.off + b), hi = __ldg(x.off + b + 1);      // with the lengths, not behind them
    if (!load_seq(bd, b, status, s) || s.nq <= i0) return;
    const int32_t at = expanded_at(x, lo, hi, s.ctx, status);
    if (at < 0) return;
    const int32_t rows = min(kRows, s.nq - i0), pos = s.ctx - s.nq + i0;     // of the first row
    // lanes 0 .. 23 hold a key's own columns, 24 .. 31 the shared ones
    const bool pe = lane >= kNope / 8;
    const uint16_t* const k0 = pe ? x.k_pe + (int64_t)at * DSA_ROPE_DIM + 8 * (lane - kNope / 8)
                                  : x.kv + ((int64_t)at * kH + head) * kExpRow + 8 * lane;
    const uint16_t* const v0 = x.kv + ((int64_t)at * kH + head) * kExpRow + kNope + 8 * lane;
    constexpr int64_t kPitch = (int64_t)kH * kExpRow;
    const int64_t k_pitch = pe ? DSA_ROPE_DIM : kPitch;
    float qf[kRows][8], acc[kRows][8], m[kRows], l[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < rows) v = __ldg(reinterpret_cast<const uint4*>(q + ((int64_t)(s.q0 + i0 + r) * kH + head) * kHeadQK + 8 * lane));
        unpack8(v, qf[r]);
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int d = 0; d < 8; ++d) acc[r][d] = 0.f;
    }
    const int32_t seen = pos + rows;             // keys that the last row sees
#pragma unroll 1
    for (int32_t j0 = 0; j0 < seen; j0 += kKeys) {
        uint4 kr[kKeys], vr[kKeys];
#pragma unroll
        for (int j = 0; j < kKeys; ++j) {
            // (a key behind the last is the last once more, and masked)
            const int64_t row = min(j0 + j, seen - 1);
            kr[j] = *reinterpret_cast<const uint4*>(k0 + row * k_pitch);
            vr[j] = *reinterpret_cast<const uint4*>(v0 + row * kPitch);
        }
        float z[kRows][kKeys];
#pragma unroll
        for (int j = 0; j < kKeys; ++j) {
            float kf[8];
            unpack8(kr[j], kf);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                float sum = 0.f;
#pragma unroll
                for (int d = 0; d < 8; ++d) sum = fmaf(qf[r][d], kf[d], sum);
                z[r][j] = sum;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int j = 0; j < kKeys; ++j)
#pragma unroll
                for (int r = 0; r < kRows; ++r) z[r][j] += __shfl_xor_sync(0xffffffffu, z[r][j], o);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            float mx = m[r];
#pragma unroll
            for (int j = 0; j < kKeys; ++j) {
                z[r][j] = j0 + j > pos + r ? -INFINITY : z[r][j] * scale_log2;
                mx = fmaxf(mx, z[r][j]);
            }
            const float off = mx == -INFINITY ? 0.f : mx, f = ex2_approx(m[r] - off);
            m[r] = mx;
            l[r] *= f;
#pragma unroll
            for (int j = 0; j < kKeys; ++j) {
                z[r][j] = ex2_approx(z[r][j] - off);
                l[r] += z[r][j];
            }
#pragma unroll
            for (int d = 0; d < 8; ++d) acc[r][d] *= f;
        }
#pragma unroll
        for (int j = 0; j < kKeys; ++j) {
            float vf[8];
            unpack8(vr[j], vf);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                // 0 times a value that the row does not see must not be NaN
                if (j0 + j > pos + r) continue;
#pragma unroll
                for (int d = 0; d < 8; ++d) acc[r][d] = fmaf(z[r][j], vf[d], acc[r][d]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (r >= rows) break;
        // (l > 0 but where every score is -inf: NaN, as of the formula)
        const float inv = 1.f / l[r];
        const int64_t row = (int64_t)(s.q0 + i0 + r) * kH + head;
        reinterpret_cast<uint4*>(out + row * kHeadV)[lane] =
            make_uint4(pack_bf16x2(acc[r][0] * inv, acc[r][1] * inv), pack_bf16x2(acc[r][2] * inv, acc[r][3] * inv),
                       pack_bf16x2(acc[r][4] * inv, acc[r][5] * inv), pack_bf16x2(acc[r][6] * inv, acc[r][7] * inv));
        if (lse && lane == 0) lse[row] = (m[r] + log2f(l[r])) * kLn2;
    }
}

}  // namespace

bool prompt_rows_suit(const BatchDev& bd) { return bd.max_ctx <= 64 && bd.max_q * bd.max_ctx <= 512; }

cudaError_t launch_prompt_rows(const BatchDev& bd, const uint16_t* q, const ExpandedDev& x, float sm_scale,
                               uint16_t* out, float* lse, int32_t* status, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    // (without expanded rows a sequence's first block says all)
    cfg.gridDim = x.rows == 0 ? dim3(1, (unsigned)bd.B, 1)
                              : dim3(kH / kWarps, (unsigned)bd.B, (unsigned)((bd.max_q + kRows - 1) / kRows));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, prompt_rows_kernel, bd, x, q, sm_scale * kLog2e, out, lse, status);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace dsa
