// tree_commit.cu -- the accepted path of a drafted tree moves behind the
// committed cache rows.
//
// The path is a set of bits j_0 < j_1 < ..; row c + j_i goes to c + i.  A CTA
// takes one sequence in one layer, a thread one 16-byte column of its rows
// (72 of the latent row, 16 of the index key) in path order, eight rows
// loaded at a time.  In place this is safe without any barrier: j_i >= i and
// the j are strictly increasing, so the rows that a batch of eight writes are
// never among those that later batches read, and a batch is read before it
// is written.  64 trees in 8 layers (10 MB moved): 3.8 us; 4 in one: 2.5 us,
// a launch and three round trips (lengths, mask, rows).
#include "internal.h"
#include "tree.h"

namespace dsa {
namespace {

constexpr int kThreads = 96;                       // 72 + 16 columns
constexpr int kKvCols = kDQK / 8, kIdxCols = kDIdx / 8;

struct Path {
    int32_t c, count;
    uint64_t bits;
    bool ok;
};

__device__ __forceinline__ Path path_of(const BatchDev& bd, const uint64_t* mask, const int32_t* accepted, int b,
                                        const SeqInfo& sq, int32_t* status) {
    Path p{sq.ctx - sq.nq, 0, 0u, true};
    const int32_t node = __ldg(accepted + b);
    if (node < -1 || node >= sq.nq) {
        latch_status(status, DSA_ERR_BAD_INDEX);
        p.ok = false;
    } else if (sq.nq > DSA_MAX_TREE) {
        latch_status(status, DSA_ERR_BAD_BATCH);
        p.ok = false;
    } else if (node >= 0) {
        p.bits = visible_bits(__ldg(reinterpret_cast<const unsigned long long*>(mask) + sq.q0 + node), node);
        p.count = __popcll(p.bits);
    }
    return p;
}

// write_len: this launch also writes ctx_new (it is not the ctx_len that the
// other CTAs still read).
__global__ void __launch_bounds__(kThreads)
    tree_commit_kernel(const BatchDev bd, const PagesDev pg, const uint64_t* __restrict__ mask,
                       const int32_t* __restrict__ accepted, int64_t cache_rows, uint16_t* kv, uint16_t* k_idx,
                       int32_t* ctx_new, bool write_len, int32_t* path_bad, int32_t* status) {
    __shared__ int32_t from[DSA_MAX_TREE], to[DSA_MAX_TREE];
    const int b = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x;
    SeqInfo sq;
    if (!load_seq(bd, b, status, sq)) return;
    Path p = path_of(bd, mask, accepted, b, sq, status);
    bool bad = false;
    if (tid < DSA_MAX_TREE && tid < sq.nq && p.ok && (p.bits >> tid) & 1u) {
        const int32_t i = __popcll(p.bits & ((1ull << tid) - 1u));
        from[i] = cache_row(bd, pg, b, p.c + tid);
        to[i] = cache_row(bd, pg, b, p.c + i);
        bad = from[i] < 0 || to[i] < 0 || from[i] >= cache_rows || to[i] >= cache_rows;
    }
    bad = __syncthreads_or(bad);
    if (bad) {
        if (tid == 0) latch_status(status, DSA_ERR_BAD_INDEX);
        p.count = 0;
    }
    if (layer == 0 && tid == 0) {
        if (write_len) ctx_new[b] = p.c + p.count;
        else path_bad[b] = bad ? 1 : 0;
    }
    uint4* base;
    int64_t pitch;
    if (tid < kKvCols) {
        if (!kv) return;
        pitch = kKvCols;
        base = reinterpret_cast<uint4*>(kv) + (int64_t)layer * cache_rows * pitch + tid;
    } else {
        if (tid >= kKvCols + kIdxCols || !k_idx) return;
        pitch = kIdxCols;
        base = reinterpret_cast<uint4*>(k_idx) + (int64_t)layer * cache_rows * pitch + (tid - kKvCols);
    }
    for (int32_t i0 = 0; i0 < p.count; i0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (i0 + u < p.count && from[i0 + u] != to[i0 + u]) v[u] = base[from[i0 + u] * pitch];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (i0 + u < p.count && from[i0 + u] != to[i0 + u]) base[to[i0 + u] * pitch] = v[u];
    }
}

// ctx_new when it is the ctx_len that the moves read.
__global__ void __launch_bounds__(128)
    tree_commit_lengths_kernel(const BatchDev bd, const uint64_t* __restrict__ mask,
                               const int32_t* __restrict__ accepted, const int32_t* __restrict__ path_bad,
                               int32_t* ctx_new, int32_t* status) {
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b >= bd.B) return;
    SeqInfo sq{bd.q_off[b], bd.q_off[b + 1] - bd.q_off[b], ctx_new[b]};
    if (sq.q0 < 0 || sq.q0 + sq.nq > bd.total_q || sq.nq < 0 || sq.nq > bd.max_q || sq.nq > sq.ctx ||
        sq.ctx > bd.max_ctx)
        return;                                    // latched by the moves
    const Path p = path_of(bd, mask, accepted, b, sq, status);
    ctx_new[b] = p.c + (path_bad[b] ? 0 : p.count);
}

}  // namespace

cudaError_t launch_tree_commit(const BatchDev& bd, const PagesDev& pg, const uint64_t* mask, const int32_t* accepted,
                               int32_t layers, int64_t cache_rows, uint16_t* kv, uint16_t* k_idx, int32_t* ctx_new,
                               int32_t* scratch, int32_t* status, cudaStream_t stream) {
    const bool separate = ctx_new == bd.ctx_len;
    tree_commit_kernel<<<dim3((unsigned)bd.B, (unsigned)layers), kThreads, 0, stream>>>(
        bd, pg, mask, accepted, cache_rows, kv, k_idx, ctx_new, !separate, scratch, status);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launches(1);
    if (!separate) return e;
    tree_commit_lengths_kernel<<<(unsigned)((bd.B + 127) / 128), 128, 0, stream>>>(bd, mask, accepted, scratch, ctx_new,
                                                                               status);
    e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace dsa
