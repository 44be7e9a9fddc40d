// prompt.h -- definitions shared by the calls for prompts and shared prefixes:
// rotary positions, the expanded form of the latent attention, and attention
// behind a prefix that sequences share.
#pragma once
#include "internal.h"
#include "tree.h"

namespace dsa {

constexpr int kNope = DSA_NOPE_DIM;              // 192 key columns of a head's expanded row ..
constexpr int kHeadV = DSA_V_HEAD_DIM;           // .. and 256 value columns behind them
constexpr int kHeadQK = kNope + DSA_ROPE_DIM;    // 256
constexpr int kExpRow = DSA_KVB_ROWS;            // 448
constexpr int kExpRoom = DSA_EXPANDED_ROOM;      // a sequence's expanded rows begin at a multiple of this

// Device view of dsa_expanded.
struct ExpandedDev {
    int32_t rows;
    const int32_t* off;
    uint16_t* kv;
    uint16_t* k_pe;
};

// Where a sequence's expanded rows begin, whose room is lo .. hi; -1 (and a latched
// DSA_ERR_BAD_BATCH) if that is not aligned, leaves the buffers or is too small for ctx rows.
__device__ __forceinline__ int32_t expanded_at(const ExpandedDev& x, int32_t lo, int32_t hi, int32_t ctx,
                                               int32_t* status) {
    const int64_t need = ((int64_t)ctx + kExpRoom - 1) / kExpRoom * kExpRoom;
    if (lo >= 0 && lo % kExpRoom == 0 && hi <= x.rows && (int64_t)hi - lo >= need) return lo;
    latch_status(status, DSA_ERR_BAD_BATCH);
    return -1;
}

// The last b with start[b] <= x (start[0] = 0, ascending, n entries): of empty
// sequences that begin at one place the last, which is the one that holds x.
__device__ __forceinline__ int last_at_or_below(const int32_t* start, int n, int32_t x) {
    int lo = 0, hi = n;
    while (lo + 1 < hi) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Device view of dsa_groups.
struct GroupsDev {
    int32_t n;
    const int32_t *off, *shared;
};

// The sum of v over the threads before this one of a block of `warps` warps, and
// over all of it in `all`; `sums` has a place for each warp.
__device__ __forceinline__ int32_t block_sum_before(int32_t v, int warps, int32_t* sums, int32_t& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t n = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += n;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int32_t before = incl - v;
    all = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) before += sums[w];
        all += sums[w];
    }
    return before;
}

// CTA pairs of kernel `f` that can be resident at once on the current device,
// at most `most`.
int resident_pairs(const void* f, int threads, size_t smem, int most);

cudaError_t launch_rope_table(int32_t rows, int32_t first, int32_t dim, double base, const dsa_rope_scaling* scaling,
                              float* cos_t, float* sin_t, cudaStream_t stream);
cudaError_t launch_rope(int32_t total_q, int32_t heads, int32_t dim, const uint16_t* x, int64_t x_token, int64_t x_head,
                        const float* cos_t, const float* sin_t, int32_t table_rows, const int32_t* positions,
                        bool neighbour, bool inverse, uint16_t* out, int64_t out_token, int64_t out_head,
                        int32_t* status, cudaStream_t stream);

size_t mla_expand_scratch_bytes(const BatchDev& bd);
cudaError_t launch_mla_expand(const BatchDev& bd, const PagesDev& pg, const uint16_t* kv, const uint16_t* w_kvb,
                              const int32_t* first, const ExpandedDev& x, void* scratch, int32_t* status,
                              cudaStream_t stream);

size_t prompt_mla_scratch_bytes(const BatchDev& bd);
cudaError_t launch_prompt_mla(const BatchDev& bd, const uint16_t* q, const ExpandedDev& x, float sm_scale,
                              uint16_t* out, float* lse, void* scratch, int32_t* status, cudaStream_t stream);

// Few new rows over short contexts (prompt_rows.cu).
bool prompt_rows_suit(const BatchDev& bd);
cudaError_t launch_prompt_rows(const BatchDev& bd, const uint16_t* q, const ExpandedDev& x, float sm_scale,
                               uint16_t* out, float* lse, int32_t* status, cudaStream_t stream);

size_t prefix_mla_scratch_bytes(const BatchDev& bd, int32_t groups);
cudaError_t launch_prefix_mla(const BatchDev& bd, const GroupsDev& gr, const PagesDev& pg, const uint16_t* q,
                              const uint16_t* kv, const uint64_t* mask, float sm_scale, uint16_t* out, float* lse,
                              void* scratch, int32_t* status, cudaStream_t stream);

}  // namespace dsa
