// tree.h -- definitions shared by the kernels of a step of drafted tokens.
#pragma once
#include "internal.h"

namespace dsa {

// Device view of dsa_pages; table == nullptr: contiguous caches.
struct PagesDev {
    int32_t shift = 0;          // log2 of the page size
    int32_t max_pages = 0, pool_pages = 0;
    const int32_t* table = nullptr;
};

// Cache row of position pos of sequence b; -1 for a block-table entry outside
// the pool.
__device__ __forceinline__ int32_t cache_row(const BatchDev& bd, const PagesDev& pg, int b, int32_t pos) {
    if (!pg.table) return (int32_t)(b * bd.stride + pos);
    const int32_t page = __ldg(pg.table + (int64_t)b * pg.max_pages + (pos >> pg.shift));
    if ((uint32_t)page >= (uint32_t)pg.pool_pages) return -1;
    return (page << pg.shift) + (pos & ((1 << pg.shift) - 1));
}

// The bits of a row's mask that count: new rows at or below its own index.
__device__ __forceinline__ uint64_t visible_bits(uint64_t mask, int32_t i) { return mask & (~0ull >> (63 - i)); }

size_t step_tables_bytes(int32_t batch);
cudaError_t launch_step_tables(const BatchDev& bd, const PagesDev& pg, const int32_t* n_new, const int32_t* ctx_old,
                               const int32_t* parent, const int32_t* held_old, int32_t* held,
                               const int32_t* free_pages, const int32_t* free_range, int32_t* free_out,
                               int32_t* slots, int32_t* positions, uint64_t* mask, int32_t* scratch, int32_t* status,
                               cudaStream_t stream);

cudaError_t launch_latent_append(int32_t total_q, const uint16_t* x, int64_t x_stride, const float* gamma, float eps,
                                 const float* cos_t, const float* sin_t, int32_t table_rows,
                                 const int32_t* positions, const int32_t* slots, int64_t cache_rows, uint16_t* kv,
                                 int32_t* status, cudaStream_t stream);

size_t tree_mla_scratch_bytes(const BatchDev& bd);
cudaError_t launch_tree_mla(const BatchDev& bd, const PagesDev& pg, const uint16_t* q, const uint16_t* kv,
                            const uint64_t* mask, float sm_scale, uint16_t* out, float* lse, void* scratch,
                            int32_t* status, cudaStream_t stream);

cudaError_t launch_tree_topk(const BatchDev& bd, const float* scores, int64_t ld, const uint64_t* mask, int k,
                             int32_t* idx, int32_t* status, cudaStream_t stream);

cudaError_t launch_tree_commit(const BatchDev& bd, const PagesDev& pg, const uint64_t* mask, const int32_t* accepted,
                               int32_t layers, int64_t cache_rows, uint16_t* kv, uint16_t* k_idx, int32_t* ctx_new,
                               int32_t* scratch, int32_t* status, cudaStream_t stream);

}  // namespace dsa
