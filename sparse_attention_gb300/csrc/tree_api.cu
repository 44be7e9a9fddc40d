// tree_api.cu -- the extern "C" entry points of a step of drafted tokens over
// a cache (declared and documented in include/dsa.h): host-side argument
// checks and the workspace layout.
#include <algorithm>
#include <cmath>

#include "api_checks.h"

using namespace dsa;

namespace {

// The calls of a step run one after another in their stream, so their scratch
// overlaps behind the status header; each asks for its own.
size_t tables_ws(const dsa_batch* b) { return with_header(step_tables_bytes(b->batch)); }
size_t attention_ws(const dsa_batch* b) { return with_header(tree_mla_scratch_bytes(to_dev(b))); }

}  // namespace

extern "C" {

dsa_status dsa_tree_workspace_size(const dsa_batch* batch, size_t* bytes) {
    if (!bytes) return DSA_ERR_INVALID_ARG;
    if (!batch) {
        *bytes = with_header(0);
        return DSA_OK;
    }
    if (batch->batch < 1 || batch->batch > 65535 || batch->total_q < 0 || batch->max_q < 0 || batch->max_ctx < 0)
        return DSA_ERR_INVALID_ARG;
    *bytes = (std::max(tables_ws(batch), attention_ws(batch)) + 255) / 256 * 256;
    return DSA_OK;
}

dsa_status dsa_step_tables(const dsa_batch* batch, const dsa_pages* pages, const int32_t* n_new,
                           const int32_t* ctx_old, const int32_t* parent, const int32_t* n_pages_old,
                           int32_t* n_pages, const int32_t* free_pages, const int32_t* free_range,
                           int32_t* free_range_out, int32_t* slots, int32_t* positions, uint64_t* mask, void* ws,
                           size_t ws_bytes, void* stream) {
    dsa_status st = check(batch, pages);
    if (st != DSA_OK || (st = check_ws(ws, ws_bytes, tables_ws(batch))) != DSA_OK) return st;
    if (!given(n_new, 4) || !given(ctx_old, 4) || !aligned(parent, 4) || !aligned(mask, 8)) return DSA_ERR_INVALID_ARG;
    if (batch->total_q > 0 && (!given(slots, 4) || !given(positions, 4))) return DSA_ERR_INVALID_ARG;
    if (pages && (!given(n_pages_old, 4) || !given(n_pages, 4) || !given(free_pages, 4) || !given(free_range, 4) ||
                  !given(free_range_out, 4)))
        return DSA_ERR_INVALID_ARG;
    return cuda_status(launch_step_tables(to_dev(batch), to_dev(pages), n_new, ctx_old, parent, n_pages_old, n_pages,
                                          free_pages, free_range, free_range_out, slots, positions, mask,
                                          static_cast<int32_t*>(scratch_of(ws)), static_cast<int32_t*>(ws),
                                          static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_latent_append(int32_t total_q, const uint16_t* x, int64_t x_stride, const float* gamma, float eps,
                             const float* cos_t, const float* sin_t, int32_t table_rows, const int32_t* positions,
                             const int32_t* slots, int64_t cache_rows, uint16_t* kv, void* ws, size_t ws_bytes,
                             void* stream) {
    if (total_q < 0 || total_q >= (1 << 26)) return DSA_ERR_INVALID_ARG;
    if (check_ws(ws, ws_bytes, with_header(0)) != DSA_OK) return DSA_ERR_WORKSPACE;
    if (total_q == 0) return DSA_OK;
    if (x_stride < kDQK || x_stride % 8 != 0 || table_rows < 0 || cache_rows < 0) return DSA_ERR_INVALID_ARG;
    if (!given(x) || !given(gamma) || !given(cos_t) || !given(sin_t) || !given(positions, 4) || !given(slots, 4) ||
        !given(kv))
        return DSA_ERR_INVALID_ARG;
    if (!(eps > 0.f) || eps == INFINITY) return DSA_ERR_INVALID_ARG;
    return cuda_status(launch_latent_append(total_q, x, x_stride, gamma, eps, cos_t, sin_t, table_rows, positions,
                                            slots, cache_rows, kv, static_cast<int32_t*>(ws),
                                            static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_tree_mla_fwd(const dsa_batch* batch, const dsa_pages* pages, const uint16_t* q, const uint16_t* kv,
                            const uint64_t* mask, float sm_scale, uint16_t* out, float* lse, void* ws,
                            size_t ws_bytes, void* stream) {
    dsa_status st = check(batch, pages);
    if (st != DSA_OK) return st;
    if (batch->max_q > DSA_MAX_TREE) return DSA_ERR_UNSUPPORTED;
    if (batch->total_q >= (1 << 25)) return DSA_ERR_UNSUPPORTED;     // 64 query rows each, in int32 TMA coordinates
    if ((st = check_ws(ws, ws_bytes, attention_ws(batch))) != DSA_OK) return st;
    if (batch->total_q == 0 || batch->max_q == 0 || batch->max_ctx == 0) return DSA_OK;      // no row can be
    if (!given(q) || !given(kv) || !given(mask, 8) || !given(out) || !aligned(lse, 16)) return DSA_ERR_INVALID_ARG;
    if (!(sm_scale > 0.f) || sm_scale == INFINITY) return DSA_ERR_INVALID_ARG;
    return cuda_status(launch_tree_mla(to_dev(batch), to_dev(pages), q, kv, mask, sm_scale, out, lse, scratch_of(ws),
                                       static_cast<int32_t*>(ws), static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_tree_topk(const dsa_batch* batch, const float* scores, int64_t ld, const uint64_t* mask, int k,
                         int32_t* idx, void* ws, size_t ws_bytes, void* stream) {
    const dsa_status st = check(batch);
    if (st != DSA_OK) return st;
    if (k < 1 || k > kMaxTopk) return DSA_ERR_INVALID_ARG;
    if (batch->max_q > DSA_MAX_TREE) return DSA_ERR_UNSUPPORTED;
    if (check_ws(ws, ws_bytes, with_header(0)) != DSA_OK) return DSA_ERR_WORKSPACE;
    if (batch->total_q == 0 || batch->max_q == 0) return DSA_OK;
    if (!given(scores) || !given(mask, 8) || !given(idx)) return DSA_ERR_INVALID_ARG;
    if (ld < batch->max_ctx || ld % 4 != 0) return DSA_ERR_INVALID_ARG;
    return cuda_status(launch_tree_topk(to_dev(batch), scores, ld, mask, k, idx, static_cast<int32_t*>(ws),
                                        static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_tree_commit(const dsa_batch* batch, const dsa_pages* pages, const uint64_t* mask,
                           const int32_t* accepted, int32_t layers, int64_t cache_rows, uint16_t* kv, uint16_t* k_idx,
                           int32_t* ctx_new, void* ws, size_t ws_bytes, void* stream) {
    dsa_status st = check(batch, pages);
    if (st != DSA_OK || (st = check_ws(ws, ws_bytes, tables_ws(batch))) != DSA_OK) return st;
    if (layers < 1 || layers > 65535 || cache_rows < 0) return DSA_ERR_INVALID_ARG;
    const int64_t rows = pages ? (int64_t)pages->pool_pages * pages->page_size : batch->batch * batch->cache_stride;
    if (pages ? cache_rows != rows : cache_rows < rows) return DSA_ERR_INVALID_ARG;
    if (!given(accepted, 4) || !given(ctx_new, 4)) return DSA_ERR_INVALID_ARG;
    if (batch->total_q > 0 && !given(mask, 8)) return DSA_ERR_INVALID_ARG;      // no row: no node to accept
    if (!aligned(kv, 16) || !aligned(k_idx, 16)) return DSA_ERR_INVALID_ARG;
    return cuda_status(launch_tree_commit(to_dev(batch), to_dev(pages), mask, accepted, layers, cache_rows, kv, k_idx,
                                          ctx_new, static_cast<int32_t*>(scratch_of(ws)), static_cast<int32_t*>(ws),
                                          static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
