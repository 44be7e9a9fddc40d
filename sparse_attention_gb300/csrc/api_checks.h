// api_checks.h -- host-side argument checks that the extern "C" entry points
// of the drafted step, of prompts and of shared prefixes have in common.
#pragma once
#include <cmath>

#include "internal.h"
#include "tree.h"

namespace dsa {

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool given(const void* p, unsigned n = 16) { return p && aligned(p, n); }

// The batch alone, for a call that touches no cache.
inline dsa_status check(const dsa_batch* b) {
    if (!b || b->batch < 1 || b->batch > 65535 || b->total_q < 0 || b->max_q < 0 || b->max_ctx < 0)
        return DSA_ERR_INVALID_ARG;
    if (b->cache_stride < b->max_ctx || !given(b->q_off, 4) || !given(b->ctx_len, 4)) return DSA_ERR_INVALID_ARG;
    return b->max_q > (1 << 19) || b->total_q >= (1 << 26) ? DSA_ERR_UNSUPPORTED : DSA_OK;
}

// The batch with its caches: contiguous, or paged (then the cache stride only
// bounds max_ctx).
inline dsa_status check(const dsa_batch* b, const dsa_pages* p) {
    const dsa_status st = check(b);
    if (st != DSA_OK) return st;
    if (!p) return b->cache_stride < (int64_t(1) << 31) / b->batch ? DSA_OK : DSA_ERR_UNSUPPORTED;
    if (p->page_size < 16 || p->page_size > 1024 || (p->page_size & (p->page_size - 1)) != 0) return DSA_ERR_INVALID_ARG;
    if (p->pool_pages < 1 || p->max_pages < 1 || (int64_t)p->max_pages * p->page_size < b->max_ctx ||
        !given(p->block_table, 4))
        return DSA_ERR_INVALID_ARG;
    return (int64_t)p->pool_pages * p->page_size < (int64_t(1) << 31) ? DSA_OK : DSA_ERR_UNSUPPORTED;
}

inline BatchDev to_dev(const dsa_batch* b) {
    return BatchDev{b->batch, b->total_q, b->max_q, b->max_ctx, b->cache_stride, b->q_off, b->ctx_len};
}

inline PagesDev to_dev(const dsa_pages* p) {
    PagesDev d;
    if (!p) return d;
    while ((1 << d.shift) < p->page_size) ++d.shift;
    d.max_pages = p->max_pages;
    d.pool_pages = p->pool_pages;
    d.table = p->block_table;
    return d;
}

inline size_t with_header(size_t scratch) { return kWsHeaderBytes + scratch; }

inline dsa_status check_ws(const void* ws, size_t bytes, size_t needed) {
    return given(ws) && bytes >= needed ? DSA_OK : DSA_ERR_WORKSPACE;
}

inline void* scratch_of(void* ws) { return static_cast<uint8_t*>(ws) + kWsHeaderBytes; }

inline bool positive(float x) { return x > 0.f && x < INFINITY; }

}  // namespace dsa
