// prompt_api.cu -- the extern "C" entry points of rotary positions, of the
// expanded form of the latent attention and of shared prefixes (declared and
// documented in include/dsa.h): host-side argument checks and workspace sizes.
#include <algorithm>
#include <cmath>

#include "api_checks.h"
#include "prompt.h"

using namespace dsa;

namespace {

bool good_dim(int32_t dim) { return dim >= 16 && dim <= DSA_MAX_ROPE_DIM && dim % 16 == 0; }

constexpr int64_t kMaxStride = int64_t(1) << 36;
constexpr int32_t kMaxRopeHeads = 1 << 16;

// Bytes from a tensor's first element to behind its last.  Unsigned: 2^26 tokens and
// 2^16 heads at the largest strides span 2^63 + 2^53 bytes.
uint64_t extent(int32_t tokens, int64_t token, int32_t heads, int64_t head, int32_t dim) {
    return 2 * ((uint64_t)(tokens - 1) * (uint64_t)token + (uint64_t)(heads - 1) * (uint64_t)head + (uint64_t)dim);
}

// (addresses stay below 2^57, so the sums stay below 2^64)
bool overlap(const void* a, uint64_t a_bytes, const void* b, uint64_t b_bytes) {
    const uint64_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + b_bytes && y < x + a_bytes;
}

// The two calls of the expanded form run one after another in their stream, so
// their scratch overlaps behind the status header.
size_t prompt_ws(const dsa_batch* b) {
    return with_header(std::max(prompt_mla_scratch_bytes(to_dev(b)), mla_expand_scratch_bytes(to_dev(b))));
}

size_t prefix_ws(const dsa_batch* b, const dsa_groups* g) {
    return with_header(prefix_mla_scratch_bytes(to_dev(b), g->groups));
}

dsa_status check(const dsa_expanded* x) {
    if (!x || x->rows < 0 || !given(x->off, 4)) return DSA_ERR_INVALID_ARG;
    return x->rows == 0 || (given(x->kv) && given(x->k_pe)) ? DSA_OK : DSA_ERR_INVALID_ARG;
}

ExpandedDev to_dev(const dsa_expanded* x) { return ExpandedDev{x->rows, x->off, x->kv, x->k_pe}; }

}  // namespace

extern "C" {

dsa_status dsa_rope_table(int32_t rows, int32_t first, int32_t dim, double base, const dsa_rope_scaling* scaling,
                          float* cos_t, float* sin_t, void* stream) {
    if (rows < 0 || first < 0 || (int64_t)rows + first > (int64_t(1) << 31) || !good_dim(dim)) return DSA_ERR_INVALID_ARG;
    if (!(base >= 1.0) || !std::isfinite(base)) return DSA_ERR_INVALID_ARG;
    if (scaling) {
        if (!(scaling->factor >= 1.0) || !std::isfinite(scaling->factor) || scaling->original_ctx < 0 ||
            !positive(scaling->mscale))
            return DSA_ERR_INVALID_ARG;
        if (scaling->original_ctx > 0 &&
            (base == 1.0 || !positive(scaling->beta_fast) || !positive(scaling->beta_slow)))
            return DSA_ERR_INVALID_ARG;
    }
    if (rows == 0) return DSA_OK;
    if (!given(cos_t) || !given(sin_t)) return DSA_ERR_INVALID_ARG;
    const uint64_t bytes = (uint64_t)rows * (uint64_t)dim * 4;
    if (overlap(cos_t, bytes, sin_t, bytes)) return DSA_ERR_INVALID_ARG;
    return cuda_status(launch_rope_table(rows, first, dim, base, scaling, cos_t, sin_t,
                                         static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_rope(int32_t total_q, int32_t heads, int32_t dim, const uint16_t* x, int64_t x_token, int64_t x_head,
                    const float* cos_t, const float* sin_t, int32_t table_rows, const int32_t* positions,
                    int32_t flags, uint16_t* out, int64_t out_token, int64_t out_head, void* ws, size_t ws_bytes,
                    void* stream) {
    if (total_q < 0 || total_q >= (1 << 26) || heads < 1 || heads > kMaxRopeHeads || !good_dim(dim)) return DSA_ERR_INVALID_ARG;
    if (table_rows < 0 || (flags & ~(DSA_ROPE_NEIGHBOUR | DSA_ROPE_INVERSE))) return DSA_ERR_INVALID_ARG;
    if (check_ws(ws, ws_bytes, with_header(0)) != DSA_OK) return DSA_ERR_WORKSPACE;
    if (total_q == 0) return DSA_OK;
    if (!given(x) || !given(out) || !given(cos_t) || !given(sin_t) || !given(positions, 4)) return DSA_ERR_INVALID_ARG;
    for (int64_t s : {x_token, x_head, out_token, out_head})
        if (s < 0 || s % 8 != 0 || s > kMaxStride) return DSA_ERR_INVALID_ARG;
    // tokens of whole heads, or heads of whole tokens
    const bool by_token = (heads == 1 || out_head >= dim) &&
                          (total_q == 1 || out_token >= (heads - 1) * out_head + dim);
    const bool by_head = (total_q == 1 || out_token >= dim) &&
                         (heads == 1 || out_head >= (total_q - 1) * out_token + dim);
    if (!by_token && !by_head) return DSA_ERR_INVALID_ARG;
    const bool place = x == out && (total_q == 1 || x_token == out_token) && (heads == 1 || x_head == out_head);
    if (!place && overlap(x, extent(total_q, x_token, heads, x_head, dim), out,
                          extent(total_q, out_token, heads, out_head, dim)))
        return DSA_ERR_INVALID_ARG;
    return cuda_status(launch_rope(total_q, heads, dim, x, x_token, x_head, cos_t, sin_t, table_rows, positions,
                                   (flags & DSA_ROPE_NEIGHBOUR) != 0, (flags & DSA_ROPE_INVERSE) != 0, out, out_token,
                                   out_head, static_cast<int32_t*>(ws), static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_prompt_workspace_size(const dsa_batch* batch, size_t* bytes) {
    if (!bytes || !batch || batch->batch < 1 || batch->batch > 65535 || batch->total_q < 0 || batch->max_q < 0 ||
        batch->max_ctx < 0)
        return DSA_ERR_INVALID_ARG;
    *bytes = (prompt_ws(batch) + 255) / 256 * 256;
    return DSA_OK;
}

dsa_status dsa_mla_expand(const dsa_batch* batch, const dsa_pages* pages, const uint16_t* kv, const uint16_t* w_kv_b,
                          const int32_t* first, const dsa_expanded* expanded, void* ws, size_t ws_bytes,
                          void* stream) {
    dsa_status st = check(batch, pages);
    if (st != DSA_OK || (st = check(expanded)) != DSA_OK) return st;
    if (check_ws(ws, ws_bytes, prompt_ws(batch)) != DSA_OK) return DSA_ERR_WORKSPACE;
    if (batch->max_ctx == 0 || expanded->rows == 0) return DSA_OK;      // no row can be
    if (!given(kv) || !given(w_kv_b) || !aligned(first, 4)) return DSA_ERR_INVALID_ARG;
    return cuda_status(launch_mla_expand(to_dev(batch), to_dev(pages), kv, w_kv_b, first, to_dev(expanded),
                                         scratch_of(ws), static_cast<int32_t*>(ws),
                                         static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_prompt_mla_fwd(const dsa_batch* batch, const uint16_t* q, const dsa_expanded* expanded, float sm_scale,
                              uint16_t* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    dsa_status st = check(batch);
    if (st != DSA_OK || (st = check(expanded)) != DSA_OK) return st;
    if (check_ws(ws, ws_bytes, prompt_ws(batch)) != DSA_OK) return DSA_ERR_WORKSPACE;
    if (!positive(sm_scale)) return DSA_ERR_INVALID_ARG;
    if (batch->total_q == 0 || batch->max_q == 0 || batch->max_ctx == 0) return DSA_OK;
    // (without expanded rows the call only finds the sequences that have new ones)
    if (expanded->rows > 0 && (!given(q) || !given(out) || !aligned(lse, 16))) return DSA_ERR_INVALID_ARG;
    return cuda_status(launch_prompt_mla(to_dev(batch), q, to_dev(expanded), sm_scale, out, lse, scratch_of(ws),
                                         static_cast<int32_t*>(ws), static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_prefix_workspace_size(const dsa_batch* batch, const dsa_groups* groups, size_t* bytes) {
    if (!bytes || !batch || batch->batch < 1 || batch->batch > 65535 || batch->total_q < 0 || batch->max_q < 0 ||
        batch->max_ctx < 0 || !groups || groups->groups < 1 || groups->groups > batch->batch)
        return DSA_ERR_INVALID_ARG;
    *bytes = (prefix_ws(batch, groups) + 255) / 256 * 256;
    return DSA_OK;
}

dsa_status dsa_prefix_mla_fwd(const dsa_batch* batch, const dsa_groups* groups, const dsa_pages* pages,
                              const uint16_t* q, const uint16_t* kv, const uint64_t* mask, float sm_scale,
                              uint16_t* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    const dsa_status st = check(batch, pages);
    if (st != DSA_OK) return st;
    if (!groups || groups->groups < 1 || groups->groups > batch->batch || !given(groups->off, 4) ||
        !given(groups->shared, 4))
        return DSA_ERR_INVALID_ARG;
    if (batch->max_q > DSA_MAX_TREE) return DSA_ERR_UNSUPPORTED;
    if (batch->total_q >= (1 << 25)) return DSA_ERR_UNSUPPORTED;     // 64 query rows each, in int32 TMA coordinates
    if (check_ws(ws, ws_bytes, prefix_ws(batch, groups)) != DSA_OK) return DSA_ERR_WORKSPACE;
    if (!positive(sm_scale)) return DSA_ERR_INVALID_ARG;
    if (batch->total_q == 0 || batch->max_q == 0 || batch->max_ctx == 0) return DSA_OK;      // no row can be
    if (!given(q) || !given(kv) || !aligned(mask, 8) || !given(out) || !aligned(lse, 16)) return DSA_ERR_INVALID_ARG;
    return cuda_status(launch_prefix_mla(to_dev(batch), GroupsDev{groups->groups, groups->off, groups->shared},
                                         to_dev(pages), q, kv, mask, sm_scale, out, lse, scratch_of(ws),
                                         static_cast<int32_t*>(ws), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
