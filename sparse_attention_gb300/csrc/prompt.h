// prompt.h -- definitions of rotary positions.
#pragma once
#include "internal.h"
#include "tree.h"

namespace dsa {

cudaError_t launch_rope_table(int32_t rows, int32_t first, int32_t dim, double base, const dsa_rope_scaling* scaling,
                              float* cos_t, float* sin_t, cudaStream_t stream);
cudaError_t launch_rope(int32_t total_q, int32_t heads, int32_t dim, const uint16_t* x, int64_t x_token, int64_t x_head,
                        const float* cos_t, const float* sin_t, int32_t table_rows, const int32_t* positions,
                        bool neighbour, bool inverse, uint16_t* out, int64_t out_token, int64_t out_head,
                        int32_t* status, cudaStream_t stream);

}  // namespace dsa
