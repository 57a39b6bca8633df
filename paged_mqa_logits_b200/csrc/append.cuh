// Arguments of the append kernels (append.cu).
#pragma once
#include <cuda_runtime.h>

#include <type_traits>

#include "cache.cuh"

namespace mqa {

struct AppendTensor {
    const void* tokens;
    void* cache;
    void* values;  // may be NULL
    int64_t stride_t, stride_h;
};

struct AppendArgs {
    AppendTensor x[2];
    const int32_t* block_table;
    const int32_t* context_lens;
    const int32_t* row_offsets;  // NULL: per_row tokens a row
    StatusWords status;
    int32_t batch, num_tokens, per_row, heads, page_size, ps_shift, num_pages, max_pages;
};

cudaError_t launch_append(bool fp8, int head_dim, int dtype, const AppendArgs& a, int tensors,
                          void* stream, bool pdl);

}  // namespace mqa
