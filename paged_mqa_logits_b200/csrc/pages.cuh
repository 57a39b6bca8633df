// Arguments of the page kernels (pages.cu).
#pragma once
#include <cuda_runtime.h>

#include "cache.cuh"

namespace mqa {

struct PagesArgs {
    StatusWords status;
    int32_t batch, out_batch, max_pages, num_pages, page_size, ps_shift;
};

struct CopyArgs {
    StatusWords status;
    void* cache[MQA_PAGES_MAX_CACHES];
    uint32_t chunks[MQA_PAGES_MAX_CACHES];  // 16-byte pieces of a page
    const int32_t* src;
    const int32_t* dst;
    const int32_t* count;  // may be NULL
    int32_t n, num_caches, num_pages;
};

cudaError_t launch_fork(const int32_t* table, const int32_t* lens, const int32_t* parents,
                        int32_t* refs, int32_t* out_table, int32_t* out_lens, const PagesArgs& a,
                        void* stream, bool pdl);
cudaError_t launch_resize(int device, int32_t* table, int32_t* lens, const int32_t* new_lens,
                          int32_t* refs, int32_t* src, int32_t* dst, const PagesArgs& a,
                          void* stream, bool pdl);
cudaError_t launch_compact(int32_t* table, const int32_t* lens, int32_t* refs, int32_t* src,
                           int32_t* dst, int32_t* count, int32_t* map, const PagesArgs& a,
                           void* stream, bool pdl);
cudaError_t launch_copy(const CopyArgs& a, void* stream, bool pdl);

}  // namespace mqa
