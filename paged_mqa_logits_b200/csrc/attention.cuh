// Arguments and the split rule of the attention kernels (attention.cu).
#pragma once
#include <cuda_runtime.h>

#include "cache.cuh"

namespace mqa {

struct AttentionArgs {
    const void* q;
    const uint8_t* k;
    const uint8_t* v;
    const int32_t* block_table;
    const int32_t* context_lens;
    const int32_t* schedule;  // dense
    const int32_t* indices;   // selected tokens
    void* out;
    float* lse;               // may be NULL
    float* part_o;            // [slots][Hk][rows][D]
    float* part_ml;           // [slots][Hk][rows][4]: maximum, sum, sum of unrounded p
    int64_t q_sb, q_sn, q_sh; // strides of q in elements
    uint32_t page_bytes;      // of one cache: Hk heads
    StatusWords status;
    float scale_log2;         // softmax_scale * log2(e)
    int32_t batch, next_n, heads, kv_heads, group;
    int32_t rows;             // query rows of one work item and kv head: group * next_n, or group (selected)
    int32_t page_size, ps_shift, num_pages, max_pages;
    int32_t num_ctas;         // dense: S
    int32_t topk, splits;     // selected: list length, CTAs per list
};

// CTAs that share one list of `topk` tokens: enough for a CTA on every SM, at most
// one per 256 entries (8 of a CTA's warps, 32 tokens each).
inline int topk_splits(int64_t lists, int topk, int sms) {
    int64_t s = sms / (lists > 0 ? lists : 1);
    const int64_t most = (topk + 255) / 256;
    if (s > most) s = most;
    return s < 1 ? 1 : (int)s;
}

// Slots of partial results: dense, two per part of the schedule (the row it
// starts inside of, the row it ends inside of); selected, one per CTA.
inline int64_t attention_slots(const AttentionArgs& a) {
    if (a.topk == 0) return 2 * (int64_t)a.num_ctas;
    return a.splits > 1 ? (int64_t)a.batch * a.next_n * a.splits : 0;
}

// attention_wide.cu: the kernel for more than 16 query rows a kv head.
template <int D, typename T, bool kList>
cudaError_t launch_wide(int device, const AttentionArgs& a, void* stream, bool pdl);

cudaError_t launch_attention(int device, int head_dim, int dtype, const AttentionArgs& a,
                             void* stream, bool pdl);

}  // namespace mqa
