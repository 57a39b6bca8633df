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
    int32_t num_ctas;         // dense: S, the parts of the schedule,
    int32_t deal;             // and the CTAs that they are dealt to
    int32_t topk, splits;     // selected: list length, CTAs per list,
    bool small;               // of 4 warps
};

// Selected: the CTAs that share one list of `topk` tokens, and if they are small (4
// warps and 8 or 16 query rows of a kv head, several to an SM).
// - More lists than SMs: one small CTA a list. An SM then always has one that computes
//   while others wait for their loads (300 lists of 2048, D = 64: 40 -> 28 us, 256 of
//   1000: 21 -> 16 us, 2192 of 43: 56 -> 15 us, against CTAs of 16 or 12 warps one after
//   the other).
// - With more than 16 query rows a kv head, lists of up to 128 tokens, a small CTA for
//   every 16 rows: each has one step to do, and the tile of attention_wide.cu only a
//   chain of waits (480 lists of 7, 25 rows: 27 -> 10 us; 300 of 128, 64 rows: 28 -> 21;
//   but 148 of 128, 128 rows: 11.5 there, 20 here).
// - Lists that one CTA does in a step or two are not split, which saves the joining
//   and its launch (20 lists of 512: 15.7 -> 13.5 us a call, 6.8 -> 7.0 on the GPU; 45 of
//   777, D = 64: 7.4 -> 6.5; but 16 of 1024, D = 128: 7.1 split, 9.2 whole).
// - Few lists: a small CTA for every 128 tokens, if each can have an SM (8 lists of 2048:
//   8.2 -> 7.1 us).
// - In between, large CTAs, one an SM, with 256 tokens or more (128 lists of 2048: 21 us;
//   28 with 4 small ones).
// Where lists are split, all parts together are no more than the SMs: so much workspace
// serves any number of lists.
struct ListSplit { int splits; bool small; };
inline ListSplit split_list(int64_t lists, int topk, int rows, int head_dim, int sms) {
    const bool narrow = rows <= 16;
    if (narrow && (lists > sms || topk <= 128)) return {1, true};
    if (topk <= 128 && (rows <= 64 || lists * ((rows + 15) / 16) <= 3 * sms)) return {1, true};
    if (topk <= (narrow && head_dim == 64 ? 1024 : 512)) return {1, false};
    const int64_t small = (topk + 127) / 128, large = (topk + 255) / 256;
    if (narrow && lists * small <= sms) return {(int)small, true};
    int64_t s = sms / (lists > 0 ? lists : 1);
    if (s > large) s = large;
    return {s < 1 ? 1 : (int)s, false};
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
