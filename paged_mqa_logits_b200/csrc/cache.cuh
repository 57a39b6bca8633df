// Device pieces shared by the cache kernels (attention, append, pages).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "ptx.cuh"
#include "mqa_cache.h"

namespace mqa {

constexpr int kMaxBatch = 32768;  // of the attention and the page calls

// Where a kernel reports: the library's word (never NULL) and the caller's (may be).
struct StatusWords {
    uint32_t* lib;
    int32_t* caller;
    uint32_t flags;
};

__device__ __forceinline__ void report(const StatusWords& s, uint32_t bits) {
    atomicOr(s.lib, bits);
    if (s.caller != nullptr) atomicOr(reinterpret_cast<uint32_t*>(s.caller), bits);
}

// For what is clamped or skipped in every mode and named in validate mode only.
__device__ __forceinline__ void report_checked(const StatusWords& s, uint32_t bits) {
    if (s.flags & MQA_FLAG_VALIDATE) report(s, bits);
}

// A length, clamped to what the block table can hold.
__device__ __forceinline__ int clamp_len(const StatusWords& s, int len, int most) {
    if (len < 0 || len > most) {
        report_checked(s, MQA_STATUS_BAD_CONTEXT);
        len = len < 0 ? 0 : most;
    }
    return len;
}

}  // namespace mqa
