// Host-side helpers shared by the C entry points (defined in api.cu).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "mqa_logits.h"

namespace mqa {

// Record the message of a failed call on this host thread and return `code`.
int fail(int code, const char* fmt, ...);
int cuda_fail(cudaError_t e, const char* what);

// Compute capability 10.0 check of the current device; also gives its index and
// its copy of the library's status word.
int check_arch(int* device_out, uint32_t** lib_status = nullptr);

bool env_flag(const char* name);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }

constexpr int kMaxCtas = 4096;  // of a schedule

// Raises a kernel's dynamic shared memory limit to `smem` on the current device
// (asked of the runtime only once per device and kernel: `done` is the caller's). Every call
// for a kernel gives the same `smem`, so that calls on several host threads agree.
template <typename Kernel>
inline cudaError_t allow_smem(Kernel kernel, int device, uint32_t smem, uint32_t (&done)[64]) {
    if (device < 0 || device >= 64 || done[device] < smem) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        if (device >= 0 && device < 64) done[device] = smem;
    }
    return cudaSuccess;
}

// Launch with programmatic dependent launch: the kernel may start while the
// previous one in the stream drains, and waits for it in griddep_wait().
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, uint32_t smem,
                              void* stream, bool pdl, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace mqa
