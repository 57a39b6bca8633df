// Quantising appends: new tokens of every row into the FP8 and FP4 paged caches.
//
// One thread quantises 16 consecutive elements (an FP4 scale block; an FP8
// token's 2 to 8 threads share their maximum by shuffles), so a token's bytes
// are read once in 16-byte loads and written once in 8- or 16-byte stores.
// Bound by memory: 48 thousand tokens of 8 heads, K and V, D = 128, with the values
// (449 MB) take 83 us, 0.84 of the copy rate; 127 thousand FP8 keys (82 MB) 16 us, 0.81.
// One token each of 128 rows takes 2.7 us, a launch.
#include <cuda_runtime.h>

#include "append.cuh"
#include "host.cuh"

namespace mqa {
namespace {

constexpr int kThreads = 256;

// 16 elements of type T (two 16-byte loads) as fp32, exactly.
template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&x)[16]) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    const uint4 b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&v)[16]) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// Two fp32 values as e4m3 (low byte = a), to nearest even, at most 448.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Eight fp32 values as packed e2m1 codes (value 0 in the lowest nibble), to
// nearest even, at most 6.
__device__ __forceinline__ uint32_t to_e2m1x8(const float* v) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    const uint32_t mag = r & 0x77777777u;  // a zero keeps no sign: bit 3 of mag + 7 is set for mag >= 1
    return mag | (r & (mag + 0x77777777u) & 0x88888888u);
}

__device__ __forceinline__ void from_e2m1x8(uint32_t w, float* v) {
    uint32_t c[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3]) : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&c[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// Page and slot of new token t (page -1: it has none and is not written).
struct Place {
    int page, slot;
};

__device__ __forceinline__ Place place_of(const AppendArgs& a, int t) {
    int b, left;  // left: the tokens of the row from t on
    if (a.row_offsets != nullptr) {
        int lo = -1, hi = a.batch;  // the last row that begins at or before t (-1: none does)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (__ldg(a.row_offsets + mid) <= t) lo = mid; else hi = mid - 1;
        }
        b = lo;
        if (b < 0 || b >= a.batch) return {-1, 0};
        left = __ldg(a.row_offsets + b + 1) - t;
        if (left <= 0) return {-1, 0};
    } else {
        b = t / a.per_row;
        left = (b + 1) * a.per_row - t;
    }
    const int64_t pos = (int64_t)__ldg(a.context_lens + b) - left;
    if (pos < 0 || pos >= (int64_t)a.max_pages * a.page_size) {
        report_checked(a.status, MQA_STATUS_BAD_CONTEXT);
        return {-1, 0};
    }
    const int page = __ldg(a.block_table + (int64_t)b * a.max_pages + (pos >> a.ps_shift));
    if (page < 0 || page >= a.num_pages) {
        report_checked(a.status, MQA_STATUS_BAD_PAGE);
        return {-1, 0};
    }
    return {page, (int)(pos & (a.page_size - 1))};
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) append_fp4_kernel(AppendArgs a) {
    constexpr int kBlocks = D / 16;
    ptx::griddep_wait();
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t blk = i % kBlocks, th = i / kBlocks;
    const uint32_t t = th / a.heads, h = th - t * a.heads;
    if (t >= (uint32_t)a.num_tokens) return;
    const AppendTensor& x = a.x[blockIdx.y];
    float v[16];
    load16(static_cast<const T*>(x.tokens) + t * x.stride_t + h * x.stride_h + blk * 16, v);
    const Place p = place_of(a, (int)t);
    if (p.page < 0) return;
    float most = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) most = fmaxf(most, fabsf(v[k]));
    // 6 m has at most 7 significant bits for every midpoint m of e4m3, so for
    // bf16 and f16 inputs rounding the quotient to fp32 first never crosses one
    uint32_t sc = to_e4m3x2(__fdiv_rn(most, 6.f), 0.f) & 0xffu;
    if (sc == 0) sc = 1;  // 2^-9
    const float s = from_e4m3x2(sc).x;
    // x / s by a product with 1 / s, which is off by less than 2^-22 of it, then rounded
    // to 17 bits: x has at most 11 and s times a midpoint of e2m1 at most 7, so a
    // quotient that is no midpoint lies 2^-11 of it or more away from each, and one
    // that is becomes it again. (16 divisions instead: 97 us for 82, 0.72 of the copy
    // rate for 0.85.)
    const float inv = __fdiv_rn(1.f, s);
#pragma unroll
    for (int k = 0; k < 16; ++k)
        v[k] = __uint_as_float((__float_as_uint(v[k] * inv) + 0x40u) & 0xffffff80u);
    const uint2 code = make_uint2(to_e2m1x8(v), to_e2m1x8(v + 8));
    const int64_t head_bytes = (int64_t)a.page_size * (D / 2 + D / 16);
    uint8_t* block = static_cast<uint8_t*>(x.cache) + ((int64_t)p.page * a.heads + h) * head_bytes;
    *reinterpret_cast<uint2*>(block + p.slot * (D / 2) + blk * 8) = code;
    block[a.page_size * (D / 2) + p.slot * kBlocks + blk] = (uint8_t)sc;
    if (x.values != nullptr) {
        from_e2m1x8(code.x, v);
        from_e2m1x8(code.y, v + 8);
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] *= s;
        store16(static_cast<T*>(x.values) + (int64_t)th * D + blk * 16, v);
    }
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) append_fp8_kernel(AppendArgs a) {
    constexpr int kBlocks = D / 16;
    ptx::griddep_wait();
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t blk = i % kBlocks, t = i / kBlocks;
    const bool inside = t < (uint32_t)a.num_tokens;
    const AppendTensor& x = a.x[0];
    float v[16] = {};
    if (inside) load16(static_cast<const T*>(x.tokens) + t * x.stride_t + blk * 16, v);
    float most = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) most = fmaxf(most, fabsf(v[k]));
#pragma unroll
    for (int o = kBlocks / 2; o > 0; o >>= 1)
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (!inside) return;
    const Place p = place_of(a, (int)t);
    if (p.page < 0) return;
    // 448 = 1.75 * 2^8: the least power of two that is not below most / 448
    const uint32_t bits = __float_as_uint(most);
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = most > 0.f ? max(e, -126) : 0;
    const float s = __uint_as_float((uint32_t)(127 + e) << 23);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        w[k] = to_e4m3x2(v[4 * k] * inv, v[4 * k + 1] * inv) |
               to_e4m3x2(v[4 * k + 2] * inv, v[4 * k + 3] * inv) << 16;
    uint8_t* page = static_cast<uint8_t*>(x.cache) + (int64_t)p.page * a.page_size * (D + 4);
    *reinterpret_cast<uint4*>(page + p.slot * D + blk * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    if (blk == 0) *reinterpret_cast<float*>(page + a.page_size * D + p.slot * 4) = s;
    if (x.values != nullptr) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 lo = from_e4m3x2(w[k] & 0xffffu), hi = from_e4m3x2(w[k] >> 16);
            v[4 * k] = lo.x * s;
            v[4 * k + 1] = lo.y * s;
            v[4 * k + 2] = hi.x * s;
            v[4 * k + 3] = hi.y * s;
        }
        store16(static_cast<T*>(x.values) + (int64_t)t * D + blk * 16, v);
    }
}

template <int D, typename T>
cudaError_t launch_as(bool fp8, const AppendArgs& a, int tensors, void* stream, bool pdl) {
    const uint32_t threads = (uint32_t)a.num_tokens * a.heads * (D / 16);
    const dim3 grid((threads + kThreads - 1) / kThreads, tensors);
    if constexpr (D == 32) {
        return launch_pdl(append_fp8_kernel<D, T>, grid, dim3(kThreads), 0, stream, pdl, a);
    } else {
        return fp8 ? launch_pdl(append_fp8_kernel<D, T>, grid, dim3(kThreads), 0, stream, pdl, a)
                   : launch_pdl(append_fp4_kernel<D, T>, grid, dim3(kThreads), 0, stream, pdl, a);
    }
}

}  // namespace

cudaError_t launch_append(bool fp8, int head_dim, int dtype, const AppendArgs& a, int tensors,
                          void* stream, bool pdl) {
    const bool bf = dtype == MQA_DTYPE_BF16;
    switch (head_dim) {
        case 32: return bf ? launch_as<32, __nv_bfloat16>(true, a, tensors, stream, pdl)
                           : launch_as<32, __half>(true, a, tensors, stream, pdl);
        case 64: return bf ? launch_as<64, __nv_bfloat16>(fp8, a, tensors, stream, pdl)
                           : launch_as<64, __half>(fp8, a, tensors, stream, pdl);
        default: return bf ? launch_as<128, __nv_bfloat16>(fp8, a, tensors, stream, pdl)
                           : launch_as<128, __half>(fp8, a, tensors, stream, pdl);
    }
}

}  // namespace mqa
