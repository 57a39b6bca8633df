// Attention over the FP4 cache for many query rows a kv head (33 to 128): both
// products on the 5th-generation tensor core.
//
// A tile is 128 tokens. S = Q K^T (M = 128 query rows, N = 128 tokens) with Q in
// TMEM and K, dequantised to f16, in shared memory; P = 2^(S - m) goes back to TMEM
// over S, and O += P V with P as the A operand from TMEM and V in shared memory
// (tokens are the contraction, so V is the MN-major operand and needs no
// transpose). Rows are TMEM lanes, so maxima and sums of a row need no exchange but
// the one between the two warps that share a row's columns.
//
// Warps: 0-7 softmax (warp w: rows 32 (w % 4).., columns 64 (w / 4)..), 8-11
// dequantise (32 tokens of each tile, through a ring of asynchronous copies of
// their own), 12 issues the MMAs. S, K and V have two buffers each; S of the next
// tile is issued ahead of the current tile's O.
//
// m is raised, and O rescaled, only when a score exceeds it by kSlack (see
// attention.cu). All waits are bounded: on a timeout the status word gets
// MQA_STATUS_TIMEOUT and every role leaves.
#include "attention_walk.cuh"
#include "host.cuh"

namespace mqa {
namespace {

constexpr int kTokens = 128;       // of a tile
constexpr int kSoftmaxWarps = 8;
constexpr int kDequantWarps = 4;
constexpr int kMmaWarp = kSoftmaxWarps + kDequantWarps;
constexpr int kWideThreads = 32 * (kMmaWarp + 1);
constexpr uint64_t kTimeoutNs = 2000000000ull;
// TMEM columns: two S buffers (P over their first halves), O, Q.
constexpr int kColS = 0, kColO = 256, kColQ = 384, kColumns = 512;

template <int D>
struct Wide {
    static constexpr int kRow = D / 2, kScales = D / 16;
    static constexpr int kSlot = 2 * kSpan * (kRow + kScales);
    static constexpr int kStages = 4;
    static constexpr int kBuf = kTokens * D * 2;  // a tile of K or V: [D / 64][128 tokens][64] f16, 128-byte swizzle
    static constexpr int kK = 0, kV = 2 * kBuf, kRing = 4 * kBuf;
    static constexpr int kExch = kRing + kDequantWarps * kStages * kSlot;  // [2][2][128] fp32
    static constexpr int kBars = kExch + 2 * 2 * 128 * 4;
    static constexpr int kSmem = kBars + 256 + 1024;  // slack for aligning the base
    static_assert(kSmem <= 232448, "more shared memory than a CTA can have");
};

struct Bars {
    uint64_t k_full[2], v_full[2];  // the dequantising warps arrive
    uint64_t s_full[2];             // S computed (and its K buffer free)
    uint64_t p_full[2];             // the softmax warps arrive
    uint64_t pv_done[2];            // O updated (S and V buffers free)
    uint64_t q_full;                // the softmax warps arrive: a row's Q is in TMEM
    uint64_t pair[4];               // the two warps of a row quarter
    uint64_t drain;
    int32_t abort;
    uint32_t tmem;
};
static_assert(sizeof(Bars) <= 256, "barriers");

// Waits for phase `parity`, taken by lane 0 for the warp. False: give up.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, Bars* bars,
                                           const StatusWords& st, int lane) {
    bool ok = true;
    if (lane == 0 && !ptx::mbar_try_wait(bar, parity)) {
        const uint64_t t0 = ptx::globaltimer();
        volatile int32_t* abort = &bars->abort;
        while (!ptx::mbar_try_wait_sleep(bar, parity, kWaitSliceNs)) {
            if (*abort) {
                ok = false;
                break;
            }
            if (ptx::globaltimer() - t0 > kTimeoutNs) {
                report(st, MQA_STATUS_TIMEOUT);
                *abort = 1;
                ok = false;
                break;
            }
        }
    }
    return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

__device__ __forceinline__ void fence_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// 64 or 16 consecutive columns of this thread's TMEM lane, waited for.
__device__ __forceinline__ void tmem_read64(uint32_t taddr, float (&v)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19,"
        "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37,"
        "%38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55,"
        "%56, %57, %58, %59, %60, %61, %62, %63}"
        ", [%64];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]),
          "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]),
          "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]),
          "=f"(v[29]), "=f"(v[30]), "=f"(v[31]), "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]),
          "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]), "=f"(v[40]), "=f"(v[41]), "=f"(v[42]),
          "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]), "=f"(v[48]), "=f"(v[49]),
          "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]), "=f"(v[56]),
          "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63])
        : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_read16(uint32_t taddr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}"
        ", [%16];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr) : "memory");
}

__device__ __forceinline__ int tiles_of(const Walk& w) { return (w.t1 - w.t0 + kTokens - 1) / kTokens; }

// This lane's token (`row` of the tile) from its ring slot's codes and scales to f16.
template <int D>
__device__ __forceinline__ void dequant_row(uint32_t codes, uint32_t scales, uint32_t tile, int lane, int row) {
    uint32_t sc[D / 64];
    if constexpr (D == 128) {
        const uint2 v = lds64(scales + lane * 8);
        sc[0] = v.x;
        sc[1] = v.y;
    } else {
        sc[0] = lds32(scales + lane * 4);
    }
    const uint32_t line = tile + row * 128;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
        const uint4 v = lds128(codes + tile_at<D>(lane, j * 16));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        const uint32_t h = e4m3x2_to_f16(sc[j / 2] >> ((j & 1) * 16));
        const uint32_t s[2] = {__byte_perm(h, h, 0x1010), __byte_perm(h, h, 0x3232)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t f[4];
            e2m1_to_f16(w[i], f);
            const int u = 4 * j + i;  // 16-byte unit of the row
            sts128(line + (u >> 3) * (kTokens * 128) + (((u & 7) ^ (row & 7)) << 4),
                   mul_f16x2(f[0], s[i / 2]), mul_f16x2(f[1], s[i / 2]), mul_f16x2(f[2], s[i / 2]),
                   mul_f16x2(f[3], s[i / 2]));
        }
    }
}

template <int D, typename T, bool kList>
__global__ void __launch_bounds__(kWideThreads, 1) attention_wide_kernel(const AttentionArgs a) {
    using W = Wide<D>;
    extern __shared__ uint8_t raw_smem[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~(uintptr_t)1023);
    const uint32_t base = ptx::smem_u32(smem);
    float* exch = reinterpret_cast<float*>(smem + W::kExch);
    Bars* bars = reinterpret_cast<Bars*>(smem + W::kBars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == kMmaWarp) ptx::tmem_alloc(&bars->tmem, kColumns);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&bars->k_full[i], kDequantWarps);
            ptx::mbar_init(&bars->v_full[i], kDequantWarps);
            ptx::mbar_init(&bars->s_full[i], 1);
            ptx::mbar_init(&bars->p_full[i], kSoftmaxWarps);
            ptx::mbar_init(&bars->pv_done[i], 1);
        }
        ptx::mbar_init(&bars->q_full, kSoftmaxWarps);
        for (int i = 0; i < 4; ++i) ptx::mbar_init(&bars->pair[i], 2);
        ptx::mbar_init(&bars->drain, 1);
        bars->abort = 0;
        ptx::fence_mbar_init();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = bars->tmem;

    ptx::griddep_wait();
    if constexpr (!kList) dense_extras<D>(a, warp, lane);

    int pair = blockIdx.x * a.kv_heads;  // dense: the next (head, part) pair
    const int pairs_end = pair + a.kv_heads;
    int it = 0;                          // tiles so far: buffers and phases go by it
    bool ok = true;

    if (warp >= kSoftmaxWarps && warp < kMmaWarp) {
        // ------------------------------------------------------------ dequantise
        const int dw = warp - kSoftmaxWarps, row = dw * kSpan + lane;
        const uint32_t ring = base + W::kRing + dw * (W::kStages * W::kSlot);
        do {
            Range r = open_range<kList>(a, blockIdx.x, pair, pairs_end);
            SpanLoader<D, kTokens, kList, true> loads;
            loads.open(a, r, lane, dw * kSpan);
#pragma unroll
            for (int s = 0; s < W::kStages - 1; ++s) loads.issue(a, ring + s * W::kSlot, s);
            int load_stage = W::kStages - 1, stage = 0;
            while (ok && r.more) {
                const int n = tiles_of(r.w);
                for (int j = 0; j < n; ++j, ++it) {
                    ptx::cp_async_wait<W::kStages - 2>();
                    __syncwarp();
                    loads.issue(a, ring + load_stage * W::kSlot, load_stage);
                    load_stage = load_stage + 1 == W::kStages ? 0 : load_stage + 1;
                    const uint32_t slot = ring + stage * W::kSlot;
                    stage = stage + 1 == W::kStages ? 0 : stage + 1;
                    const uint32_t b = it & 1, before = ((it >> 1) & 1) ^ 1;
                    ok = wait_phase(&bars->s_full[b], before, bars, a.status, lane);
                    if (!ok) break;
                    dequant_row<D>(slot, slot + 2 * kSpan * W::kRow, base + W::kK + b * W::kBuf, lane, row);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&bars->k_full[b]);
                    ok = wait_phase(&bars->pv_done[b], before, bars, a.status, lane);
                    if (!ok) break;
                    dequant_row<D>(slot + kSpan * W::kRow, slot + 2 * kSpan * W::kRow + kSpan * W::kScales,
                                   base + W::kV + b * W::kBuf, lane, row);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&bars->v_full[b]);
                }
                next_row<kList>(a, r);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
        } while (ok && pair < pairs_end && !kList);
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMAs
        const uint32_t id_qk = ptx::instr_desc(0, 0, 128, kTokens);
        const uint32_t id_pv = ptx::instr_desc(0, 0, 128, D) | (1u << 16);  // B is MN-major
        auto scores = [&](int i) {
            const uint32_t b = i & 1;
            if (!wait_phase(&bars->pv_done[b], ((i >> 1) & 1) ^ 1, bars, a.status, lane)) return false;
            if (!wait_phase(&bars->k_full[b], (i >> 1) & 1, bars, a.status, lane)) return false;
            ptx::tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t kd = ptx::smem_desc(
                        base + W::kK + b * W::kBuf + (k >> 2) * (kTokens * 128) + (k & 3) * 32, 16, 1024, ptx::SW_128B);
                    ptx::mma_f16_ts(tmem + kColS + b * 128, tmem + kColQ + k * 8, kd, id_qk, k > 0);
                }
                ptx::tc_commit(&bars->s_full[b]);
            }
            __syncwarp();
            return true;
        };
        int seg = 0;
        do {
            Range r = open_range<kList>(a, blockIdx.x, pair, pairs_end);
            while (ok && r.more) {
                const int n = tiles_of(r.w);
                if (n > 0) {
                    ok = wait_phase(&bars->q_full, seg & 1, bars, a.status, lane) && scores(it);
                    ++seg;
                }
                for (int j = 0; ok && j < n; ++j, ++it) {
                    if (j + 1 < n) ok = scores(it + 1);
                    const uint32_t b = it & 1, phase = (it >> 1) & 1;
                    ok = ok && wait_phase(&bars->v_full[b], phase, bars, a.status, lane) &&
                         wait_phase(&bars->p_full[b], phase, bars, a.status, lane);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    if (lane == 0) {
#pragma unroll
                        for (int k = 0; k < kTokens / 16; ++k) {
                            // 64-element pieces of D lie kTokens * 128 bytes apart, 8-token groups 1024
                            const uint64_t vd = ptx::smem_desc(base + W::kV + b * W::kBuf + k * 2048,
                                                               kTokens * 128, 1024, ptx::SW_128B);
                            ptx::mma_f16_ts(tmem + kColO, tmem + kColS + b * 128 + k * 8, vd, id_pv, j > 0 || k > 0);
                        }
                        ptx::tc_commit(&bars->pv_done[b]);
                    }
                    __syncwarp();
                }
                next_row<kList>(a, r);
            }
        } while (ok && pair < pairs_end && !kList);
        if (lane == 0) {  // nothing of this CTA's MMAs is under way when it ends
            ptx::tc_commit(&bars->drain);
            const uint64_t t0 = ptx::globaltimer();
            while (!ptx::mbar_try_wait_sleep(&bars->drain, 0, kWaitSliceNs))
                if (ptx::globaltimer() - t0 > kTimeoutNs) {
                    report(a.status, MQA_STATUS_TIMEOUT);
                    break;
                }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        const int q4 = warp & 3, half = warp >> 2;
        const int row = q4 * 32 + lane;
        const bool active = q4 * 32 < a.rows;  // the quarter has query rows
        const uint32_t lanes = tmem + ((uint32_t)(q4 * 32) << 16);
        uint32_t swaps = 0;
        // the other warp's value for this row
        auto swap = [&](float mine, float& other) {
            float* at = exch + (swaps & 1) * 256;
            at[half * 128 + row] = mine;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bars->pair[q4]);
            const bool got = wait_phase(&bars->pair[q4], swaps & 1, bars, a.status, lane);
            other = at[(half ^ 1) * 128 + row];
            ++swaps;
            return got;
        };
        const bool flip = a.scale_log2 < 0.f;  // a negative scale goes into q, so that the largest score is the largest S
        do {
            Range r = open_range<kList>(a, blockIdx.x, pair, pairs_end);
            while (ok && r.more) {
                const Walk w = r.w;
                const int n = tiles_of(w);
                const int draft = kList ? r.draft : min(row / a.group, a.next_n - 1);
                const int h = r.hk * a.group + (kList ? row : row - draft * a.group);
                const int64_t at_row = ((int64_t)w.b * a.next_n + draft) * a.heads + h;
                float fac = fabsf(a.scale_log2), m = kUnset, l = 0.f;
                const int limit = min(max(w.ctx - a.next_n + 1 + draft, 0), w.ctx);
                if (n > 0) {
                    if (active) {
                        // ---- this half of the row's q to TMEM
                        uint32_t wds[D / 4];
                        const T* q = static_cast<const T*>(a.q) + (int64_t)w.b * a.q_sb + (int64_t)draft * a.q_sn +
                                     (int64_t)h * a.q_sh + half * (D / 2);
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            const uint4 v = row < a.rows ? __ldg(reinterpret_cast<const uint4*>(q) + i) : make_uint4(0, 0, 0, 0);
                            wds[4 * i] = v.x; wds[4 * i + 1] = v.y; wds[4 * i + 2] = v.z; wds[4 * i + 3] = v.w;
                        }
                        if (flip) {
#pragma unroll
                            for (int i = 0; i < D / 4; ++i) wds[i] ^= 0x80008000u;
                        }
                        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                            uint32_t most = 0;
#pragma unroll
                            for (int i = 0; i < D / 4; ++i)
                                most = max(most, max(wds[i] & 0x7fffu, (wds[i] >> 16) & 0x7fffu));
                            float other;
                            ok = swap(__uint_as_float(most), other);
                            if (!ok) break;
                            most = max(most, __float_as_uint(other));
                            float up, down;
                            q_power(most, up, down);
                            fac *= down;
#pragma unroll
                            for (int i = 0; i < D / 4; ++i)
                                wds[i] = pack_f16(__uint_as_float(wds[i] << 16) * up,
                                                  __uint_as_float(wds[i] & 0xffff0000u) * up);
                        }
#pragma unroll
                        for (int i = 0; i < D / 64; ++i)
                            ptx::tmem_st16(lanes + kColQ + half * (D / 4) + 16 * i,
                                           reinterpret_cast<const uint32_t(&)[16]>(wds[16 * i]));
                        ptx::tmem_st_wait();
                    }
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&bars->q_full);
                }
                for (int j = 0; j < n; ++j, ++it) {
                    const uint32_t b = it & 1, phase = (it >> 1) & 1;
                    const int t = w.t0 + j * kTokens;
                    uint32_t sees[2] = {~0u, ~0u};  // the 64 columns that the row sees
                    bool all;
                    if constexpr (kList) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int e = t + half * 64 + i * 32 + lane;
                            const int tok = e < w.t1 ? __ldg(a.indices + (int64_t)w.item * a.topk + e) : -1;
                            sees[i] = __ballot_sync(0xffffffffu, tok >= 0 && tok < w.ctx);
                        }
                        all = (sees[0] & sees[1]) == ~0u;
                    } else {
                        all = t + kTokens <= min(w.t1, w.ctx - a.next_n + 1);
                        if (!all) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int k = min(max(limit - t - half * 64 - i * 32, 0), 32);
                                sees[i] = k == 32 ? ~0u : (1u << k) - 1;
                            }
                        }
                    }
                    ok = wait_phase(&bars->s_full[b], phase, bars, a.status, lane);
                    if (!ok) break;
                    if (active) {
                        ptx::tc_fence_after();
                        float s[64];
                        tmem_read64(lanes + kColS + b * 128 + half * 64, s);
                        ptx::tc_fence_before();
                        if (!all) {
#pragma unroll
                            for (int i = 0; i < 64; ++i)
                                if (!((sees[i >> 5] >> (i & 31)) & 1)) s[i] = -3e38f;
                        }
                        float top[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            top[i] = s[i];
#pragma unroll
                            for (int k = 4; k < 64; k += 4) top[i] = fmaxf(top[i], s[k + i]);
                        }
                        const float mine = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * fac;
                        float other;
                        ok = swap(mine, other);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        const float most = fmaxf(mine, other);
                        const bool raise = most > m + kSlack;
                        if (__any_sync(0xffffffffu, raise)) {
                            const float by = raise ? ex2(m - most) : 1.f;
                            if (raise) m = most;
                            l *= by;
                            if (j > 0) {
                                ok = wait_phase(&bars->pv_done[b ^ 1], ((it - 1) >> 1) & 1, bars, a.status, lane);
                                if (!ok) break;
                                ptx::tc_fence_after();
#pragma unroll
                                for (int i = 0; i < D / 32; ++i) {
                                    float o[16];
                                    tmem_read16(lanes + kColO + half * (D / 2) + 16 * i, o);
#pragma unroll
                                    for (int k = 0; k < 16; ++k) o[k] *= by;
                                    ptx::tmem_st16(lanes + kColO + half * (D / 2) + 16 * i,
                                                   reinterpret_cast<const uint32_t(&)[16]>(o));
                                }
                            }
                        }
                        // P goes over S: the columns of this half's P were read by the other
                        // warp before the swap
                        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t p[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                float e0 = ex2(fmaf(s[32 * i + 2 * k], fac, -m));
                                float e1 = ex2(fmaf(s[32 * i + 2 * k + 1], fac, -m));
                                if (!all) {
                                    if (!((sees[i] >> (2 * k)) & 1)) e0 = 0.f;
                                    if (!((sees[i] >> (2 * k + 1)) & 1)) e1 = 0.f;
                                }
                                sum[2 * (k & 1)] += e0;
                                sum[2 * (k & 1) + 1] += e1;
                                p[k] = pack_f16(e0, e1);
                            }
                            ptx::tmem_st16(lanes + kColS + b * 128 + half * 32 + 16 * i, p);
                        }
                        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                        ptx::tmem_st_wait();
                        ptx::tc_fence_before();
                    }
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&bars->p_full[b]);
                }
                if (!ok) break;
                // ---- the row's result
                if (n > 0) {
                    ok = wait_phase(&bars->pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1, bars, a.status, lane);
                    if (!ok) break;
                    ptx::tc_fence_after();
                }
                if (active) {
                    float other;
                    ok = swap(l, other);
                    if (!ok) break;
                    l += other;
                    int64_t slot;
                    const bool whole = row_is_whole<kList>(a, r, slot);
                    const int64_t at_part = (slot * a.kv_heads + r.hk) * a.rows + row;
                    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        float o[16];
                        if (n > 0) {
                            tmem_read16(lanes + kColO + half * (D / 2) + 16 * i, o);
                        } else {
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = 0.f;
                        }
                        if (row < a.rows) {
                            const int d = half * (D / 2) + 16 * i;
                            if (whole) {
                                uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + at_row * D + d);
                                uint32_t v[8];
#pragma unroll
                                for (int k = 0; k < 8; ++k) v[k] = pack<T>(o[2 * k] * inv, o[2 * k + 1] * inv);
                                out[0] = make_uint4(v[0], v[1], v[2], v[3]);
                                out[1] = make_uint4(v[4], v[5], v[6], v[7]);
                            } else {
                                float4* out = reinterpret_cast<float4*>(a.part_o + at_part * D + d);
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    out[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                            }
                        }
                    }
                    if (row < a.rows && half == 0) {
                        if (whole) {
                            if (a.lse != nullptr) a.lse[at_row] = lse_of(m, l);
                        } else {
                            *reinterpret_cast<float4*>(a.part_ml + at_part * 4) = make_float4(m, l, l, 0.f);
                        }
                    }
                }
                ptx::tc_fence_before();
                next_row<kList>(a, r);
            }
        } while (ok && pair < pairs_end && !kList);
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kColumns);
    }
}

template <int D, typename T, bool kList>
cudaError_t launch_as(int device, const AttentionArgs& a, void* stream, bool pdl) {
    static uint32_t done[64];
    const cudaError_t e = allow_smem(attention_wide_kernel<D, T, kList>, device, Wide<D>::kSmem, done);
    if (e != cudaSuccess) return e;
    const int64_t x = kList ? (int64_t)a.batch * a.next_n * a.splits * a.kv_heads : a.num_ctas;
    return launch_pdl(attention_wide_kernel<D, T, kList>, dim3((unsigned)x), dim3(kWideThreads),
                      Wide<D>::kSmem, stream, pdl, a);
}

}  // namespace

template <int D, typename T, bool kList>
cudaError_t launch_wide(int device, const AttentionArgs& a, void* stream, bool pdl) {
    return launch_as<D, T, kList>(device, a, stream, pdl);
}

template cudaError_t launch_wide<64, __half, false>(int, const AttentionArgs&, void*, bool);
template cudaError_t launch_wide<64, __half, true>(int, const AttentionArgs&, void*, bool);
template cudaError_t launch_wide<64, __nv_bfloat16, false>(int, const AttentionArgs&, void*, bool);
template cudaError_t launch_wide<64, __nv_bfloat16, true>(int, const AttentionArgs&, void*, bool);
template cudaError_t launch_wide<128, __half, false>(int, const AttentionArgs&, void*, bool);
template cudaError_t launch_wide<128, __half, true>(int, const AttentionArgs&, void*, bool);
template cudaError_t launch_wide<128, __nv_bfloat16, false>(int, const AttentionArgs&, void*, bool);
template cudaError_t launch_wide<128, __nv_bfloat16, true>(int, const AttentionArgs&, void*, bool);

}  // namespace mqa
