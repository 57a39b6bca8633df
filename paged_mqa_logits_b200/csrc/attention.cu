// Softmax attention of a few query positions over a paged cache held in 4 bits.
//
// The mathematics: o = sum_t p_t v_t / sum_t p_t with p_t = 2^(x_t - m), x_t the
// score in base 2 and m a running reference of the row that is at most its
// maximum. m is raised (and what was summed so far rescaled) only when a score
// exceeds it by kSlack, so p <= 2^kSlack fits f16 and most tiles need no rescale.
//
// One warp takes 32 tokens at a time through its own ring of asynchronous copies
// (no CTA barrier inside a row) and dequantises K and V straight into the A
// fragments of mma.sync.m16n8k16 (f16 x f16 -> f32; code * scale has at most 6
// significant bits and is exact in f16): S^T = K Q^T (16 tokens x 8 query rows),
// then O^T += V^T P^T, whose B operand is S^T's result transposed within the warp.
// The query rows are N, so 8 rows cost 8 and not 16. At the end of a row the CTA's
// warps join their (m, sum, O) through shared memory; rows that several CTAs share
// leave partial results, which combine_kernel joins.
#include "common.cuh"

#include "attention.cuh"
#include "host.cuh"

namespace mqa {
namespace {

constexpr int kSpan = 32;         // tokens of a ring slot
constexpr float kUnset = -1e30f;  // m of a row that has seen no token
constexpr float kSlack = 8.f;     // p <= 2^8

// NT: query rows of a CTA / 8. More rows take more registers, so fewer warps.
template <int D, int NT>
struct Shape {
    static constexpr int kWarps = NT == 1 ? 16 : NT == 2 ? 12 : 8;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kRow = D / 2;                       // code bytes of a token
    static constexpr int kScales = D / 16;                   // scale bytes of a token
    static constexpr int kSlot = 2 * kSpan * (kRow + kScales);  // K codes, V codes, K scales, V scales
    static constexpr int kStages = 2 * 128 / D;
    static constexpr int kRing = kWarps * kStages * kSlot;
    static constexpr int kLane = D / 8;                      // floats that a lane leaves of a row of O
    static constexpr int kRedRow = D + 4;                    // floats of a row, padded
    static constexpr int kRows = 8 * NT;
    static constexpr int kRed = kWarps * kRows * kRedRow * 4;
    static constexpr int kSmem = kRing + kRed + kWarps * kRows * 4 * 4;
    static_assert(kSmem <= 232448, "more shared memory than a CTA can have");
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// d += a (16 x 16) * b (16 x 8), f16 operands, fp32 accumulation.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of f16 that the warp holds as fragments.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Eight e2m1 codes as four f16 pairs; byte i becomes pair i (low nibble first).
__device__ __forceinline__ void e2m1_to_f16(uint32_t w, uint32_t (&o)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]) : "r"(w));
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return h;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 16 or 8 bytes global -> shared; zeros where `take` is false (nothing is read).
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool take) {
    const int bytes = take ? N : 0;
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                     ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;"
                     ::"r"(dst), "l"(src), "r"(bytes), "n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// Where a ring slot keeps byte `o` of token t's codes: rows are permuted (and, for
// 64-byte rows, their 16-byte pieces) so that the K fragments' reads (8 tokens,
// 16 or 8 bytes a lane) and the V fragments' (tokens 2c of the four lanes of a
// quad) each touch every bank once.
template <int D>
__device__ __forceinline__ uint32_t code_at(uint32_t t, uint32_t o) {
    if constexpr (D == 128)
        return (t ^ ((t >> 1) & 1)) * 64 + (o ^ ((t & 4) << 3));
    else
        return (t ^ ((t >> 2) & 1)) * 32 + o;
}

template <typename T>
__device__ __forceinline__ uint32_t pack(float a, float b) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        return pack_f16(a, b);
    }
}

// 2^top * sum as a natural logarithm; -inf where nothing was summed.
__device__ __forceinline__ float lse_of(float top, float sum) {
    return sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.693147180559945f;
}

// A CTA's walk over its rows and over this warp's chunks of them. Dense: the
// schedule's range; selected: one part of one list.
struct Walk {
    int b, last_b, last_u;  // row, and where the CTA's range ends
    int item;               // the row's index for q and out: b, or b * next_n + n (selected)
    int ctx;                // tokens of the row (dense), visible tokens (selected)
    int t0, t1;             // the CTA's tokens (list entries) of this row
};

template <bool kList>
__device__ __forceinline__ int row_ctx(const AttentionArgs& a, int b) {
    return clamp_len(a.status, __ldg(a.context_lens + b), a.max_pages << a.ps_shift);
}

// Dense: the first row at or after w.b that has tokens in this CTA's range,
// starting at unit u0 of row w.b. False: none left.
__device__ __forceinline__ bool settle(const AttentionArgs& a, Walk& w, int u0) {
    while (w.b < a.batch && (w.b < w.last_b || (w.b == w.last_b && u0 < w.last_u))) {
        w.ctx = row_ctx<false>(a, w.b);
        const int units = (w.ctx + kUnit - 1) / kUnit;
        const int u1 = w.b == w.last_b ? min(units, w.last_u) : units;
        if (u0 < u1) {
            w.item = w.b;
            w.t0 = u0 * kUnit;
            w.t1 = min(u1 * kUnit, w.ctx);
            return true;
        }
        ++w.b;
        u0 = 0;
    }
    return false;
}

// The parts of the schedule that CTA i of a dense launch takes: with Hk kv heads the
// Hk * S (head, part) pairs are dealt in order, Hk to each CTA, so that a CTA walks
// up to Hk neighbouring parts of one head as one range and rows are cut S + Hk
// times over all heads. Range k of head hk begins at part range_start(hk, k).
__host__ __device__ inline int range_start(int hk, int k, int heads, int S) {
    const int first = (int)(((int64_t)hk * S) % heads);  // parts of the head in its first CTA: heads - first
    return k == 0 ? 0 : min(S, k * heads - first);
}

template <int D, int NT, typename T, bool kList>
__global__ void __launch_bounds__(Shape<D, NT>::kThreads, 1) attention_kernel(const AttentionArgs a) {
    using S = Shape<D, NT>;
    constexpr int kWarps = S::kWarps, kThreads = S::kThreads;
    constexpr int kTiles = D / 16;   // row tiles of O^T, and contraction steps of K Q^T
    constexpr int kElems = D / 4;    // elements of a row of q or K that one lane of a quad holds
    extern __shared__ __align__(128) uint8_t smem[];
    float* red = reinterpret_cast<float*>(smem + S::kRing);
    float* red_ml = reinterpret_cast<float*>(smem + S::kRing + S::kRed);  // [warp][row][4]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const uint32_t ring = ptx::smem_u32(smem) + warp * (S::kStages * S::kSlot);
    const int row0 = blockIdx.y * S::kRows;  // first query row of this CTA

    ptx::griddep_wait();

    if constexpr (!kList) {
        if ((a.status.flags & MQA_FLAG_VALIDATE) && blockIdx.y == 0 && warp == 0) {
            KernelArgs ka{};
            ka.context_lens = a.context_lens;
            ka.schedule = a.schedule;
            ka.status = a.status.caller;
            ka.lib_status = a.status.lib;
            ka.batch = a.batch;
            ka.num_ctas = a.num_ctas;
            check_schedule(ka, blockIdx.x, lane);
        }
        // rows without tokens are in no CTA's range: their results are written here
        for (int b = blockIdx.x; b < a.batch; b += a.num_ctas) {
            if (__ldg(a.context_lens + b) > 0) continue;
            const int64_t o = (int64_t)b * a.next_n * a.heads;
            for (int j = threadIdx.x; j < a.next_n * a.heads * (D / 8); j += kThreads)
                reinterpret_cast<uint4*>(a.out)[o * (D / 8) + j] = make_uint4(0, 0, 0, 0);
            if (a.lse != nullptr)
                for (int j = threadIdx.x; j < a.next_n * a.heads; j += kThreads) a.lse[o + j] = -INFINITY;
        }
    }

    int pair = kList ? 0 : blockIdx.x * a.kv_heads;  // dense: the next (head, part) pair
    const int pairs_end = pair + a.kv_heads;
    do {
        // ---- one range of rows of one kv head
        Walk w;
        int draft = 0, part = 0, hk;
        bool more;
        if constexpr (kList) {
            hk = blockIdx.x % a.kv_heads;
            const int x = blockIdx.x / a.kv_heads;
            w.item = x / a.splits;
            part = x - w.item * a.splits;
            w.b = w.item / a.next_n;
            draft = w.item - w.b * a.next_n;
            const int full = row_ctx<kList>(a, w.b);
            w.ctx = min(max(full - a.next_n + 1 + draft, 0), full);
            const int per = ((a.topk + a.splits - 1) / a.splits + kSpan - 1) / kSpan * kSpan;
            w.t0 = min(a.topk, part * per);
            w.t1 = min(a.topk, w.t0 + per);
            more = true;
        } else {
            hk = pair / a.num_ctas;
            part = pair - hk * a.num_ctas;
            const int n = min(a.num_ctas - part, pairs_end - pair);
            pair += n;
            w.b = max(__ldg(a.schedule + 2 * part), 0);
            const int u0 = max(__ldg(a.schedule + 2 * part + 1), 0);
            w.last_b = __ldg(a.schedule + 2 * (part + n));
            w.last_u = __ldg(a.schedule + 2 * (part + n) + 1);
            more = settle(a, w, u0);
        }

        // ---- loads: a walk that runs ahead of the computation by kStages - 1 spans
        Walk lw = w;
        bool lmore = more;
        int lpos = lw.t0 + warp * kSpan;  // next span to resolve
        // The cache slot (page * page_size + slot) of this lane's token of the next
        // span, -1 for none, found one step before its copies are issued.
        int next_slot = -1;
        bool next_any = false;            // the span exists
        const int32_t* list = kList ? a.indices + (int64_t)w.item * a.topk : nullptr;

        auto resolve = [&]() {
            next_any = false;
            next_slot = -1;
            if constexpr (kList) {
                if (lpos >= lw.t1) return;
            } else {
                while (lmore && lpos >= lw.t1) {
                    ++lw.b;
                    lmore = settle(a, lw, 0);
                    lpos = lw.t0 + warp * kSpan;
                }
                if (!lmore) return;
            }
            next_any = true;
            int t = lpos + lane;
            lpos += kWarps * kSpan;
            bool ok = t < lw.t1;
            if constexpr (kList) {
                t = ok ? __ldg(list + t) : -1;
                ok = t >= 0 && t < lw.ctx;
            }
            if (ok) {
                int page = __ldg(a.block_table + (int64_t)lw.b * a.max_pages + (t >> a.ps_shift));
                if (page < 0 || page >= a.num_pages) {
                    report_checked(a.status, MQA_STATUS_BAD_PAGE);
                    page = page < 0 ? 0 : a.num_pages - 1;
                }
                next_slot = (page << a.ps_shift) | (t & (a.page_size - 1));
            }
        };

        const int64_t head_at = (int64_t)hk * a.page_size * (S::kRow + S::kScales);
        uint32_t seen = 0;  // selected: lane s keeps the mask of the visible tokens in ring slot s
        auto issue = [&](int stage) {
            if (next_any) {
                const uint32_t base = ring + stage * S::kSlot;
                constexpr int kPieces = S::kRow / 16;       // 16-byte pieces of a token's codes
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const int p = i * 32 + lane, t = p / kPieces, o = (p % kPieces) * 16;
                    const int at = __shfl_sync(0xffffffffu, next_slot, t);
                    const int64_t off = (int64_t)(max(at, 0) >> a.ps_shift) * a.page_bytes + head_at +
                                        (max(at, 0) & (a.page_size - 1)) * S::kRow + o;
                    copy_async<16>(base + code_at<D>(t, o), a.k + off, at >= 0);
                    copy_async<16>(base + kSpan * S::kRow + code_at<D>(t, o), a.v + off, at >= 0);
                }
                const int at = max(next_slot, 0);
                const int64_t off = (int64_t)(at >> a.ps_shift) * a.page_bytes + head_at +
                                    a.page_size * S::kRow + (at & (a.page_size - 1)) * S::kScales;
                const uint32_t sc = base + 2 * kSpan * S::kRow + lane * S::kScales;
                copy_async<S::kScales>(sc, a.k + off, next_slot >= 0);
                copy_async<S::kScales>(sc + kSpan * S::kScales, a.v + off, next_slot >= 0);
                if constexpr (kList) {
                    const uint32_t m = __ballot_sync(0xffffffffu, next_slot >= 0);
                    if (lane == stage) seen = m;
                }
            }
            ptx::cp_async_commit();
            resolve();
        };

        resolve();
#pragma unroll
        for (int s = 0; s < S::kStages - 1; ++s) issue(s);
        int load_stage = S::kStages - 1, stage = 0;

        // ---- rows
        while (more) {
            // q of row g of every 8, as f16 fragments; a bf16 row is scaled so that its
            // largest element lies in [2^14, 2^15)
            uint32_t qf[NT][kElems / 2];
            float fac[NT][2];  // of rows 2c and 2c + 1: what the scores are multiplied by
            int limit[NT][2];  // dense: tokens that the row's position sees
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int r = row0 + nt * 8 + g;
                const int n = kList ? draft : min(r / a.group, a.next_n - 1);
                const int h = hk * a.group + (kList ? r : r - n * a.group);
                uint4 raw[kElems / 8];
                const T* q = static_cast<const T*>(a.q) + (int64_t)w.b * a.q_sb + (int64_t)n * a.q_sn +
                             (int64_t)h * a.q_sh + c * kElems;
#pragma unroll
                for (int i = 0; i < kElems / 8; ++i)
                    raw[i] = r < a.rows ? __ldg(reinterpret_cast<const uint4*>(q) + i) : make_uint4(0, 0, 0, 0);
                const uint32_t* wds = reinterpret_cast<const uint32_t*>(raw);
                float down = a.scale_log2;
                if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                    uint32_t most = 0;  // |x| bits compare like integers
#pragma unroll
                    for (int i = 0; i < kElems / 2; ++i)
                        most = max(most, max(wds[i] & 0x7fffu, (wds[i] >> 16) & 0x7fffu));
                    most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
                    most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
                    // exponent of the largest, kept where 2^(14 - e) is a normal fp32
                    const int ex = most == 0 ? 14 : max((int)(most >> 7) - 127, -100);
                    const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
                    down *= __uint_as_float((uint32_t)(127 - 14 + ex) << 23);
#pragma unroll
                    for (int i = 0; i < kElems / 2; ++i)
                        qf[nt][i] = pack_f16(__uint_as_float(wds[i] << 16) * up,
                                             __uint_as_float(wds[i] & 0xffff0000u) * up);
                } else {
#pragma unroll
                    for (int i = 0; i < kElems / 2; ++i) qf[nt][i] = wds[i];
                }
                const int sees = min(max(w.ctx - a.next_n + 1 + n, 0), w.ctx);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    fac[nt][j] = __shfl_sync(0xffffffffu, down, 4 * (2 * c + j));
                    limit[nt][j] = __shfl_sync(0xffffffffu, sees, 4 * (2 * c + j));
                }
            }

            float o[NT][kTiles][4], sum[NT][4], m[NT][2], lraw[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sum[nt][i] = 0.f;
#pragma unroll
                    for (int j = 0; j < kTiles; ++j) o[nt][j][i] = 0.f;
                }
                m[nt][0] = m[nt][1] = kUnset;
                lraw[nt][0] = lraw[nt][1] = 0.f;
            }

            for (int t = w.t0 + warp * kSpan; t < w.t1; t += kWarps * kSpan) {
                ptx::cp_async_wait<S::kStages - 2>();
                __syncwarp();
                // which of the span's tokens rows 2c and 2c + 1 see
                uint32_t sees[NT][2];
                bool all;
                if constexpr (kList) {
                    const uint32_t s = __shfl_sync(0xffffffffu, seen, stage);
                    all = s == 0xffffffffu;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) sees[nt][0] = sees[nt][1] = s;
                } else {
                    all = t + kSpan <= min(w.t1, w.ctx - a.next_n + 1);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int n = min(max(limit[nt][j] - t, 0), kSpan);
                            sees[nt][j] = n == 32 ? 0xffffffffu : (1u << n) - 1;
                        }
                }
                issue(load_stage);
                load_stage = load_stage + 1 == S::kStages ? 0 : load_stage + 1;
                const uint32_t kc = ring + stage * S::kSlot, vc = kc + kSpan * S::kRow;
                const uint32_t ks = vc + kSpan * S::kRow, vs = ks + kSpan * S::kScales;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    // ---- scores of 16 tokens: this lane's are g and g + 8
                    float x[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[nt][i] = 0.f;
                    uint32_t kw[2][kElems / 8], s2[2][2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t tok = half * 16 + e * 8 + g;
                        if constexpr (D == 128) {
                            const uint4 v = lds128(kc + code_at<D>(tok, c * 16));
                            kw[e][0] = v.x; kw[e][1] = v.y; kw[e][2] = v.z; kw[e][3] = v.w;
                            const uint32_t h = e4m3x2_to_f16(lds16(ks + tok * 8 + c * 2));
                            s2[e][0] = __byte_perm(h, h, 0x1010);
                            s2[e][1] = __byte_perm(h, h, 0x3232);
                        } else {
                            const uint2 v = lds64(kc + code_at<D>(tok, c * 8));
                            kw[e][0] = v.x; kw[e][1] = v.y;
                            const uint32_t h = e4m3x2_to_f16(lds8(ks + tok * 4 + c));
                            s2[e][0] = s2[e][1] = __byte_perm(h, h, 0x1010);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kElems / 8; ++i) {
                        uint32_t f[2][4];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            e2m1_to_f16(kw[e][i], f[e]);
#pragma unroll
                            for (int k = 0; k < 4; ++k) f[e][k] = mul_f16x2(f[e][k], s2[e][i / 2]);
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816(x[nt], f[0][2 * k], f[1][2 * k], f[0][2 * k + 1], f[1][2 * k + 1],
                                         qf[nt][4 * i + 2 * k], qf[nt][4 * i + 2 * k + 1]);
                    }
                    // ---- y: the scores in base 2, less m
                    float y[NT][4];
                    auto scores = [&](int nt, float m0, float m1) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            y[nt][i] = fmaf(x[nt][i], fac[nt][i & 1], i & 1 ? -m1 : -m0);
                            if (!all && !((sees[nt][i & 1] >> (half * 16 + (i >> 1) * 8 + g)) & 1))
                                y[nt][i] = -INFINITY;
                        }
                    };
                    bool raise = false;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        scores(nt, m[nt][0], m[nt][1]);
                        raise |= fmaxf(fmaxf(y[nt][0], y[nt][1]), fmaxf(y[nt][2], y[nt][3])) > kSlack;
                    }
                    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            scores(nt, 0.f, 0.f);
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                float to = fmaxf(y[nt][j], y[nt][j + 2]);
#pragma unroll
                                for (int d = 4; d < 32; d <<= 1)
                                    to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, d));
                                to = fmaxf(to, m[nt][j]);
                                const float by = ex2(m[nt][j] - to);
                                m[nt][j] = to;
#pragma unroll
                                for (int i = 0; i < kTiles; ++i) {
                                    o[nt][i][j] *= by;
                                    o[nt][i][j + 2] *= by;
                                }
                                sum[nt][j] *= by;
                                lraw[nt][j] *= by;
                            }
                            scores(nt, m[nt][0], m[nt][1]);
                        }
                    }
                    uint32_t pf[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            y[nt][i] = ex2(y[nt][i]);
                            lraw[nt][i & 1] += y[nt][i];
                        }
                        pf[nt][0] = transpose8(pack_f16(y[nt][0], y[nt][1]));
                        pf[nt][1] = transpose8(pack_f16(y[nt][2], y[nt][3]));
                        // the sums of the rounded p, by rows of ones
                        mma16816(sum[nt], 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, pf[nt][0], pf[nt][1]);
                    }
                    // ---- O^T += V^T P^T: tokens 2c, 2c+1 and 2c+8, 2c+9, elements [g D/8, (g+1) D/8)
                    uint32_t vw[4][D / 64], vsc[2];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t tok = half * 16 + 2 * c + (e & 1) + 8 * (e >> 1);
                        if constexpr (D == 128) {
                            const uint2 v = lds64(vc + code_at<D>(tok, g * 8));
                            vw[e][0] = v.x; vw[e][1] = v.y;
                        } else {
                            vw[e][0] = lds32(vc + code_at<D>(tok, g * 4));
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t at = vs + (half * 16 + 2 * c + 8 * e) * S::kScales + (D == 128 ? g : g / 2);
                        vsc[e] = e4m3x2_to_f16(lds8(at) | lds8(at + S::kScales) << 8);
                    }
#pragma unroll
                    for (int i = 0; i < D / 64; ++i) {
                        // bytes of (token, next token) code pairs, even and odd elements
                        uint32_t f[2][2][4];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t lo = vw[2 * e][i], hi = vw[2 * e + 1][i];
                            e2m1_to_f16((lo & 0x0f0f0f0fu) | ((hi << 4) & 0xf0f0f0f0u), f[e][0]);
                            e2m1_to_f16(((lo >> 4) & 0x0f0f0f0fu) | (hi & 0xf0f0f0f0u), f[e][1]);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t a0 = mul_f16x2(f[0][0][k], vsc[0]), a1 = mul_f16x2(f[0][1][k], vsc[0]);
                            const uint32_t a2 = mul_f16x2(f[1][0][k], vsc[1]), a3 = mul_f16x2(f[1][1][k], vsc[1]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816(o[nt][4 * i + k], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
                        }
                    }
                }
                stage = stage + 1 == S::kStages ? 0 : stage + 1;
                __syncwarp();
            }

            // ---- the CTA's warps join their results; whole rows are written, others left as partials
            bool whole;
            int64_t slot;
            if constexpr (kList) {
                whole = a.splits == 1;
                slot = (int64_t)w.item * a.splits + part;
            } else {
                whole = w.t0 == 0 && w.t1 == w.ctx;
                slot = 2 * part + (w.t0 > 0 ? 0 : 1);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float l = lraw[nt][j];
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
                    const int row = warp * S::kRows + nt * 8 + 2 * c + j;
                    float* at = red + row * S::kRedRow + g * S::kLane;
#pragma unroll
                    for (int i = 0; i < kTiles; i += 2)
                        *reinterpret_cast<float4*>(at + 2 * i) =
                            make_float4(o[nt][i][j], o[nt][i][j + 2], o[nt][i + 1][j], o[nt][i + 1][j + 2]);
                    if (g == 0)
                        *reinterpret_cast<float4*>(red_ml + row * 4) = make_float4(m[nt][j], sum[nt][j], l, 0.f);
                }
            }
            __syncthreads();
            for (int i = threadIdx.x; i < S::kRows * (D / 4); i += kThreads) {
                const int rr = i / (D / 4), d = i % (D / 4) * 4, r = row0 + rr;
                if (r >= a.rows) break;
                float top = kUnset;
#pragma unroll
                for (int k = 0; k < kWarps; ++k) top = fmaxf(top, red_ml[(k * S::kRows + rr) * 4]);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                float total = 0.f, raw = 0.f;
#pragma unroll
                for (int k = 0; k < kWarps; ++k) {
                    const float4 ml = *reinterpret_cast<const float4*>(red_ml + (k * S::kRows + rr) * 4);
                    const float by = ex2(ml.x - top);
                    const float4 p = *reinterpret_cast<const float4*>(
                        red + (k * S::kRows + rr) * S::kRedRow + d / (D / 8) * S::kLane + d % (D / 8));
                    v.x = fmaf(p.x, by, v.x);
                    v.y = fmaf(p.y, by, v.y);
                    v.z = fmaf(p.z, by, v.z);
                    v.w = fmaf(p.w, by, v.w);
                    total = fmaf(ml.y, by, total);
                    raw = fmaf(ml.z, by, raw);
                }
                if (whole) {
                    const int n = kList ? draft : r / a.group;
                    const int64_t at = ((int64_t)w.b * a.next_n + n) * a.heads + hk * a.group + (kList ? r : r - n * a.group);
                    const float inv = total == 0.f ? 0.f : 1.f / total;
                    *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + at * D + d) =
                        make_uint2(pack<T>(v.x * inv, v.y * inv), pack<T>(v.z * inv, v.w * inv));
                    if (a.lse != nullptr && d == 0) a.lse[at] = lse_of(top, raw);
                } else {
                    const int64_t at = (slot * a.kv_heads + hk) * a.rows + r;
                    *reinterpret_cast<float4*>(a.part_o + at * D + d) = v;
                    if (d == 0) *reinterpret_cast<float4*>(a.part_ml + at * 4) = make_float4(top, total, raw, 0.f);
                }
            }
            __syncthreads();

            if constexpr (kList) {
                more = false;
            } else {
                ++w.b;
                more = settle(a, w, 0);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } while (pair < pairs_end && !kList);
}

// ---------------------------------------------------------------- combine
// Joins the partial results of one query row: `wpr` warps a row, a lane takes
// D / 32 elements of it.
constexpr int kCombineThreads = 256;

template <int D, typename T, bool kList>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const AttentionArgs a, int wpr) {
    constexpr int kV = D / 32;  // elements of a lane
    __shared__ float part[8][D + 4];
    ptx::griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows_per_cta = 8 / wpr, sub = warp % wpr;
    const int64_t id = (int64_t)blockIdx.x * rows_per_cta + warp / wpr;  // (item, hk, r)
    const int64_t per_item = (int64_t)a.kv_heads * a.rows;
    const int items = kList ? a.batch * a.next_n : a.batch;
    const bool inside = id < items * per_item;
    const int item = inside ? (int)(id / per_item) : 0;
    const int hr = (int)(id - (int64_t)item * per_item);  // hk * rows + r

    const int hk = hr / a.rows, r = hr - hk * a.rows;

    // ranges first .. last (parts of the list) hold the row's partials
    int first = 0, last = -1;
    if constexpr (kList) {
        last = a.splits - 1;
    } else {
        // the head's ranges that begin at or before the row's first token, and at or
        // before its last: warp-wide counts (they ascend)
        const int ctx = row_ctx<kList>(a, item);
        int at = 0, upto = 0;
        for (int k = lane;; k += 32) {
            const int i = range_start(hk, k, a.kv_heads, a.num_ctas);
            if (i >= a.num_ctas) break;
            const int b = __ldg(a.schedule + 2 * i), u = __ldg(a.schedule + 2 * i + 1);
            at += b < item || (b == item && u <= 0);
            upto += b < item || (b == item && (int64_t)u * kUnit < ctx);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            at += __shfl_xor_sync(0xffffffffu, at, o);
            upto += __shfl_xor_sync(0xffffffffu, upto, o);
        }
        first = max(at - 1, 0);
        last = upto - 1;
    }
    bool work = inside;
    if constexpr (!kList) work = work && last > first && row_ctx<kList>(a, item) > 0;

    float top = kUnset, total = 0.f, raw = 0.f, v[kV] = {};
    if (work) {
        for (int i = first + sub; i <= last; i += wpr) {
            const int64_t slot = kList ? (int64_t)item * a.splits + i
                                       : 2 * (int64_t)range_start(hk, i, a.kv_heads, a.num_ctas) + (i == first);
            const int64_t at = slot * per_item + hr;
            const float4 ml = *reinterpret_cast<const float4*>(a.part_ml + at * 4);
            float p[kV];
#pragma unroll
            for (int k = 0; k < kV; ++k) p[k] = a.part_o[at * D + lane * kV + k];
            const float to = fmaxf(top, ml.x);
            const float keep = ex2(top - to), by = ex2(ml.x - to);
            top = to;
            total = total * keep + ml.y * by;
            raw = raw * keep + ml.z * by;
#pragma unroll
            for (int k = 0; k < kV; ++k) v[k] = v[k] * keep + p[k] * by;
        }
    }
    if (wpr > 1) {
#pragma unroll
        for (int k = 0; k < kV; ++k) part[warp][lane * kV + k] = v[k];
        if (lane == 0) {
            part[warp][D] = top;
            part[warp][D + 1] = total;
            part[warp][D + 2] = raw;
        }
        __syncthreads();
        if (sub != 0) return;
        for (int i = 1; i < wpr; ++i) {
            const float* o = part[warp + i];
            const float to = fmaxf(top, o[D]);
            const float keep = ex2(top - to), by = ex2(o[D] - to);
            top = to;
            total = total * keep + o[D + 1] * by;
            raw = raw * keep + o[D + 2] * by;
#pragma unroll
            for (int k = 0; k < kV; ++k) v[k] = v[k] * keep + o[lane * kV + k] * by;
        }
    }
    if (!work) return;
    const int n = kList ? item % a.next_n : r / a.group;
    const int b = kList ? item / a.next_n : item;
    const int64_t at = ((int64_t)b * a.next_n + n) * a.heads + hk * a.group + (kList ? r : r - n * a.group);
    const float inv = total == 0.f ? 0.f : 1.f / total;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + at * D + lane * kV);
#pragma unroll
    for (int k = 0; k < kV; k += 2) out[k / 2] = pack<T>(v[k] * inv, v[k + 1] * inv);
    if (a.lse != nullptr && lane == 0) a.lse[at] = lse_of(top, raw);
}

template <int D, int NT, typename T, bool kList>
cudaError_t launch_as(int device, const AttentionArgs& a, void* stream, bool pdl) {
    using S = Shape<D, NT>;
    static uint32_t done[64];
    cudaError_t e = allow_smem(attention_kernel<D, NT, T, kList>, device, S::kSmem, done);
    if (e != cudaSuccess) return e;
    const int groups = (a.rows + S::kRows - 1) / S::kRows;
    const int64_t items = kList ? (int64_t)a.batch * a.next_n : a.batch;
    const int64_t x = kList ? items * a.splits * a.kv_heads : a.num_ctas;
    e = launch_pdl(attention_kernel<D, NT, T, kList>, dim3((unsigned)x, groups), dim3(S::kThreads),
                   S::kSmem, stream, pdl, a);
    if (e != cudaSuccess || (kList && a.splits == 1)) return e;
    const int64_t parts = kList ? a.splits : (a.num_ctas + a.batch * a.kv_heads - 1) / (a.batch * a.kv_heads) + 1;
    int wpr = 1;
    while (wpr < 8 && wpr * 4 < parts) wpr *= 2;
    const int64_t rows = items * a.kv_heads * a.rows;
    return launch_pdl(combine_kernel<D, T, kList>, dim3((unsigned)((rows * wpr + 7) / 8)),
                      dim3(kCombineThreads), 0, stream, pdl, a, wpr);
}

template <int D, int NT, typename T>
cudaError_t launch_kind(int device, const AttentionArgs& a, void* stream, bool pdl) {
    return a.topk > 0 ? launch_as<D, NT, T, true>(device, a, stream, pdl)
                      : launch_as<D, NT, T, false>(device, a, stream, pdl);
}

template <int D, typename T>
cudaError_t launch_rows(int device, const AttentionArgs& a, void* stream, bool pdl) {
    if (a.rows <= 8) return launch_kind<D, 1, T>(device, a, stream, pdl);
    if (a.rows <= 16) return launch_kind<D, 2, T>(device, a, stream, pdl);
    return launch_kind<D, 4, T>(device, a, stream, pdl);
}

}  // namespace

cudaError_t launch_attention(int device, int head_dim, int dtype, const AttentionArgs& a,
                             void* stream, bool pdl) {
    if (head_dim == 64)
        return dtype == MQA_DTYPE_BF16 ? launch_rows<64, __nv_bfloat16>(device, a, stream, pdl)
                                       : launch_rows<64, __half>(device, a, stream, pdl);
    return dtype == MQA_DTYPE_BF16 ? launch_rows<128, __nv_bfloat16>(device, a, stream, pdl)
                                   : launch_rows<128, __half>(device, a, stream, pdl);
}

}  // namespace mqa
