// Softmax attention of a few query positions over a paged cache held in 4 bits.
//
// The mathematics: o = sum_t p_t v_t / sum_t p_t with p_t = 2^(x_t - m), x_t the
// score in base 2 and m a running reference of the row that is at most its
// maximum. m is raised (and what was summed so far rescaled) only when a score
// exceeds it by kSlack, to kRoom below the maximum, so p fits f16, few of the small
// ones vanish, and most tiles need no rescale.
//
// One warp takes 32 tokens at a time through its own ring of asynchronous copies
// (no CTA barrier inside a row) and dequantises K and V straight into the A
// fragments of mma.sync.m16n8k16 (f16 x f16 -> f32; code * scale has at most 6
// significant bits and is exact in f16): S^T = K Q^T (16 tokens x 8 query rows),
// then O^T += V^T P^T, whose B operand is S^T's result transposed within the warp.
// The query rows are N, so 8 rows cost 8 and not 16. At the end of a row the CTA's
// warps join their (m, sum, O) through shared memory; rows that several CTAs share
// leave partial results, which combine_kernel joins.
//
// For up to 16 query rows a kv head, and more with short lists (see split_list); beyond,
// attention_wide.cu. mma.sync runs one
// m16n8k16 every two cycles an SM, which 8 rows need 2.1 of a token (D = 128, K and V)
// and 32 rows 8.5, against 6.3 cycles that HBM needs to bring it: 32 rows, lists of
// 2048 tokens, took 47 us here and 28 us there; one row of 1000 tokens 16.7 and 14.4.
//
// Measured: 64 rows of 1024 to 8192 tokens, 8 kv heads with 8 query heads each, D =
// 128: 89 us for 342 MB, 3.8 TB/s or 0.60 of the copy rate. What bounds it is issue: 63
// % of the issue slots, the integer pipe (e2m1 conversions, nibbles) at 55 %, the
// tensor pipe at 24 %, and 11 % of the time before the first and after the last
// token. Rows of 16 query heads: 154 tokens a microsecond and SM, mma.sync at 0.7.
#include <algorithm>

#include "attention_walk.cuh"
#include "host.cuh"

namespace mqa {
namespace {

// NT: query rows of a CTA / 8. More rows take more registers, so fewer warps. kSmall: CTAs
// of 4 warps, several to an SM, for token lists (see split_list) and grouped heads (see launch_as).
template <int D, int NT, bool kSmall>
struct Shape {
    static constexpr int kWarps = kSmall ? 4 : NT == 1 ? 16 : 12;
    static constexpr int kPerSm = kSmall ? (NT == 1 ? 4 : 3) : 1;
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
    static_assert(kPerSm * (kSmem + 1024) <= 233472, "more shared memory than an SM has");
};

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

template <int D, int NT, typename T, bool kList, bool kSmall>
__global__ void __launch_bounds__(Shape<D, NT, kSmall>::kThreads, Shape<D, NT, kSmall>::kPerSm)
attention_kernel(const AttentionArgs a) {
    using S = Shape<D, NT, kSmall>;
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

    __shared__ int parts;
    if (!kList) {
        const int n = parts_with_rows(a, lane);
        if (threadIdx.x == 0) parts = n;
        __syncthreads();
    }
    int pair = kList ? 0 : first_pair(a, parts, blockIdx.x);  // dense: the next (head, part) pair
    bool last;
    do {
        Range r = open_range<kList>(a, blockIdx.x, parts, pair, last);
        const Walk& w = r.w;
        const int hk = r.hk, draft = r.draft;
        SpanLoader<D, kWarps * kSpan, kList, false> loads;
        loads.open(a, r, lane, warp * kSpan);
#pragma unroll
        for (int s = 0; s < S::kStages - 1; ++s) loads.issue(a, ring + s * S::kSlot, s);
        int load_stage = S::kStages - 1, stage = 0;

        // ---- rows
        while (r.more) {
            // q of row g of every 8, as f16 fragments; a bf16 row is scaled so that its
            // largest element lies in [2^14, 2^15)
            uint32_t qf[NT][kElems / 2];
            float fac[NT][2];  // of rows 2c and 2c + 1: what the scores are multiplied by
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int row = row0 + nt * 8 + g;
                const int n = kList ? draft : min(row / a.group, a.next_n - 1);
                const int h = hk * a.group + (kList ? row : row - n * a.group);
                uint4 raw[kElems / 8];
                const T* q = static_cast<const T*>(a.q) + (int64_t)w.b * a.q_sb + (int64_t)n * a.q_sn +
                             (int64_t)h * a.q_sh + c * kElems;
#pragma unroll
                for (int i = 0; i < kElems / 8; ++i)
                    raw[i] = row < a.rows ? __ldg(reinterpret_cast<const uint4*>(q) + i) : make_uint4(0, 0, 0, 0);
                const uint32_t* wds = reinterpret_cast<const uint32_t*>(raw);
                float down = fabsf(a.scale_log2);
                uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale's sign goes into q
                if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                    uint32_t most = 0;  // |x| bits compare like integers
#pragma unroll
                    for (int i = 0; i < kElems / 2; ++i)
                        most = max(most, max(wds[i] & 0x7fffu, (wds[i] >> 16) & 0x7fffu));
                    most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
                    most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
                    float up, back;
                    q_power(most, up, back);
                    down *= back;
#pragma unroll
                    for (int i = 0; i < kElems / 2; ++i)
                        qf[nt][i] = flip ^ pack_f16(__uint_as_float(wds[i] << 16) * up,
                                                    __uint_as_float(wds[i] & 0xffff0000u) * up);
                } else {
#pragma unroll
                    for (int i = 0; i < kElems / 2; ++i) qf[nt][i] = flip ^ wds[i];
                }
                down = fmaxf(down, 1e-37f);  // a factor of 0 must not make NaN of an invisible token's -inf
#pragma unroll
                for (int j = 0; j < 2; ++j) fac[nt][j] = __shfl_sync(0xffffffffu, down, 4 * (2 * c + j));
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
                uint32_t sees[NT][2] = {};
                bool all;
                if constexpr (kList) {
                    const uint32_t s = __shfl_sync(0xffffffffu, loads.seen, stage);
                    all = s == 0xffffffffu;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) sees[nt][0] = sees[nt][1] = s;
                } else {
                    all = t + kSpan <= min(w.t1, w.ctx - a.next_n + 1);
                    if (!all) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const int draft = min((row0 + nt * 8 + 2 * c + j) / a.group, a.next_n - 1);
                                const int limit = min(max(w.ctx - a.next_n + 1 + draft, 0), w.ctx);
                                const int n = min(max(limit - t, 0), kSpan);
                                sees[nt][j] = n == 32 ? 0xffffffffu : (1u << n) - 1;
                            }
                        if (a.next_n > 1) {
                            // tokens that not every position sees: see nan_bytes. This lane's elements of O
                            // are all in one block of 16.
                            uint32_t nan = 0;
                            if (t + lane > w.ctx - a.next_n)
                                nan = clear_nan<D>(ring + stage * S::kSlot + kSpan * (2 * S::kRow + S::kScales) + lane * S::kScales);
                            for (uint32_t left = __ballot_sync(0xffffffffu, nan != 0); left; left &= left - 1) {
                                const int from = __ffs(left) - 1;
                                const uint32_t bits = __shfl_sync(0xffffffffu, nan, from);
                                if (!((bits >> (D == 128 ? g : g / 2)) & 1)) continue;
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                    for (int j = 0; j < 2; ++j)
                                        if ((sees[nt][j] >> from) & 1)
#pragma unroll
                                            for (int i = 0; i < kTiles; ++i) o[nt][i][j] = o[nt][i][j + 2] = kNan;
                            }
                            __syncwarp();
                        }
                    }
                }
                loads.issue(a, ring + load_stage * S::kSlot, load_stage);
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
                    if (!all) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (!((sees[nt][i & 1] >> (half * 16 + (i >> 1) * 8 + g)) & 1)) x[nt][i] = -INFINITY;
                    }
                    // ---- y: the scores in base 2, less m
                    float y[NT][4];
                    auto scores = [&](int nt, float m0, float m1) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            y[nt][i] = fmaf(x[nt][i], fac[nt][i & 1], i & 1 ? -m1 : -m0);
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
                                to = fmaxf(to - kRoom, m[nt][j]);
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
            int64_t slot;
            const bool whole = row_is_whole<kList>(a, r, slot);
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
                const int rr = i / (D / 4), d = i % (D / 4) * 4, row = row0 + rr;
                if (row >= a.rows) break;
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
                    const int n = kList ? draft : row / a.group;
                    const int64_t at = ((int64_t)w.b * a.next_n + n) * a.heads + hk * a.group + (kList ? row : row - n * a.group);
                    const float inv = total == 0.f ? 0.f : 1.f / total;
                    *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + at * D + d) =
                        make_uint2(pack<T>(v.x * inv, v.y * inv), pack<T>(v.z * inv, v.w * inv));
                    if (a.lse != nullptr && d == 0) a.lse[at] = lse_of(top, raw);
                } else {
                    const int64_t at = (slot * a.kv_heads + hk) * a.rows + row;
                    *reinterpret_cast<float4*>(a.part_o + at * D + d) = v;
                    if (d == 0) *reinterpret_cast<float4*>(a.part_ml + at * 4) = make_float4(top, total, raw, 0.f);
                }
            }
            __syncthreads();

            next_row<kList>(a, r);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } while (!last);
    if constexpr (!kList) {
        if (blockIdx.y == 0) dense_extras<D>(a, warp, kWarps, lane);
    }
}

// ---------------------------------------------------------------- combine
// Joins the partial results: `wpr` warps a query row, a lane takes D / 32 elements of
// it. A CTA has `passes` times 8 / wpr rows of one item and kv head, after one look for
// the ranges that hold their partials (178 rows with 71 query rows each, 2 kv heads,
// two thirds of them split: 62 -> 57 us for the call against a look for every row).
constexpr int kCombineThreads = 256;
constexpr int64_t kCombineCtas = 148 * 8;

template <int D, typename T, bool kList>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const AttentionArgs a, int wpr, int passes) {
    constexpr int kV = D / 32;  // elements of a lane
    __shared__ float part[8][D + 4];
    ptx::griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows_per_cta = 8 / wpr, sub = warp % wpr;
    const int hk = blockIdx.y % a.kv_heads;
    const int item = blockIdx.x;
    const int64_t per_item = (int64_t)a.kv_heads * a.rows;

    // ranges first .. last (parts of the list) hold the rows' partials
    int first = 0, last = -1, parts = 0, first_cta = 0;
    // the part that the head's range k begins at
    auto range_start = [&](int k) {
        if (a.kv_heads * parts <= a.deal) return k;  // no CTA has two pairs
        return k == 0 ? 0 : min(parts, first_pair(a, parts, first_cta + k) - hk * parts);
    };
    if constexpr (kList) {
        last = a.splits - 1;
    } else {
        // the head's ranges that begin at or before the row's first token, and at or
        // before its last: warp-wide counts (they ascend)
        const int ctx = row_ctx(a, item);
        if (ctx == 0) return;
        parts = parts_with_rows(a, lane);
        // the CTA that has the head's first pair: the last that begins at or before it
        first_cta = parts == 0 ? 0 : (int)(((int64_t)(hk * parts + 1) * a.deal - 1) / ((int64_t)a.kv_heads * parts));
        int at = 0, upto = 0;
        for (int k = lane;; k += 32) {
            const int i = range_start(k);
            if (i >= parts) break;
            const int b = __ldg(a.schedule + 2 * i), u = __ldg(a.schedule + 2 * i + 1);
            at += b < item || (b == item && u <= 0);
            upto += b < item || (b == item && (int64_t)u * kUnit < ctx);
        }
        at = __reduce_add_sync(0xffffffffu, at);
        upto = __reduce_add_sync(0xffffffffu, upto);
        first = max(at - 1, 0);
        last = upto - 1;
        if (last <= first) return;
    }

    for (int pass = 0; pass < passes; ++pass) {
        const int r = ((blockIdx.y / a.kv_heads) * passes + pass) * rows_per_cta + warp / wpr;
        const int64_t hr = (int64_t)hk * a.rows + r;
        float top = kUnset, total = 0.f, raw = 0.f, v[kV] = {};
        auto join = [&](float m, float l, float l_raw, const float* p) {
            const float to = fmaxf(top, m), keep = ex2(top - to), by = ex2(m - to);
            top = to;
            total = total * keep + l * by;
            raw = raw * keep + l_raw * by;
#pragma unroll
            for (int k = 0; k < kV; ++k) v[k] = v[k] * keep + p[k] * by;
        };
        if (r < a.rows) {
            for (int i = first + sub; i <= last; i += wpr) {
                const int64_t slot = kList ? (int64_t)item * a.splits + i : 2 * (int64_t)range_start(i) + (i == first);
                const int64_t at = slot * per_item + hr;
                const float4 ml = *reinterpret_cast<const float4*>(a.part_ml + at * 4);
                float p[kV];
#pragma unroll
                for (int k = 0; k < kV; ++k) p[k] = a.part_o[at * D + lane * kV + k];
                join(ml.x, ml.y, ml.z, p);
            }
        }
        if (wpr > 1) {
            if (pass > 0) __syncthreads();
#pragma unroll
            for (int k = 0; k < kV; ++k) part[warp][lane * kV + k] = v[k];
            if (lane == 0) {
                part[warp][D] = top;
                part[warp][D + 1] = total;
                part[warp][D + 2] = raw;
            }
            __syncthreads();
            if (sub != 0) continue;
            for (int i = 1; i < wpr; ++i) {
                const float* o = part[warp + i];
                join(o[D], o[D + 1], o[D + 2], o + lane * kV);
            }
        }
        if (r >= a.rows) continue;
        const int n = kList ? item % a.next_n : r / a.group;
        const int b = kList ? item / a.next_n : item;
        const int64_t at = ((int64_t)b * a.next_n + n) * a.heads + hk * a.group + (kList ? r : r - n * a.group);
        const float inv = total == 0.f ? 0.f : 1.f / total;
        uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + at * D + lane * kV);
#pragma unroll
        for (int k = 0; k < kV; k += 2) out[k / 2] = pack<T>(v[k] * inv, v[k + 1] * inv);
        if (a.lse != nullptr && lane == 0) a.lse[at] = lse_of(top, raw);
    }
}

template <int D, int NT, typename T, bool kList, bool kSmall>
cudaError_t launch_narrow(int device, const AttentionArgs& a, void* stream, bool pdl) {
    using S = Shape<D, NT, kSmall>;
    static uint32_t done[64];
    const cudaError_t e = allow_smem(attention_kernel<D, NT, T, kList, kSmall>, device, S::kSmem, done);
    if (e != cudaSuccess) return e;
    const int groups = (a.rows + S::kRows - 1) / S::kRows;
    const int64_t x = kList ? (int64_t)a.batch * a.next_n * a.splits * a.kv_heads : a.deal;
    return launch_pdl(attention_kernel<D, NT, T, kList, kSmall>, dim3((unsigned)x, groups), dim3(S::kThreads),
                      S::kSmem, stream, pdl, a);
}

template <int D, typename T, bool kList>
cudaError_t launch_as(int device, AttentionArgs a, void* stream, bool pdl) {
    // Dense: with as many (head, part) pairs as small CTAs fit, those; rows begin and end
    // in one CTA while the others compute (8 kv heads: 64 rows of 1024 to 8192 tokens 96 ->
    // 88 us, 157 rows of 48 to 299 51 -> 26; 118 rows of one token, 4 kv heads, 22 -> 10;
    // but 8 rows of 30000 to 60000, 8 kv heads, 96 -> 101).
    a.deal = a.num_ctas;
    if (!kList && a.rows <= 16) {
        const int fit = 148 * (a.rows <= 8 ? Shape<D, 1, true>::kPerSm : Shape<D, 2, true>::kPerSm);
        a.small = (int64_t)a.kv_heads * a.num_ctas >= fit;
        if (a.small) a.deal = fit;
    }
    cudaError_t e;
    if (a.rows > 16 && !(kList && a.small)) {
        e = launch_wide<D, T, kList>(device, a, stream, pdl);
    } else if (a.small) {
        e = a.rows <= 8 ? launch_narrow<D, 1, T, kList, true>(device, a, stream, pdl)
                        : launch_narrow<D, 2, T, kList, true>(device, a, stream, pdl);
    } else {
        e = a.rows <= 8 ? launch_narrow<D, 1, T, kList, false>(device, a, stream, pdl)
                        : launch_narrow<D, 2, T, kList, false>(device, a, stream, pdl);
    }
    // nothing to join: whole lists, or a table whose rows hold one unit of the schedule at
    // most (4 rows of 22 to 200 tokens, 8 kv heads: 15.5 -> 13.4 us a call)
    if (e != cudaSuccess || (kList ? a.splits == 1 : a.max_pages << a.ps_shift <= kUnit)) return e;
    const int64_t items = kList ? (int64_t)a.batch * a.next_n : a.batch;
    const int64_t pairs = items * a.kv_heads;
    const int64_t parts = kList ? a.splits : (a.deal + pairs - 1) / pairs + 1;
    int wpr = 1;
    while (wpr < 8 && wpr * 4 < parts) wpr *= 2;
    // as many CTAs as fit at once (8 to an SM), each with more rows where there are more
    int64_t chunks = (a.rows * wpr + 7) / 8;
    const int passes = (int)std::min(chunks, (pairs * chunks + kCombineCtas - 1) / kCombineCtas);
    chunks = (chunks + passes - 1) / passes;
    return launch_pdl(combine_kernel<D, T, kList>, dim3((unsigned)items, (unsigned)(a.kv_heads * chunks)),
                      dim3(kCombineThreads), 0, stream, pdl, a, wpr, passes);
}

template <int D, typename T>
cudaError_t launch_rows(int device, const AttentionArgs& a, void* stream, bool pdl) {
    return a.topk > 0 ? launch_as<D, T, true>(device, a, stream, pdl)
                      : launch_as<D, T, false>(device, a, stream, pdl);
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
