// Device pieces that the attention kernels share: number formats, the walk over a
// CTA's ranges of rows, and the asynchronous copies of 32 tokens at a time.
#pragma once
#include "common.cuh"

#include "attention.cuh"

namespace mqa {

constexpr int kSpan = 32;         // tokens of a ring slot
constexpr float kUnset = -1e30f;  // m of a row that has seen no token
constexpr float kNan = __builtin_nanf("");
// p = 2^(x - m) is rounded to f16 for the second product: 11 bits down to 2^-14, an
// absolute 2^-25 below. That is off by 2^-11 of each p at most, either way, which in the
// result is less than its own rounding to bf16 and about as much as that to f16; p in two
// f16 parts would double the second product. m is raised when an x exceeds it by kSlack (p
// stays below f16's 65504), and then to kRoom below the row's maximum: the largest p is at
// least 2^kRoom, so that a p keeps its 11 bits down to 2^-21 of the largest, and 2^17 tokens
// whose p vanish (2^-32 of it each) held at most 2^-15 of the row. With m raised to the maximum
// itself that was 2^-8 (and 1 to 4 % less time: 32 rows of two positions and 64 heads, 32768 to
// 131072 tokens, 239 us for 241 to 249; 128 lists of 2048, 32 heads, 28.1 for 28.8).
constexpr float kSlack = 15.99f, kRoom = 7.f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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

// The same of something that is there.
template <int N>
__device__ __forceinline__ void copy_async_all(uint32_t dst, const void* src) {
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
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

// NaN scales in a row's last next_n - 1 tokens, which not every position sees: all positions
// share the V operand, and 0 times NaN is NaN. Such scales of V are taken as 0, and the 16
// elements that they would have made NaN are made so in the results of the positions that
// see the token. (Long drafts of 241 us: 1 % more.)
// A bit for each of the four e4m3 bytes that is NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
    const uint32_t m = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
    return (m >> 7 | m >> 14 | m >> 21 | m >> 28) & 15u;
}

// Sets the NaN scales of a token in shared memory to 0; a bit for each.
template <int D>
__device__ __forceinline__ uint32_t clear_nan(uint32_t at) {
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        const uint32_t w = lds32(at + 4 * i), n = nan_bytes(w);
        if (n != 0) {
            const uint32_t bytes = ((n & 1) | (n & 2) << 7 | (n & 4) << 14 | (n & 8) << 21) * 255u;
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 4 * i), "r"(w & ~bytes) : "memory");
            bits |= n << (4 * i);
        }
    }
    return bits;
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

// The same where a lane reads its own token's codes, 16 bytes at a time.
template <int D>
__device__ __forceinline__ uint32_t tile_at(uint32_t t, uint32_t o) {
    if constexpr (D == 128)
        return t * 64 + (o ^ ((t << 3) & 48));
    else
        return t * 32 + (o ^ ((t << 2) & 16));
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

__device__ __forceinline__ int row_ctx(const AttentionArgs& a, int b) {
    return clamp_len(a.status, __ldg(a.context_lens + b), a.max_pages << a.ps_shift);
}

// Dense: the first row at or after w.b that has tokens in this CTA's range,
// starting at unit u0 of row w.b. False: none left.
__device__ __forceinline__ bool settle(const AttentionArgs& a, Walk& w, int u0) {
    while (w.b < a.batch && (w.b < w.last_b || (w.b == w.last_b && u0 < w.last_u))) {
        w.ctx = row_ctx(a, w.b);
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

// The parts of the schedule that the CTAs of a dense launch take: with Hk kv heads the
// (head, part) pairs of the parts that have rows are dealt in order, evenly, over the
// CTAs, so that a CTA walks neighbouring parts of one head as one range, rows are cut
// once a CTA and head at most, and batches with fewer rows than parts still use every
// CTA (26 rows of at most 7 tokens, 8 kv heads: 25 -> 11 us, 8 with small CTAs).
// The first pair of CTA c, of `parts` parts that have rows.
__device__ __forceinline__ int first_pair(const AttentionArgs& a, int parts, int c) {
    if (parts == a.deal) return c * a.kv_heads;
    return (int)((int64_t)c * a.kv_heads * parts / a.deal);
}

// A warp's count of the parts that begin at a row of the batch: the first ones. One kv
// head: all parts, which makes pair i CTA i's.
__device__ __forceinline__ int parts_with_rows(const AttentionArgs& a, int lane) {
    if (a.kv_heads == 1 || __ldg(a.schedule + 2 * (a.num_ctas - 1)) < a.batch) return a.num_ctas;
    int n = 0;
    for (int i = lane; i < a.num_ctas; i += 32) n += __ldg(a.schedule + 2 * i) < a.batch;
    return __reduce_add_sync(0xffffffffu, n);
}

// One range of rows of one kv head (dense), or one part of one list.
struct Range {
    Walk w;
    int hk, part, draft;
    bool more;
};

// Dense: opens the range at (head, part) pair `pair` of the CTA's, moves `pair` behind
// it, and says in `last` if it is the CTA's last.
// Selected: the part of the list that CTA x of the grid takes.
template <bool kList>
__device__ __forceinline__ Range open_range(const AttentionArgs& a, int x, int parts, int& pair, bool& last) {
    Range r{};
    Walk& w = r.w;
    if constexpr (kList) {
        r.hk = x % a.kv_heads;
        const int y = x / a.kv_heads;
        w.item = y / a.splits;
        r.part = y - w.item * a.splits;
        w.b = w.item / a.next_n;
        r.draft = w.item - w.b * a.next_n;
        const int full = row_ctx(a, w.b);
        w.ctx = min(max(full - a.next_n + 1 + r.draft, 0), full);
        const int per = ((a.topk + a.splits - 1) / a.splits + kSpan - 1) / kSpan * kSpan;
        w.t0 = min(a.topk, r.part * per);
        w.t1 = min(a.topk, w.t0 + per);
        w.last_b = w.b;
        w.last_u = 0;
        r.more = last = true;
    } else {
        r.draft = 0;
        const int end = first_pair(a, parts, x + 1);
        last = true;
        if (pair >= end) return r;  // no pair at all
        r.hk = pair / parts;
        r.part = pair - r.hk * parts;
        const int n = min(parts - r.part, end - pair);
        pair += n;
        last = pair == end;
        w.b = max(__ldg(a.schedule + 2 * r.part), 0);
        const int u0 = max(__ldg(a.schedule + 2 * r.part + 1), 0);
        w.last_b = __ldg(a.schedule + 2 * (r.part + n));
        w.last_u = __ldg(a.schedule + 2 * (r.part + n) + 1);
        r.more = settle(a, w, u0);
    }
    return r;
}

// Moves a range to its next row.
template <bool kList>
__device__ __forceinline__ void next_row(const AttentionArgs& a, Range& r) {
    if constexpr (kList) {
        r.more = false;
    } else {
        ++r.w.b;
        r.more = settle(a, r.w, 0);
    }
}

// Where the row's result goes: complete, or which partial slot.
template <bool kList>
__device__ __forceinline__ bool row_is_whole(const AttentionArgs& a, const Range& r, int64_t& slot) {
    if constexpr (kList) {
        slot = (int64_t)r.w.item * a.splits + r.part;
        return a.splits == 1;
    } else {
        slot = 2 * r.part + (r.w.t0 > 0 ? 0 : 1);
        return r.w.t0 == 0 && r.w.t1 == r.w.ctx;
    }
}

// What every dense launch does besides: the schedule's check in validate mode, and
// the results of rows without tokens, which are in no CTA's range.
// `warp` of the `warps` that do it.
template <int D>
__device__ __forceinline__ void dense_extras(const AttentionArgs& a, int warp, int warps, int lane) {
    if ((a.status.flags & MQA_FLAG_VALIDATE) && warp == 0) {
        KernelArgs ka{};
        ka.context_lens = a.context_lens;
        ka.schedule = a.schedule;
        ka.status = a.status.caller;
        ka.lib_status = a.status.lib;
        ka.batch = a.batch;
        ka.num_ctas = a.num_ctas;
        for (int i = blockIdx.x; i < a.num_ctas; i += gridDim.x) check_schedule(ka, i, lane);
    }
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
        if (__ldg(a.context_lens + b) > 0) continue;
        const int64_t o = (int64_t)b * a.next_n * a.heads;
        for (int j = warp * 32 + lane; j < a.next_n * a.heads * (D / 8); j += warps * 32)
            reinterpret_cast<uint4*>(a.out)[o * (D / 8) + j] = make_uint4(0, 0, 0, 0);
        if (a.lse != nullptr)
            for (int j = warp * 32 + lane; j < a.next_n * a.heads; j += warps * 32) a.lse[o + j] = -INFINITY;
    }
}

// A warp's loads, running ahead of its computation: kStep tokens from one span of 32
// to the warp's next, `off` its place in them. kTile: every warp has a span wherever
// the step has a token (zeros behind the row); else only where the span has one.
template <int D, int kStep, bool kList, bool kTile>
struct SpanLoader {
    static constexpr int kRow = D / 2, kScales = D / 16;
    Range r;
    const int32_t* list;   // selected: the row's token list
    const int32_t* table;  // the row's block table
    uint32_t head_at;
    int lane, off, pos;
    // This lane's token of the span to be copied next, found a step ahead: the token
    // (-1 for none), its page as loaded (not looked at before the copy, so that nothing
    // waits for the load), whether there is a span at all, and whether it is whole: 32
    // neighbouring tokens of one page.
    int tok, page;
    bool any, whole;
    int ahead;      // selected: the list's entry for the span after that, as loaded
    uint32_t seen;  // selected: lane s keeps the mask of the visible tokens in ring slot s

    __device__ __forceinline__ void open(const AttentionArgs& a, const Range& range, int lane_, int off_) {
        r = range;
        lane = lane_;
        off = off_;
        pos = r.w.t0 + off;
        list = kList ? a.indices + (int64_t)r.w.item * a.topk : nullptr;
        table = a.block_table + (int64_t)min(r.w.b, a.batch - 1) * a.max_pages;
        head_at = (uint32_t)r.hk * a.page_size * (kRow + kScales);
        seen = 0;
        if constexpr (kList) ahead = pos + lane < r.w.t1 ? __ldg(list + pos + lane) : -1;
        resolve(a);
    }

    __device__ __forceinline__ void resolve(const AttentionArgs& a) {
        any = false;
        tok = -1;
        while (r.more && (kTile ? pos - off : pos) >= r.w.t1) {
            next_row<kList>(a, r);
            pos = r.w.t0 + off;
            table = a.block_table + (int64_t)min(r.w.b, a.batch - 1) * a.max_pages;
        }
        if (!r.more) return;
        any = true;
        const int t = pos + lane;
        whole = !kList && pos + kSpan <= r.w.t1 && a.page_size >= kSpan;
        pos += kStep;
        if constexpr (kList) {
            tok = ahead >= 0 && ahead < r.w.ctx ? ahead : -1;
            ahead = pos + lane < r.w.t1 ? __ldg(list + pos + lane) : -1;
        } else {
            tok = t < r.w.t1 ? t : -1;
        }
        page = __ldg(table + (max(tok, 0) >> a.ps_shift));
    }

    // Copies the span's codes and scales of `caches` caches (K, then V, to slots
    // `stride` apart) into ring slot `base`: rows of codes, scales `scales` behind
    // them; zeros where there is no token.
    template <int kCaches>
    __device__ __forceinline__ void copy(const AttentionArgs& a, const uint8_t* c0, const uint8_t* c1, uint32_t base,
                                         uint32_t stride, uint32_t scales, uint32_t scale_stride) {
        constexpr int kPieces = kRow / 16;  // 16-byte pieces of a token's codes
        auto place = [](int t, int o) { return kTile ? tile_at<D>(t, o) : code_at<D>(t, o); };
        if ((uint32_t)page >= (uint32_t)a.num_pages) {
            if (tok >= 0) report_checked(a.status, MQA_STATUS_BAD_PAGE);
            page = page < 0 ? 0 : a.num_pages - 1;
        }
        const uint32_t in = (uint32_t)max(tok, 0) & (a.page_size - 1);
        const int64_t at = (int64_t)page * a.page_bytes + head_at;  // of the page and head
        const int64_t sc = at + (a.page_size * kRow + in * kScales);
        if (whole) {
            // one stretch of one page: this lane's piece i is 512 i bytes behind its first
            const int64_t from = at + (in - lane) * kRow + lane * 16;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const uint32_t to = base + place((i * 32 + lane) / kPieces, (i * 32 + lane) % kPieces * 16);
                copy_async_all<16>(to, c0 + from + i * 512);
                if (kCaches == 2) copy_async_all<16>(to + stride, c1 + from + i * 512);
            }
            copy_async_all<kScales>(base + scales + lane * kScales, c0 + sc);
            if (kCaches == 2) copy_async_all<kScales>(base + scales + scale_stride + lane * kScales, c1 + sc);
        } else {
            const int64_t mine = tok >= 0 ? at + in * kRow : -1;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int p = i * 32 + lane, t = p / kPieces, o = (p % kPieces) * 16;
                const int64_t from = __shfl_sync(0xffffffffu, mine, t);
                const uint32_t to = base + place(t, o);
                copy_async<16>(to, c0 + max(from, (int64_t)0) + o, from >= 0);
                if (kCaches == 2) copy_async<16>(to + stride, c1 + max(from, (int64_t)0) + o, from >= 0);
            }
            copy_async<kScales>(base + scales + lane * kScales, c0 + sc, tok >= 0);
            if (kCaches == 2) copy_async<kScales>(base + scales + scale_stride + lane * kScales, c1 + sc, tok >= 0);
        }
    }

    // One cache's span: codes, then scales. One copy group, empty if there is no span.
    __device__ __forceinline__ void issue_one(const AttentionArgs& a, const uint8_t* cache, uint32_t base) {
        if (any) copy<1>(a, cache, nullptr, base, 0, kSpan * kRow, 0);
        ptx::cp_async_commit();
        resolve(a);
    }

    // Both caches' (ring slot number `stage`): K codes, V codes, K scales, V scales.
    __device__ __forceinline__ void issue(const AttentionArgs& a, uint32_t base, int stage) {
        if (any) {
            copy<2>(a, a.k, a.v, base, kSpan * kRow, 2 * kSpan * kRow, kSpan * kScales);
            if constexpr (kList) {
                const uint32_t m = __ballot_sync(0xffffffffu, tok >= 0);
                if (lane == stage) seen = m;
            }
        }
        ptx::cp_async_commit();
        resolve(a);
    }
};

// The power of two that a row of q is multiplied by (its bits `most`: the largest |x|
// of a bf16 row), so that its largest element lies in [2^14, 2^15), and what undoes it.
__device__ __forceinline__ void q_power(uint32_t most, float& up, float& down) {
    // kept where both are normal fp32
    const int ex = most == 0 ? 14 : max((int)(most >> 7) - 127, -100);
    up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
    down = __uint_as_float((uint32_t)(127 - 14 + ex) << 23);
}

}  // namespace mqa
