// Attention over the FP4 cache for many query rows a kv head (17 to 128): both
// products on the 5th-generation tensor core.
//
// A tile is 128 tokens. S = Q K^T (M = 128 query rows, N = 128 tokens) with Q and K,
// dequantised to f16, in shared memory; P = 2^(S - m) goes back to TMEM, and
// O += P V with P as the A operand from TMEM and V in shared memory (tokens are the
// contraction, so V is the MN-major operand and needs no transpose). Rows are TMEM
// lanes: a thread has a row, and maxima and sums need no exchange. With 64 rows or
// fewer (32 or fewer), the rows stand in TMEM twice (four times), and each copy takes
// its half (quarter) of every tile's tokens, with zeros in the other columns of P:
// all warps have work, and the copies are summed at the end of the row.
//
// Warps: 0 issues S and 1 O; 2 and 3 fill the results of rows without tokens; 4-7 and
// 8-11 softmax (a warp has 32 rows; the two groups take tiles in turn, so that one
// group's exponentials run while the other's products do), 12-15 dequantise K and
// 16-19 V (32 tokens of each tile, through rings of asynchronous copies of their own:
// bulk copies of whole pages by warps 2 and 3 instead took 239 us for 228). K and V
// have two buffers of f16, S three.
//
// m is raised, by whole numbers so that every rescaling is exact, only when the p of
// 32 tokens sum to more than kMost (so that none is outside f16), and then to kRoom
// below the largest score. A tile is computed with the m that its
// group knows; at its end the group learns the m that O has by then (`ref`, settled
// in turn, tile by tile) and scales whichever of P and O is behind, which is rare. So
// a tile needs one pass over S, and the groups wait for each other only where one
// of them is late. All waits are bounded: on a timeout the status word gets
// MQA_STATUS_TIMEOUT and every role leaves.
//
// Measured: 32 rows of 32768 to 131072 tokens, two positions of 64 heads, one kv head,
// D = 128: 240 us for 380 MB and 172 GFLOP; the products need 0.43 of that at the bf16
// peak. What bounds it is latency: a tile's chain (dequantise, S, softmax, P,
// O) takes longer than its 1.7 us share, with two tiles in each stage; leaving out any
// one of its parts (the exponentials, the conversions, half of the products, the
// copies) saves 10 to 20 %. A row of its own costs about 8 us besides: q, the first
// tile's chain and the result do not overlap the row before.
#include "attention_walk.cuh"
#include "host.cuh"

namespace mqa {
namespace {

constexpr int kTokens = 128;       // of a tile
constexpr int kSoftmaxWarps = 8;
constexpr int kDequantWarps = 4;   // for each of K and V
// First warps: 0 issues S, 1 issues O (the lowest numbers, since the hardware prefers
// older warps and everything waits for these two; 2 and 3 keep the others' places
// in their quarters of TMEM), then the softmax and the dequantising warps.
constexpr int kMmaWarp = 0, kSoftmaxWarp = 4, kDequantWarp = kSoftmaxWarp + kSoftmaxWarps;
constexpr int kWideThreads = 32 * (kDequantWarp + 2 * kDequantWarps);
constexpr float kMost = 65504.f;
// Registers of a thread: at launch (what the compiler gives 640 threads; the launch checks
// it), and of the roles' four-warp groups afterwards, which together take no more, so that
// the softmax groups' request is met once the others have given theirs back (32 rows of
// two positions and 64 heads, 32768 to 131072 tokens: 227 -> 222 us). The walk, the copies
// and the last tokens' scales do not fit 64 in the dequantising warps (5 rows of up to 79593
// tokens, three positions of 48 heads on 8, D = 64: 104 us, 101.5 with 72); with 80, and 136
// for the softmax, 128 lists of 2048 take 34.5 us for 28.2.
constexpr int kRegsLaunch = 96, kRegsMma = 48, kRegsSoftmax = 144, kRegsDequant = 72;
static_assert(kRegsMma + 2 * kRegsSoftmax + 2 * kRegsDequant <= kWideThreads / 128 * kRegsLaunch, "registers");
constexpr uint64_t kTimeoutNs = 2000000000ull;
// TMEM columns: three S buffers of 128 (P over their second halves), O. With three, S
// is two tiles ahead and no group waits for a product; Q is in shared memory for it.
constexpr int kBufS = 3, kColP = 64, kColO = 128 * kBufS, kColumns = 512;
constexpr uint32_t kTmem = 0;  // where an allocation of all 512 columns begins

template <int D>
struct Wide {
    static constexpr int kRow = D / 2, kScales = D / 16;
    static constexpr int kSlot = kSpan * (kRow + kScales);
    static constexpr int kStages = 3;
    static constexpr int kBuf = kTokens * D * 2;  // a tile of K or V: [D / 64][128 tokens][64] f16, 128-byte swizzle
    static constexpr int kK = 0, kV = 2 * kBuf, kQ = 4 * kBuf;
    // [2][128][32] fp32: where copies of rows are summed; for D = 128 in Q's place, which
    // is free then (and a group's part of it is what the same warps write next)
    static constexpr int kSum = D == 128 ? kQ : kQ + kBuf;
    static constexpr int kRing = kSum + 2 * 128 * 32 * 4;
    static constexpr int kExch = kRing + 2 * kDequantWarps * kStages * kSlot;  // [2][2][128] fp32
    static constexpr int kRef = kExch + 2 * 2 * 128 * 4;                       // [128] fp32: m of each row
    static constexpr int kTot = kRef + 128 * 4;                                // [2][128] fp32: sums of p
    static constexpr int kBars = kTot + 2 * 128 * 4;
    static constexpr int kSmem = kBars + 384 + 1024;  // slack for aligning the base
    static_assert(kSmem <= 232448, "more shared memory than a CTA can have");
};

struct Bars {
    uint64_t k_full[2], v_full[2];  // the dequantising warps arrive
    uint64_t s_full[kBufS];         // S computed (and its K buffer free)
    uint64_t p_full[kBufS];         // a group's warps arrive: P written
    uint64_t s_free[kBufS];         // P used
    uint64_t pv_done[2];            // V used
    uint64_t q_full;                // the softmax warps arrive: Q is in shared memory
    uint64_t turn[4][2];            // a row quarter's m is settled for the tile
    uint64_t pair[4];               // the two warps of a row quarter exchange values
    uint64_t copies[2];             // a group's warps: at the row's end, where rows stand in copies
    uint64_t drain[2];
    // the NaN scales of V in the tokens that not every position of a row sees (nan_bytes), by
    // the row's number modulo 4: written by the warps that dequantise V, read at the row's end
    uint32_t nan[4][4];
    int32_t abort;
    uint32_t tmem;
};
static_assert(sizeof(Bars) <= 384, "barriers");

// The warp's arrival: by the lane whose `lead` is 1, without a branch.
__device__ __forceinline__ void arrive(uint32_t lead, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}"
        ::"r"(ptx::smem_u32(bar)), "r"(lead) : "memory");
}

// The whole four-warp group comes here.
template <int kRegs>
__device__ __forceinline__ void set_registers() {
    if constexpr (kRegs > kRegsLaunch)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Waits for phase `parity`, by one thread. False: give up. A wait tells a phase from
// the one before it, not from the one before that: who waits must know that the
// barrier's phase before the awaited one is over. Each wait below has that from an
// earlier wait of the same warp on the same barrier, or from one that its comment names.
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, Bars* bars, const StatusWords& st) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer();
    volatile int32_t* abort = &bars->abort;
    while (!ptx::mbar_try_wait_sleep(bar, parity, kWaitSliceNs)) {
        if (*abort) return false;
        if (ptx::globaltimer() - t0 > kTimeoutNs) {
            report(st, MQA_STATUS_TIMEOUT);
            *abort = 1;
            return false;
        }
    }
    return true;
}

// The same for a warp, which stays together: every lane looks once, lane 0 waits.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, Bars* bars,
                                           const StatusWords& st, int lane) {
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
    bool ok = true;
    if (lane == 0) ok = wait_one(bar, parity, bars, st);
    return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

// D[tmem] (+)= A[tmem] * B[smem], f16 operands, issued by the lane whose `lead` is 1.
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead) : "memory");
}

// The same with A from shared memory.
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead) : "memory");
}

__device__ __forceinline__ void commit(uint32_t lead, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        ::"r"(ptx::smem_u32(bar)), "r"(lead) : "memory");
}

__device__ __forceinline__ void fence_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// 32 or 16 consecutive columns of this thread's TMEM lane, waited for.
__device__ __forceinline__ void tmem_read32(uint32_t taddr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19,"
        "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}"
        ", [%32];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]),
          "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]),
          "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]),
          "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
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

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
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
    const uint32_t line = (tile + row * 128) | ((row & 7) << 4);  // a 16-byte unit's place: its number, xor row % 8
    const uint32_t from = codes + tile_at<D>(lane, 0);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
        const uint4 v = lds128(from ^ (j * 16));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        const uint32_t h = e4m3x2_to_f16(sc[j / 2] >> ((j & 1) * 16));
        const uint32_t s[2] = {__byte_perm(h, h, 0x1010), __byte_perm(h, h, 0x3232)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t f[4];
            e2m1_to_f16(w[i], f);
            const int u = 4 * j + i;
            sts128((line ^ ((u & 7) << 4)) + (u >> 3) * (kTokens * 128), mul_f16x2(f[0], s[i / 2]),
                   mul_f16x2(f[1], s[i / 2]), mul_f16x2(f[2], s[i / 2]), mul_f16x2(f[3], s[i / 2]));
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
    float* ref = reinterpret_cast<float*>(smem + W::kRef);
    Bars* bars = reinterpret_cast<Bars*>(smem + W::kBars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == kMmaWarp) ptx::tmem_alloc(&bars->tmem, kColumns);
    if (warp == kSoftmaxWarp) {
        // a lane a barrier
        uint64_t* bar = nullptr;
        uint32_t arrivals = 1;
        if (lane < 2) bar = &bars->k_full[lane], arrivals = kDequantWarps;
        else if (lane < 4) bar = &bars->v_full[lane - 2], arrivals = kDequantWarps;
        else if (lane < 6) bar = &bars->pv_done[lane - 4];
        else if (lane < 9) bar = &bars->s_full[lane - 6];
        else if (lane < 12) bar = &bars->p_full[lane - 9], arrivals = kSoftmaxWarps / 2;
        else if (lane < 15) bar = &bars->s_free[lane - 12];
        else if (lane < 23) bar = &bars->turn[0][0] + (lane - 15);
        else if (lane < 27) bar = &bars->pair[lane - 23], arrivals = 2;
        else if (lane < 29) bar = &bars->copies[lane - 27], arrivals = kSoftmaxWarps / 2;
        else if (lane < 31) bar = &bars->drain[lane - 29];
        else bar = &bars->q_full, arrivals = kSoftmaxWarps;
        ptx::mbar_init(bar, arrivals);
        if (lane == 0) bars->abort = 0;
        ptx::fence_mbar_init();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    constexpr uint32_t tmem = kTmem;

    ptx::griddep_wait();

    const int parts = kList ? 1 : parts_with_rows(a, lane);
    int pair = kList ? 0 : first_pair(a, parts, blockIdx.x);  // dense: the next (head, part) pair
    bool last = true;
    // Tiles so far: buffers and phases go by their number. Tile i is in S buffer i % 3,
    // for the i / 3-th time.
    int it = 0;
    bool ok = true;

    if (warp < kSoftmaxWarp) set_registers<kRegsMma>();
    if (warp >= kDequantWarp) {
        set_registers<kRegsDequant>();
        // ------------------------------------------------------------ dequantise
        const bool is_v = warp >= kDequantWarp + kDequantWarps;
        const int dw = (warp - kDequantWarp) & 3, row = dw * kSpan + lane;
        const uint32_t ring = base + W::kRing + (warp - kDequantWarp) * (W::kStages * W::kSlot);
        const uint32_t tiles = base + (is_v ? W::kV : W::kK);
        uint64_t* const full = is_v ? bars->v_full : bars->k_full;
        uint32_t seg = 0;
        do {
            Range r = open_range<kList>(a, blockIdx.x, parts, pair, last);
            SpanLoader<D, kTokens, kList, true> loads;
            loads.open(a, r, lane, dw * kSpan);
#pragma unroll
            for (int s = 0; s < W::kStages - 1; ++s) loads.issue_one(a, is_v ? a.v : a.k, ring + s * W::kSlot);
            int load_stage = W::kStages - 1, stage = 0;
            while (ok && r.more) {
                const int n = tiles_of(r.w);
                for (int j = 0; j < n; ++j, ++it) {
                    ptx::cp_async_wait<W::kStages - 2>();
                    __syncwarp();
                    loads.issue_one(a, is_v ? a.v : a.k, ring + load_stage * W::kSlot);
                    load_stage = load_stage + 1 == W::kStages ? 0 : load_stage + 1;
                    const uint32_t slot = ring + stage * W::kSlot;
                    stage = stage + 1 == W::kStages ? 0 : stage + 1;
                    const uint32_t b = it & 1;
                    if (it >= 2) {  // the tile before last in this buffer has been used
                        ok = is_v ? wait_phase(&bars->pv_done[b], ((it >> 1) & 1) ^ 1, bars, a.status, lane)
                                  : wait_phase(&bars->s_full[(it - 2) % kBufS], (it - 2) / kBufS & 1, bars, a.status, lane);
                    }
                    if (!ok) break;
                    if constexpr (!kList) {
                        if (is_v && a.next_n > 1) {  // this lane's token: the i-th of those that not every position sees?
                            const int i = r.w.t0 + j * kTokens + row - (r.w.ctx - a.next_n + 1);
                            if (i >= 0 && i < a.next_n - 1)
                                bars->nan[seg & 3][i] = clear_nan<D>(slot + kSpan * W::kRow + lane * W::kScales);
                        }
                    }
                    dequant_row<D>(slot, slot + kSpan * W::kRow, tiles + b * W::kBuf, lane, row);
                    fence_async_smem();
                    __syncwarp();
                    arrive(lane == 0, &full[b]);
                }
                ++seg;
                next_row<kList>(a, r);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
        } while (ok && !last);
    } else if (warp <= kMmaWarp + 1) {
        // ------------------------------------------------------------ MMAs: the warp walks, lane 0 issues
        const bool is_s = warp == kMmaWarp;
        const uint32_t lead = lane == 0;
        constexpr uint32_t id_qk = ptx::instr_desc(0, 0, 128, kTokens);
        constexpr uint32_t id_pv = ptx::instr_desc(0, 0, 128, D) | (1u << 16);  // B is MN-major
        // K-major: 8-token groups 1024 bytes apart; MN-major: those, and 64-element
        // pieces of D kTokens * 128 apart. Addresses are in 16-byte units.
        const uint64_t k0 = ptx::smem_desc(base + W::kK, 16, 1024, ptx::SW_128B);
        const uint64_t q0 = ptx::smem_desc(base + W::kQ, 16, 1024, ptx::SW_128B);
        const uint64_t v0 = ptx::smem_desc(base + W::kV, kTokens * 128, 1024, ptx::SW_128B);
        int seg = 0;
        do {
            Range r = open_range<kList>(a, blockIdx.x, parts, pair, last);
            while (ok && r.more) {
                const int n = tiles_of(r.w);
                if (is_s && n > 0) ok = wait_phase(&bars->q_full, seg++ & 1, bars, a.status, lane);
                for (int j = 0; ok && j < n; ++j, ++it) {
                    const uint32_t b = it & 1, phase = (it >> 1) & 1, sb = it % kBufS, s_phase = it / kBufS & 1;
                    if (is_s) {
                        ok = wait_phase(&bars->k_full[b], phase, bars, a.status, lane) &&
                             wait_phase(&bars->s_free[sb], s_phase ^ 1, bars, a.status, lane);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        const uint64_t kd = k0 + b * (W::kBuf / 16);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            mma_ss(lead, kTmem + sb * 128, q0 + (k >> 2) * (kTokens * 128 / 16) + (k & 3) * 2,
                                   kd + (k >> 2) * (kTokens * 128 / 16) + (k & 3) * 2, id_qk, k > 0);
                        commit(lead, &bars->s_full[sb]);
                    } else {
                        ok = wait_phase(&bars->v_full[b], phase, bars, a.status, lane) &&
                             wait_phase(&bars->p_full[sb], s_phase, bars, a.status, lane);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        const uint64_t vd = v0 + b * (W::kBuf / 16);
#pragma unroll
                        for (int k = 0; k < kTokens / 16; ++k)
                            mma_ts(lead, kTmem + kColO, kTmem + sb * 128 + kColP + k * 8, vd + k * 128, id_pv,
                                   j > 0 || k > 0);
                        commit(lead, &bars->pv_done[b]);
                        commit(lead, &bars->s_free[sb]);
                    }
                }
                next_row<kList>(a, r);
            }
        } while (ok && !last);
        // nothing of this CTA's MMAs is under way when it ends
        commit(lead, &bars->drain[is_s]);
        if (lane == 0) {
            const uint64_t t0 = ptx::globaltimer();
            while (!ptx::mbar_try_wait_sleep(&bars->drain[is_s], 0, kWaitSliceNs))
                if (ptx::globaltimer() - t0 > kTimeoutNs) {
                    report(a.status, MQA_STATUS_TIMEOUT);
                    break;
                }
        }
        __syncwarp();
    } else if (warp >= kSoftmaxWarp) {
        // ------------------------------------------------------------ softmax
        set_registers<kRegsSoftmax>();
        const int q4 = warp & 3, group = (warp - kSoftmaxWarp) >> 2;
        const int blocks = a.rows <= 32 ? 1 : a.rows <= 64 ? 2 : 4;  // of 32 rows; 4 / blocks copies of them
        const int place = q4 * 32 + lane;                 // of this thread in TMEM
        const int row = q4 % blocks * 32 + lane;          // its query row,
        const int copy = q4 / blocks;                     // which copy of it, with columns
        const int chunk0 = copy * blocks, chunk1 = chunk0 + blocks;  // [32 chunk0, 32 chunk1) of a tile
        const bool active = row - lane < a.rows;          // the quarter has query rows
        const uint32_t lanes = tmem + ((uint32_t)(q4 * 32) << 16);
        uint32_t swaps = 0, seg = 0, meets = 0;  // exchanges, rows and meetings so far
        // a meeting of the group's warps
        auto meet = [&]() {
            __syncwarp();
            arrive(lane == 0, &bars->copies[group]);
            return wait_phase(&bars->copies[group], meets++ & 1, bars, a.status, lane);
        };
        // the other group's value for this row
        auto swap = [&](float mine, float& other) {
            float* at = exch + (swaps & 1) * 256;
            at[group * 128 + place] = mine;
            __syncwarp();
            arrive(lane == 0, &bars->pair[q4]);
            const bool got = wait_phase(&bars->pair[q4], swaps & 1, bars, a.status, lane);
            other = at[(group ^ 1) * 128 + place];
            ++swaps;
            return got;
        };
        const bool flip = a.scale_log2 < 0.f;  // a negative scale goes into q, so that the largest score is the largest S
        do {
            Range r = open_range<kList>(a, blockIdx.x, parts, pair, last);
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
                        // ---- this group's half of the row's q, where the MMA reads it
                        uint32_t wds[D / 4];
                        const T* q = static_cast<const T*>(a.q) + (int64_t)w.b * a.q_sb + (int64_t)draft * a.q_sn +
                                     (int64_t)h * a.q_sh + group * (D / 2);
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
                        for (int i = 0; i < D / 16; ++i) {
                            const int u = group * (D / 16) + i;  // 16-byte unit of the row
                            sts128(base + W::kQ + (u >> 3) * (kTokens * 128) + place * 128 + (((u & 7) ^ (place & 7)) << 4),
                                   wds[4 * i], wds[4 * i + 1], wds[4 * i + 2], wds[4 * i + 3]);
                        }
                    }
                    fence_async_smem();
                    ptx::tc_fence_before();
                    __syncwarp();
                    arrive(lane == 0, &bars->q_full);
                }
                fac = fmaxf(fac, 1e-37f);  // a factor of 0 must not make NaN of an invisible column's -inf
                const int it0 = it;
                const uint64_t fac2 = ptx::f32x2_pack(fac, fac);
                // two partial sums of p, relative to m, before its rounding to f16: the lse needs
                // those, and for the result the roundings, 2^-11 of each p either way, matter no
                // less in the products than in the sum
                uint64_t l2 = 0;
                auto scale_l = [&](float by) {
                    float l0, l1;
                    ptx::f32x2_unpack(l2, l0, l1);
                    l2 = ptx::f32x2_pack(l0 * by, l1 * by);
                };
                auto scale_p = [&](uint32_t at, float power) {  // 32 columns of P, by 2^power in two steps within f16
                    ptx::tmem_st_wait();
                    float p[16];
                    tmem_read16(at, p);
                    uint32_t v[16];
                    const float h = ceilf(0.5f * power), b0 = ex2(h), b1 = ex2(power - h);
                    const uint32_t by0 = pack_f16(b0, b0), by1 = pack_f16(b1, b1);
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = mul_f16x2(mul_f16x2(__float_as_uint(p[k]), by0), by1);
                    ptx::tmem_st16(at, v);
                };
                for (int j = (it & 1) ^ group; j < n; j += 2) {
                    const int it = it0 + j;
                    const uint32_t b = group, sb = it % kBufS;
                    const uint32_t s_at = lanes + sb * 128, p_at = s_at + kColP;
                    const int t = w.t0 + j * kTokens;
                    uint32_t see0 = ~0u, see1 = ~0u, see2 = ~0u, see3 = ~0u;  // the columns that the row sees
                    bool all;
                    if constexpr (kList) {
                        auto listed = [&](int i) {
                            const int e = t + i * 32 + lane;
                            const int tok = e < w.t1 ? __ldg(a.indices + (int64_t)w.item * a.topk + e) : -1;
                            return __ballot_sync(0xffffffffu, tok >= 0 && tok < w.ctx);
                        };
                        see0 = listed(0);
                        see1 = listed(1);
                        see2 = listed(2);
                        see3 = listed(3);
                        all = (see0 & see1 & see2 & see3) == ~0u;
                    } else {
                        all = t + kTokens <= min(w.t1, w.ctx - a.next_n + 1);
                        auto upto = [&](int i) {
                            const int k = min(max(limit - t - i * 32, 0), 32);
                            return k == 32 ? ~0u : (1u << k) - 1;
                        };
                        if (!all) {
                            see0 = upto(0);
                            see1 = upto(1);
                            see2 = upto(2);
                            see3 = upto(3);
                        }
                    }
                    ok = wait_phase(&bars->s_full[sb], it / kBufS & 1, bars, a.status, lane);
                    if (!ok) break;
                    if (active) {
                        ptx::tc_fence_after();
                        // P goes over S from the last columns on: those of S that it takes are
                        // read by then. A loop of small code: unrolled, the kernel's roles
                        // together no longer fit the instruction cache.
#pragma unroll 1
                        for (int i = chunk1 - 1; i >= chunk0; --i) {
                            float s[32];
                            uint32_t p[16];
                            uint64_t sum;
                            auto read = [&]() {
                                tmem_read32(s_at + 32 * i, s);
                                if (!all) {
                                    const uint32_t see = i == 0 ? see0 : i == 1 ? see1 : i == 2 ? see2 : see3;
#pragma unroll
                                    for (int k = 0; k < 32; ++k) s[k] = (see >> k) & 1 ? s[k] : -INFINITY;
                                }
                            };
                            auto powers = [&]() {
                                const uint64_t m2 = ptx::f32x2_pack(-m, -m);
                                uint64_t sums[2];
#pragma unroll
                                for (int k = 0; k < 16; ++k) {
                                    float e0, e1;
                                    ptx::f32x2_unpack(ptx::fma_f32x2(ptx::f32x2_pack(s[2 * k], s[2 * k + 1]), fac2, m2), e0, e1);
                                    e0 = ex2(e0);
                                    e1 = ex2(e1);
                                    const uint64_t e2 = ptx::f32x2_pack(e0, e1);
                                    sums[k & 1] = k < 2 ? e2 : add_f32x2(sums[k & 1], e2);
                                    p[k] = pack_f16(e0, e1);
                                }
                                sum = add_f32x2(sums[0], sums[1]);
                            };
                            read();
                            powers();
                            // no p is above the sums: within f16, or m has to rise
                            float sum0, sum1;
                            ptx::f32x2_unpack(sum, sum0, sum1);
                            if (__any_sync(0xffffffffu, sum0 + sum1 > kMost)) {
                                read();
                                float most[2] = {s[0], s[1]};
#pragma unroll
                                for (int k = 2; k < 30; k += 4) {
                                    most[0] = max3(most[0], s[k], s[k + 1]);
                                    most[1] = max3(most[1], s[k + 2], s[k + 3]);
                                }
                                // every row of the warp goes along, to what it sees here: the
                                // rescaling costs the warp the same, and the next one comes later
                                const float to = fmaxf(m, floorf(max3(max3(most[0], s[30], s[31]), most[1], most[1]) * fac) - kRoom);
                                scale_l(ex2(m - to));
#pragma unroll 1
                                for (int k = chunk1 - 1; k > i; --k) scale_p(p_at + 16 * k, m - to);
                                m = to;
                                powers();
                            }
                            l2 = add_f32x2(l2, sum);
                            ptx::tmem_st16(p_at + 16 * i, p);
                        }
                        if (blocks < 4) {  // the other copies' columns
                            const uint32_t zero[16] = {};
#pragma unroll 1
                            for (int i = 0; i < 4; ++i)
                                if (i < chunk0 || i >= chunk1) ptx::tmem_st16(p_at + 16 * i, zero);
                        }
                        // ---- the m that O has after the tile before
                        if (it > 0) {
                            ok = wait_phase(&bars->turn[q4][b ^ 1], ((it - 1) >> 1) & 1, bars, a.status, lane);
                            if (!ok) break;
                        }
                        const float had = j > 0 ? ref[place] : m;
                        if (__any_sync(0xffffffffu, had != m)) {
                            const float to = fmaxf(had, m);
                            if (__any_sync(0xffffffffu, m < to)) {  // P is behind
                                scale_l(ex2(m - to));
                                
#pragma unroll 1
                                for (int k = chunk0; k < chunk1; ++k) scale_p(p_at + 16 * k, m - to);
                            }
                            if (__any_sync(0xffffffffu, had < to)) {  // O is behind
                                ok = wait_phase(&bars->s_free[(it - 1) % kBufS], (it - 1) / kBufS & 1, bars, a.status, lane);
                                if (!ok) break;
                                ptx::tc_fence_after();
                                const float by = ex2(had - to);
#pragma unroll 1
                                for (int i = 0; i < D / 32; ++i) {
                                    float o[32];
                                    tmem_read32(lanes + kColO + 32 * i, o);
#pragma unroll
                                    for (int k = 0; k < 32; ++k) o[k] *= by;
                                    ptx::tmem_st16(lanes + kColO + 32 * i, reinterpret_cast<const uint32_t(&)[16]>(o[0]));
                                    ptx::tmem_st16(lanes + kColO + 32 * i + 16, reinterpret_cast<const uint32_t(&)[16]>(o[16]));
                                }
                            }
                            m = to;
                        }
                        if (j == 0 || had != m) ref[place] = m;
                        __syncwarp();
                        arrive(lane == 0, &bars->turn[q4][b]);
                        ptx::tmem_st_wait();
                        ptx::tc_fence_before();
                    }
                    __syncwarp();
                    arrive(lane == 0, &bars->p_full[sb]);
                }
                it = it0 + n;
                if (!ok) break;
                // ---- the row's result: each group has half of its columns
                if (!active) {
                    // nothing of it; but the next row is not begun before all have begun this one
                    ok = n == 0 || wait_phase(&bars->q_full, seg & 1, bars, a.status, lane);
                    if (!ok) break;
                } else {
                    if (n > 0) {
                        // the last tile's turn comes first: with it, its S buffer's use before
                        // that is known to be over, and the wait cannot take that for this one
                        ok = wait_phase(&bars->turn[q4][(it - 1) & 1], ((it - 1) >> 1) & 1, bars, a.status, lane) &&
                             wait_phase(&bars->s_free[(it - 1) % kBufS], (it - 1) / kBufS & 1, bars, a.status, lane);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        const float to = ref[place];
                        float l0, l1;
                        ptx::f32x2_unpack(l2, l0, l1);
                        l = (l0 + l1) * ex2(m - to);
                        m = to;
                    }
                    float other;
                    ok = swap(l, other);
                    if (!ok) break;
                    l = group ? other + l : l + other;
                    float by = 1.f;  // what this copy's O is multiplied by
                    if (n > 0 && blocks < 4) {
                        float* tot = reinterpret_cast<float*>(smem + W::kTot) + group * 128;
                        tot[place] = l;
                        ok = meet();
                        if (!ok) break;
                        float top = kUnset;
                        for (int k = row; k < 128; k += 32 * blocks) top = fmaxf(top, ref[k]);
                        l = 0.f;
                        for (int k = row; k < 128; k += 32 * blocks) l += tot[k] * ex2(ref[k] - top);
                        by = ex2(m - top);
                        m = top;
                    }
                    // Written before the last tile's v_full, which its products and so the wait above
                    // are behind; and a row four on is dequantised only after the products of the
                    // row before last, for which both groups have left this one.
                    uint32_t nan = 0;  // in tokens that this position sees
                    if constexpr (!kList) {
#pragma unroll 1
                        for (int i = 0; i < draft; ++i) {
                            const int t = w.ctx - a.next_n + 1 + i;
                            if (t >= w.t0 && t < w.t1) nan |= bars->nan[seg & 3][i];
                        }
                    }
                    int64_t slot;
                    const bool whole = row_is_whole<kList>(a, r, slot);
                    const int64_t at_part = (slot * a.kv_heads + r.hk) * a.rows + row;
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    // 8 elements of the row's result, from element d on
                    auto put = [&](int d, const float* o) {
                        if (row >= a.rows) return;
                        const float f = (nan >> (d >> 4)) & 1 ? kNan : whole ? inv : 1.f;
                        if (whole) {
                            *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + at_row * D + d) =
                                make_uint4(pack<T>(o[0] * f, o[1] * f), pack<T>(o[2] * f, o[3] * f),
                                           pack<T>(o[4] * f, o[5] * f), pack<T>(o[6] * f, o[7] * f));
                        } else {
                            float4* out = reinterpret_cast<float4*>(a.part_o + at_part * D + d);
                            out[0] = make_float4(o[0] * f, o[1] * f, o[2] * f, o[3] * f);
                            out[1] = make_float4(o[4] * f, o[5] * f, o[6] * f, o[7] * f);
                        }
                    };
                    if (n == 0 || blocks == 4) {
#pragma unroll 1
                        for (int i = 0; i < D / 32; ++i) {
                            float o[16] = {};
                            const int d = group * (D / 2) + 16 * i;
                            if (n > 0) tmem_read16(lanes + kColO + d, o);
                            if (copy == 0) {
                                put(d, o);
                                put(d + 8, o + 8);
                            }
                        }
                    } else {
                        // 32 columns at a time: every copy leaves its own, then a warp sums
                        // 32 / (4 / blocks) of them over the copies
                        const uint32_t sums = base + W::kSum + group * (128 * 32 * 4);
#pragma unroll 1
                        for (int i = 0; i < D / 64; ++i) {
                            const int d = group * (D / 2) + 32 * i;
                            float o[32];
                            tmem_read32(lanes + kColO + d, o);
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                sts128(sums + place * 128 + ((k ^ (place & 7)) << 4), __float_as_uint(o[4 * k] * by),
                                       __float_as_uint(o[4 * k + 1] * by), __float_as_uint(o[4 * k + 2] * by),
                                       __float_as_uint(o[4 * k + 3] * by));
                            ok = meet();
                            if (!ok) break;
#pragma unroll 1
                            for (int e = 8 * blocks * copy; e < 8 * blocks * (copy + 1); e += 8) {
                                float v[8] = {};
                                for (int k = row; k < 128; k += 32 * blocks) {
                                    const uint4 x = lds128(sums + k * 128 + (((e >> 2) ^ (k & 7)) << 4));
                                    const uint4 y = lds128(sums + k * 128 + (((e >> 2) + 1 ^ (k & 7)) << 4));
                                    v[0] += __uint_as_float(x.x); v[1] += __uint_as_float(x.y);
                                    v[2] += __uint_as_float(x.z); v[3] += __uint_as_float(x.w);
                                    v[4] += __uint_as_float(y.x); v[5] += __uint_as_float(y.y);
                                    v[6] += __uint_as_float(y.z); v[7] += __uint_as_float(y.w);
                                }
                                put(d + e, v);
                            }
                            ok = meet();
                            if (!ok) break;
                        }
                        if (!ok) break;
                    }
                    if (row < a.rows && group == 0 && copy == 0) {
                        if (whole) {
                            if (a.lse != nullptr) a.lse[at_row] = lse_of(m, l);
                        } else {
                            *reinterpret_cast<float4*>(a.part_ml + at_part * 4) = make_float4(m, l, l, 0.f);
                        }
                    }
                }
                ptx::tc_fence_before();
                seg += n > 0;
                next_row<kList>(a, r);
            }
        } while (ok && !last);
    }

    if constexpr (!kList) {
        if (warp == 2 || warp == 3) dense_extras<D>(a, warp - 2, 2, lane);
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
    // a kernel launched with fewer registers would wait for them without end
    static const int registers = [] {
        cudaFuncAttributes at;
        return cudaFuncGetAttributes(&at, attention_wide_kernel<D, T, kList>) == cudaSuccess ? at.numRegs : 0;
    }();
    if ((registers + 7) / 8 * 8 < kRegsLaunch) return cudaErrorInvalidConfiguration;
    const int64_t x = kList ? (int64_t)a.batch * a.next_n * a.splits * a.kv_heads : a.deal;
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
