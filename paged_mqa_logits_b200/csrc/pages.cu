// Page tables and reference counts: fork, resize, compact; and the copy of pages.
//
// Every decision is a function of the tables, lengths and counts alone: free
// pages are ranked by number (prefix sums over page_refs), rows by index, and
// the atomics on page_refs only add, so no result depends on thread order.
#include "pages.cuh"

#include <cooperative_groups.h>

#include "host.cuh"

namespace mqa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPer = 8;                           // page counts per thread and round of a scan
constexpr int kRound = kPlanThreads * kPer;

// Exclusive prefix sum over the CTA (kPlanThreads threads); `total` gets the sum.
// `tmp` holds 33 ints of shared memory; all threads call.
__device__ __forceinline__ int block_scan(int v, int* tmp, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) tmp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int s = tmp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        tmp[lane] = s;
    }
    __syncthreads();
    total = tmp[31];
    const int before = (warp ? tmp[warp - 1] : 0) + x - v;
    __syncthreads();
    return before;
}

// The page counts [first, first + kPer) (1 behind the pool: neither free nor, for
// compact, looked at).
__device__ __forceinline__ void load_refs(const int32_t* refs, int first, int num, int (&r)[kPer]) {
    if (first + kPer <= num && (reinterpret_cast<uintptr_t>(refs) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < kPer; i += 4) {
            const int4 v = *reinterpret_cast<const int4*>(refs + first + i);
            r[i] = v.x; r[i + 1] = v.y; r[i + 2] = v.z; r[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) r[i] = first + i < num ? refs[first + i] : 1;
    }
}

__device__ __forceinline__ int pages_of(const PagesArgs& a, int len) {
    return (int)(((int64_t)len + a.page_size - 1) >> a.ps_shift);
}

__device__ __forceinline__ int len_of(const PagesArgs& a, const int32_t* lens, int b) {
    return clamp_len(a.status, lens[b], a.max_pages << a.ps_shift);
}

__device__ __forceinline__ bool good_page(const PagesArgs& a, int p) {
    if (p >= 0 && p < a.num_pages) return true;
    report_checked(a.status, MQA_STATUS_BAD_PAGE);
    return false;
}

// ---------------------------------------------------------------- fork
// CTA x takes old row x's references off and writes new row x with its own on; a
// row that goes on from itself keeps its counts untouched.
__global__ void __launch_bounds__(128) fork_kernel(const int32_t* table, const int32_t* lens,
                                                   const int32_t* parents, int32_t* refs,
                                                   int32_t* out_table, int32_t* out_lens,
                                                   PagesArgs a) {
    ptx::griddep_wait();
    const int r = blockIdx.x;
    int parent = -1;
    if (r < a.out_batch) {
        parent = parents[r];
        if (parent < 0 || parent >= a.batch) {
            if (parent != -1 && threadIdx.x == 0) report_checked(a.status, MQA_STATUS_BAD_CONTEXT);
            parent = -1;
        }
    }
    if (r < a.batch && parent != r) {
        const int n = pages_of(a, len_of(a, lens, r));
        const int32_t* row = table + (int64_t)r * a.max_pages;
        for (int j = threadIdx.x; j < n; j += blockDim.x)
            if (good_page(a, row[j])) atomicSub(refs + row[j], 1);
    }
    if (r < a.out_batch) {
        const int len = parent >= 0 ? len_of(a, lens, parent) : 0;
        const int n = pages_of(a, len);
        const int32_t* row = table + (int64_t)max(parent, 0) * a.max_pages;
        int32_t* out = out_table + (int64_t)r * a.max_pages;
        for (int j = threadIdx.x; j < a.max_pages; j += blockDim.x) {
            const int p = j < n ? row[j] : -1;
            out[j] = p;
            if (j < n && parent != r && good_page(a, p)) atomicAdd(refs + p, 1);
        }
        if (threadIdx.x == 0) out_lens[r] = len;
    }
}

// ---------------------------------------------------------------- resize
// One CTA, since every step hangs on prefix sums over the rows or the pool and the
// work is a few thousand entries. (1) every row's need of pages and the prefix sums
// over the rows; (2) a scan of page_refs ranks the free pages, and the page of rank r
// goes to the row whose range of ranks holds r; it ends once every need is met; (3)
// lengths, releases and the counts of replaced pages (after the scan, so that nothing
// freed here is taken here). What bounds it are chains of loads from L2: four rows or
// eight pages a thread are loaded together, and the next pages while the present
// ones are ranked.
constexpr int kRows = 4;  // of a thread at a time in step 1

// kCached: where the row's new pages start in its table, and whether the first of
// them takes another's place, is kept in shared memory (else found again).
template <bool kCached>
__global__ void __launch_bounds__(kPlanThreads) resize_kernel(int32_t* table, int32_t* lens,
                                                              const int32_t* new_lens,
                                                              int32_t* refs, int32_t* src,
                                                              int32_t* dst, PagesArgs a) {
    extern __shared__ int pre[];             // [batch + 1]: ranks before each row
    int* start = pre + a.batch + 1;          // [batch]: first new entry * 2 + (takes another's place)
    __shared__ int tmp[33];
    ptx::griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    const int most = a.max_pages << a.ps_shift;
    int total = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads * kRows) {
        int old[kRows], now[kRows], end[kRows], need[kRows], sum = 0;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int b = b0 + tid * kRows + i;
            old[i] = b < a.batch ? lens[b] : 0;
            now[i] = b < a.batch ? new_lens[b] : 0;
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int b = b0 + tid * kRows + i;
            old[i] = clamp_len(a.status, old[i], most);
            now[i] = clamp_len(a.status, now[i], most);
            end[i] = now[i] > old[i] && (old[i] & (a.page_size - 1))
                         ? table[(int64_t)b * a.max_pages + pages_of(a, old[i]) - 1] : -1;
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const bool partly = now[i] > old[i] && (old[i] & (a.page_size - 1));
            if (!partly || !good_page(a, end[i]) || refs[end[i]] <= 1) end[i] = -1;
            need[i] = (now[i] > old[i] ? pages_of(a, now[i]) - pages_of(a, old[i]) : 0) + (end[i] >= 0);
            sum += need[i];
        }
        int all;
        int before = total + block_scan(sum, tmp, all);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int b = b0 + tid * kRows + i;
            if (b >= a.batch) break;
            src[b] = end[i];
            dst[b] = -1;
            pre[b] = before;
            if (kCached) start[b] = (pages_of(a, old[i]) - (end[i] >= 0)) * 2 + (end[i] >= 0);
            before += need[i];
        }
        total += all;
    }
    if (tid == 0) pre[a.batch] = total;
    __syncthreads();
    auto start_of = [&](int b) {
        if (kCached) return start[b];
        const int swaps = src[b] >= 0;
        return (pages_of(a, len_of(a, lens, b)) - swaps) * 2 + swaps;
    };

    int found = 0;
    int r[kPer];
    if (total > 0) load_refs(refs, tid * kPer, a.num_pages, r);
    for (int p0 = 0; p0 < a.num_pages && found < total; p0 += kRound) {
        int free = 0, sum, next[kPer];
        load_refs(refs, p0 + kRound + tid * kPer, a.num_pages, next);
#pragma unroll
        for (int i = 0; i < kPer; ++i) free += r[i] == 0;
        int rank = found + block_scan(free, tmp, sum);
        if (free > 0 && rank < total) {
            int lo = 0, hi = a.batch - 1;  // the last row that begins at or before rank
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (pre[mid] <= rank) lo = mid; else hi = mid - 1;
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (r[i] != 0 || rank >= total) continue;
                const int page = p0 + tid * kPer + i;
                while (pre[lo + 1] <= rank) ++lo;
                const int at = start_of(lo);
                table[(int64_t)lo * a.max_pages + (at >> 1) + rank - pre[lo]] = page;
                if ((at & 1) && rank == pre[lo]) dst[lo] = page;
                refs[page] = 1;
                ++rank;
            }
        }
        found += sum;
#pragma unroll
        for (int i = 0; i < kPer; ++i) r[i] = next[i];
    }
    __syncthreads();
    if (found < total) {
        if (tid == 0) report(a.status, MQA_STATUS_NO_PAGES);
        for (int b = tid; b < a.batch; b += kPlanThreads) {
            if (pre[b + 1] == pre[b] || pre[b + 1] <= found) continue;
            // at most one row was given a part of its pages: they go back
            const int at = start_of(b);
            int32_t* row = table + (int64_t)b * a.max_pages + (at >> 1);
            for (int k = pre[b]; k < found; ++k) {
                refs[row[k - pre[b]]] = 0;
                row[k - pre[b]] = k == pre[b] && (at & 1) ? src[b] : -1;
            }
            src[b] = -1;
            dst[b] = -1;
        }
        __syncthreads();
    }

    for (int b0 = (tid >> 5) * 32; b0 < a.batch; b0 += kPlanThreads) {
        const int b = b0 + lane;
        int had = 0, has = 0;
        if (b < a.batch) {
            const int old = lens[b], want = new_lens[b], from = src[b];
            had = min(max(old, 0), most);
            int now = min(max(want, 0), most);
            if (pre[b + 1] > found && pre[b + 1] > pre[b]) now = had;
            if (from >= 0) atomicSub(refs + from, 1);
            lens[b] = now;
            had = pages_of(a, had);
            has = pages_of(a, now);
        }
        uint32_t shrinks = __ballot_sync(0xffffffffu, has < had);
        while (shrinks) {
            const int k = __ffs(shrinks) - 1;
            shrinks &= shrinks - 1;
            const int from = __shfl_sync(0xffffffffu, has, k), to = __shfl_sync(0xffffffffu, had, k);
            int32_t* row = table + (int64_t)(b0 + k) * a.max_pages;
            for (int j = from + lane; j < to; j += 32) {
                if (good_page(a, row[j])) atomicSub(refs + row[j], 1);
                row[j] = -1;
            }
        }
    }
}

// ---------------------------------------------------------------- compact
// A cluster of 8 CTAs, each with a contiguous eighth of the pool: counts the pages in
// use (N), then the used pages at N and above and the free ones below N, ranks both
// (the eighths' counts go through distributed shared memory), pairs them, and moves
// the counts. (One CTA took 26 us for 22 thousand pages.)
constexpr int kPlanCtas = 8;

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(int32_t* refs, int32_t* src,
                                                                    int32_t* dst, int32_t* count,
                                                                    int32_t* map, PagesArgs a) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ int tmp[33];
    __shared__ int mine[3];  // this CTA's pages in use; to move; holes to fill
    ptx::griddep_wait();
    const int tid = threadIdx.x, half = a.num_pages / 2, rank = (int)cluster.block_rank();
    const int per = ((a.num_pages + kPlanCtas - 1) / kPlanCtas + kPer - 1) / kPer * kPer;
    const int begin = (int)min((int64_t)rank * per, (int64_t)a.num_pages), end = min(a.num_pages - begin, per) + begin;
    auto counts = [&](int n, int& m, int& h) {  // of the slice, per thread: n < 0: the pages in use
        m = h = 0;
        for (int first = begin + tid * kPer; first < end; first += kRound) {
            int r[kPer];
            load_refs(refs, first, a.num_pages, r);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int p = first + i;
                const bool live = r[i] > 0;
                m += p < end && live && (n < 0 || p >= n);
                h += p < end && p < n && !live;
            }
        }
    };
    int m, h, live, n = 0;
    counts(-1, m, h);
    block_scan(m, tmp, live);
    if (tid == 0) mine[0] = live;
    cluster.sync();
    for (int c = 0; c < kPlanCtas; ++c) n += *cluster.map_shared_rank(&mine[0], c);
    int all_m, all_h;
    counts(n, m, h);
    block_scan(m, tmp, all_m);
    block_scan(h, tmp, all_h);
    if (tid == 0) {
        mine[1] = all_m;
        mine[2] = all_h;
    }
    cluster.sync();
    int moves = 0, holes = 0, total = 0;
    for (int c = 0; c < kPlanCtas; ++c) {
        const int cm = *cluster.map_shared_rank(&mine[1], c), ch = *cluster.map_shared_rank(&mine[2], c);
        moves += c < rank ? cm : 0;
        holes += c < rank ? ch : 0;
        total += cm;
    }
    for (int p0 = begin; p0 < end; p0 += kRound) {
        const int first = p0 + tid * kPer;
        int r[kPer], sum;
        load_refs(refs, first, a.num_pages, r);
        m = h = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int p = first + i;
            m += p < end && p >= n && r[i] > 0;
            h += p < end && p < n && r[i] <= 0;
        }
        // both counts stay below 2^16 a round: one scan for the two
        const int both = block_scan(m | h << 16, tmp, sum);
        int mr = moves + (both & 0xffff), hr = holes + (both >> 16);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int p = first + i;
            if (p >= end) break;
            if (p >= n && r[i] > 0) src[mr++] = p;
            if (p < n && r[i] <= 0) dst[hr++] = p;
            map[p] = r[i] > 0 ? p : -1;
        }
        moves += sum & 0xffff;
        holes += sum >> 16;
    }
    cluster.sync();
    const int threads = kPlanCtas * kPlanThreads;
    for (int i = rank * kPlanThreads + tid; i < half; i += threads) {
        if (i < total) {
            const int s = src[i], d = dst[i];
            const int r = refs[s];
            map[s] = d;
            refs[d] = r;
            refs[s] = 0;
        } else {
            src[i] = -1;
            dst[i] = -1;
        }
    }
    if (rank == 0 && tid == 0) *count = total;
    cluster.sync();  // no CTA ends while another may read its counts
}

__global__ void __launch_bounds__(128) compact_table_kernel(int32_t* table, const int32_t* lens,
                                                            const int32_t* map, PagesArgs a) {
    ptx::griddep_wait();
    const int b = blockIdx.x;
    const int n = pages_of(a, len_of(a, lens, b));
    int32_t* row = table + (int64_t)b * a.max_pages;
    for (int j = threadIdx.x; j < n; j += blockDim.x)
        if (good_page(a, row[j])) row[j] = map[row[j]];
}

// ---------------------------------------------------------------- copy
// A warp copies a page of one cache at a time, four 16-byte pieces a lane in flight;
// the pairs of the warp's next page are loaded meanwhile. 70 thousand
// pages of 2304 bytes, K and V: 0.84 of the copy rate. (A CTA a page left half of its
// threads idle on them: 0.77.)
constexpr int kCopyThreads = 256, kCopyWarps = kCopyThreads / 32;

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyArgs a) {
    ptx::griddep_wait();
    const int n = a.count != nullptr ? min(max(*a.count, 0), a.n) : a.n;
    const uint32_t chunks = a.chunks[blockIdx.y];
    const uint32_t lane = threadIdx.x & 31;
    uint4* const pool = static_cast<uint4*>(a.cache[blockIdx.y]);
    const int step = gridDim.x * kCopyWarps;
    int i = blockIdx.x * kCopyWarps + (threadIdx.x >> 5);
    int s = i < n ? a.src[i] : -1, d = i < n ? a.dst[i] : -1;
    while (i < n) {
        const int next = i + step;
        const int s1 = next < n ? a.src[next] : -1, d1 = next < n ? a.dst[next] : -1;
        if (s >= 0 && s < a.num_pages && d >= 0 && d < a.num_pages) {
            const uint4* from = pool + (int64_t)s * chunks;
            uint4* to = pool + (int64_t)d * chunks;
            for (uint32_t c = lane; c < chunks; c += 128) {
                uint4 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (c + 32 * k < chunks) v[k] = __ldcs(from + c + 32 * k);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (c + 32 * k < chunks) __stcs(to + c + 32 * k, v[k]);
            }
        } else if (lane == 0 && (s < -1 || s >= a.num_pages || d < -1 || d >= a.num_pages)) {
            report_checked(a.status, MQA_STATUS_BAD_PAGE);
        }
        i = next;
        s = s1;
        d = d1;
    }
}

}  // namespace

cudaError_t launch_fork(const int32_t* table, const int32_t* lens, const int32_t* parents,
                        int32_t* refs, int32_t* out_table, int32_t* out_lens, const PagesArgs& a,
                        void* stream, bool pdl) {
    return launch_pdl(fork_kernel, dim3(max(a.batch, a.out_batch)), dim3(128), 0, stream, pdl,
                      table, lens, parents, refs, out_table, out_lens, a);
}

cudaError_t launch_resize(int device, int32_t* table, int32_t* lens, const int32_t* new_lens,
                          int32_t* refs, int32_t* src, int32_t* dst, const PagesArgs& a,
                          void* stream, bool pdl) {
    // the limit is always raised to the most that a batch can need: set to this call's need,
    // a smaller call on another host thread could lower it between the two
    constexpr uint32_t kMostCached = 200000, kMost = (kMaxBatch + 1) * 4;
    static uint32_t done[2][64];
    const uint32_t pre = (uint32_t)(a.batch + 1) * 4;
    const bool cached = pre * 2 <= kMostCached;
    const uint32_t smem = cached ? pre * 2 : pre;
    if (smem > 40000) {
        const cudaError_t e = cached ? allow_smem(resize_kernel<true>, device, kMostCached, done[1])
                                     : allow_smem(resize_kernel<false>, device, kMost, done[0]);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(cached ? resize_kernel<true> : resize_kernel<false>, dim3(1),
                      dim3(kPlanThreads), smem, stream, pdl, table, lens, new_lens, refs, src, dst, a);
}

cudaError_t launch_compact(int32_t* table, const int32_t* lens, int32_t* refs, int32_t* src,
                           int32_t* dst, int32_t* count, int32_t* map, const PagesArgs& a,
                           void* stream, bool pdl) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kPlanCtas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {kPlanCtas, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, compact_plan_kernel, refs, src, dst, count, map, a);
    if (e != cudaSuccess || a.batch == 0) return e;
    return launch_pdl(compact_table_kernel, dim3(a.batch), dim3(128), 0, stream, pdl, table, lens,
                      map, a);
}

cudaError_t launch_copy(const CopyArgs& a, void* stream, bool pdl) {
    // as many CTAs as the SMs hold at once, over all caches
    const int most = (148 * 6 + a.num_caches - 1) / a.num_caches;
    const int want = (int)(((int64_t)a.n + kCopyWarps - 1) / kCopyWarps);
    return launch_pdl(copy_kernel, dim3(want < most ? want : most, a.num_caches), dim3(kCopyThreads), 0, stream, pdl, a);
}

}  // namespace mqa
