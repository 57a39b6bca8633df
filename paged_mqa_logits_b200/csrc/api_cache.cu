// The C ABI declared in include/mqa_cache.h: host-side checks and launches.
#include <cuda_runtime.h>

#include "append.cuh"
#include "attention.cuh"
#include "host.cuh"
#include "pages.cuh"

namespace mqa {
namespace {

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

int sm_count(int device, int* out) {
    static int cached[64];
    if (device >= 0 && device < 64 && cached[device] > 0) {
        *out = cached[device];
        return MQA_OK;
    }
    const cudaError_t e = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, device);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute(SM count)");
    if (device >= 0 && device < 64) cached[device] = *out;
    return MQA_OK;
}

int check_flags(uint32_t flags) {
    if (flags & ~(uint32_t)(MQA_FLAG_VALIDATE | MQA_FLAG_NO_PDL))
        return fail(MQA_ERR_INVALID_ARG, "unknown flag bits 0x%x", flags);
    return MQA_OK;
}

uint32_t with_env(uint32_t flags) {
    return flags | (env_flag("MQA_LOGITS_VALIDATE") ? MQA_FLAG_VALIDATE : 0u);
}

// What every paged cache's call checks of its shape.
int check_pool(int batch, int page_size, int ps_min, int num_pages, int max_pages) {
    if (batch < 0) return fail(MQA_ERR_INVALID_ARG, "batch must be >= 0 (got %d)", batch);
    if (!pow2(page_size) || page_size < ps_min || page_size > 256)
        return fail(MQA_ERR_INVALID_ARG, "page_size must be a power of two in [%d, 256] (got %d)",
                    ps_min, page_size);
    if (num_pages < 1) return fail(MQA_ERR_INVALID_ARG, "num_pages must be >= 1");
    if (max_pages < 1) return fail(MQA_ERR_INVALID_ARG, "max_pages_per_row must be >= 1");
    if ((int64_t)num_pages * page_size > INT32_MAX)
        return fail(MQA_ERR_UNSUPPORTED, "num_pages * page_size must be < 2^31");
    if ((int64_t)max_pages * page_size > INT32_MAX)
        return fail(MQA_ERR_UNSUPPORTED, "max_pages_per_row * page_size must be < 2^31");
    return MQA_OK;
}

// A buffer of a call: NULL or no bytes overlap nothing.
struct Buffer {
    const void* at;
    int64_t bytes;
};

bool overlap(const Buffer& a, const Buffer& b) {
    const char *x = static_cast<const char*>(a.at), *y = static_cast<const char*>(b.at);
    return x && y && a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes;
}

// Whether one of the first `written` buffers overlaps any other.
template <int N>
bool any_overlap(const Buffer (&all)[N], int written) {
    for (int i = 0; i < written; ++i)
        for (int j = i + 1; j < N; ++j)
            if (overlap(all[i], all[j])) return true;
    return false;
}

constexpr int kMostTokens = INT32_MAX - 65535;  // of a row, or of a token list

int check_attention(const mqa_attention_params* p) {
    if (!p) return fail(MQA_ERR_INVALID_ARG, "params is NULL");
    int rc = check_pool(p->batch, p->page_size, 16, p->num_pages, p->max_pages_per_row);
    if (rc != MQA_OK) return rc;
    if (p->next_n < 1 || p->next_n > 4)
        return fail(MQA_ERR_INVALID_ARG, "next_n must be in 1..4 (got %d)", p->next_n);
    if (p->num_heads < 1 || p->num_kv_heads < 1 || p->num_heads % p->num_kv_heads)
        return fail(MQA_ERR_INVALID_ARG, "num_kv_heads must divide num_heads (got %d, %d)",
                    p->num_kv_heads, p->num_heads);
    // the rows that share a tile: all positions' of a kv head, or (lists) one position's
    if (p->num_heads / p->num_kv_heads * (int64_t)(p->topk > 0 ? 1 : p->next_n) > 128 || p->num_kv_heads > 4096)
        return fail(MQA_ERR_UNSUPPORTED,
                    "num_heads / num_kv_heads * next_n (lists: without next_n) must be <= 128 and "
                    "num_kv_heads <= 4096 (got %d / %d * %d)", p->num_heads, p->num_kv_heads, p->next_n);
    if (p->head_dim != 64 && p->head_dim != 128)
        return fail(MQA_ERR_UNSUPPORTED, "head_dim must be 64 or 128 (got %d)", p->head_dim);
    if (p->dtype != MQA_DTYPE_BF16 && p->dtype != MQA_DTYPE_F16)
        return fail(MQA_ERR_INVALID_ARG, "dtype must be bf16 or f16 (got %d)", p->dtype);
    if (p->topk < 0) return fail(MQA_ERR_INVALID_ARG, "topk must be >= 0 (got %d)", p->topk);
    // the kernels step a whole tile past a row's end
    if (p->topk > kMostTokens)
        return fail(MQA_ERR_UNSUPPORTED, "topk must be <= %d (got %d)", kMostTokens, p->topk);
    if ((int64_t)p->max_pages_per_row * p->page_size > kMostTokens)
        return fail(MQA_ERR_UNSUPPORTED, "max_pages_per_row * page_size must be <= %d", kMostTokens);
    if (p->topk == 0 && (p->num_ctas < 1 || p->num_ctas > kMaxCtas))
        return fail(MQA_ERR_INVALID_ARG, "num_ctas must be in 1..%d (got %d)", kMaxCtas, p->num_ctas);
    if (p->batch > kMaxBatch)
        return fail(MQA_ERR_INVALID_ARG, "batch must be <= %d (got %d)", kMaxBatch, p->batch);
    return MQA_OK;
}

// The part of the arguments that the split follows from.
int split_of(const mqa_attention_params* p, int device, AttentionArgs& a) {
    int sms = 0;
    const int rc = sm_count(device, &sms);
    if (rc != MQA_OK) return rc;
    a.batch = p->batch;
    a.next_n = p->next_n;
    a.heads = p->num_heads;
    a.kv_heads = p->num_kv_heads;
    a.group = p->num_heads / p->num_kv_heads;
    a.rows = p->topk > 0 ? a.group : a.group * p->next_n;
    a.num_ctas = p->num_ctas;
    a.topk = p->topk;
    const ListSplit s = p->topk > 0 ? split_list((int64_t)p->batch * p->next_n * p->num_kv_heads, p->topk, a.rows,
                                                 p->head_dim, sms)
                                    : ListSplit{1, false};
    a.splits = s.splits;
    a.small = s.small;
    return MQA_OK;
}

uint64_t workspace_of(const AttentionArgs& a, int head_dim) {
    return (uint64_t)attention_slots(a) * a.kv_heads * a.rows * (head_dim + 4) * 4;
}

}  // namespace
}  // namespace mqa

extern "C" {

int mqa_attention_workspace_size(const mqa_attention_params* params, uint64_t* bytes) {
    using namespace mqa;
    if (!bytes) return fail(MQA_ERR_INVALID_ARG, "bytes is NULL");
    int rc = check_attention(params);
    if (rc != MQA_OK) return rc;
    *bytes = 0;
    if (params->batch == 0) return MQA_OK;
    int dev = 0;
    rc = check_arch(&dev);
    if (rc != MQA_OK) return rc;
    // one row and position: the lists that are cut into most parts
    mqa_attention_params one = *params;
    if (one.topk > 0) one.batch = one.next_n = 1;
    AttentionArgs a{};
    rc = split_of(&one, dev, a);
    if (rc != MQA_OK) return rc;
    *bytes = workspace_of(a, one.head_dim);
    if (a.splits > 1) {  // any number of lists has no more parts than SMs (split_list)
        int sms = 0;
        rc = sm_count(dev, &sms);
        if (rc != MQA_OK) return rc;
        a.splits = sms / a.kv_heads;
        *bytes = workspace_of(a, one.head_dim);
    }
    return MQA_OK;
}

int paged_mqa_attention_fp4(const void* q, const void* k_cache, const void* v_cache,
                            const int32_t* block_table, const int32_t* context_lens,
                            const int32_t* schedule, const int32_t* indices, void* out,
                            float* lse, void* workspace, const mqa_attention_params* params,
                            void* stream) {
    using namespace mqa;
    int rc = check_attention(params);
    if (rc != MQA_OK) return rc;
    const mqa_attention_params& p = *params;
    rc = check_flags(p.flags);
    if (rc != MQA_OK) return rc;
    if (p.batch == 0) return MQA_OK;
    if (!q || !k_cache || !v_cache || !block_table || !context_lens || !out)
        return fail(MQA_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if (p.topk == 0 ? !schedule : !indices)
        return fail(MQA_ERR_INVALID_ARG, p.topk == 0 ? "schedule is NULL" : "indices is NULL");
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(workspace, 16))
        return fail(MQA_ERR_INVALID_ARG,
                    "q, k_cache, v_cache, out and workspace must be 16-byte aligned");
    if (!aligned(block_table, 4) || !aligned(context_lens, 4) || !aligned(schedule, 4) ||
        !aligned(indices, 4) || !aligned(lse, 4) || !aligned(p.status, 4))
        return fail(MQA_ERR_INVALID_ARG, "int32 and fp32 buffers must be 4-byte aligned");
    if (p.q_stride_b % 8 || p.q_stride_n % 8 || p.q_stride_h % 8)
        return fail(MQA_ERR_INVALID_ARG, "the strides of q must be multiples of 8 elements");
    int dev = 0;
    uint32_t* lib_status = nullptr;
    rc = check_arch(&dev, &lib_status);
    if (rc != MQA_OK) return rc;
    AttentionArgs a{};
    rc = split_of(params, dev, a);
    if (rc != MQA_OK) return rc;
    const uint64_t need = workspace_of(a, p.head_dim);
    if (need > 0 && (!workspace || p.workspace_bytes < need))
        return fail(MQA_ERR_INVALID_ARG, "workspace must hold %llu bytes (got %llu)",
                    (unsigned long long)need, (unsigned long long)(workspace ? p.workspace_bytes : 0));
    if ((int64_t)p.batch * p.next_n * a.splits > INT32_MAX ||
        (int64_t)p.batch * p.next_n * p.num_heads > INT32_MAX / 8)
        return fail(MQA_ERR_UNSUPPORTED, "batch * next_n * num_heads is too large");
    a.q = q;
    a.k = static_cast<const uint8_t*>(k_cache);
    a.v = static_cast<const uint8_t*>(v_cache);
    a.block_table = block_table;
    a.context_lens = context_lens;
    a.schedule = schedule;
    a.indices = indices;
    a.out = out;
    a.lse = lse;
    a.part_ml = static_cast<float*>(workspace);
    a.part_o = a.part_ml + attention_slots(a) * a.kv_heads * a.rows * 4;
    a.q_sb = p.q_stride_b;
    a.q_sn = p.q_stride_n;
    a.q_sh = p.q_stride_h;
    a.page_size = p.page_size;
    a.ps_shift = log2_of(p.page_size);
    a.num_pages = p.num_pages;
    a.max_pages = p.max_pages_per_row;
    a.page_bytes = (uint32_t)p.num_kv_heads * p.page_size * (p.head_dim / 2 + p.head_dim / 16);
    a.status = {lib_status, p.status, with_env(p.flags)};
    a.scale_log2 = p.softmax_scale * 1.44269504088896f;
    const cudaError_t e = launch_attention(dev, p.head_dim, p.dtype, a, stream,
                                           (p.flags & MQA_FLAG_NO_PDL) == 0);
    if (e != cudaSuccess) return cuda_fail(e, "attention launch");
    return MQA_OK;
}

static int run_append(bool fp8, const void* k, const void* v, void* k_cache, void* v_cache,
                      const int32_t* block_table, const int32_t* context_lens,
                      const int32_t* row_offsets, void* k_values, void* v_values,
                      const mqa_append_params* params, void* stream) {
    using namespace mqa;
    if (!params) return fail(MQA_ERR_INVALID_ARG, "params is NULL");
    const mqa_append_params& p = *params;
    int rc = check_pool(p.batch, p.page_size, fp8 ? 8 : 16, p.num_pages, p.max_pages_per_row);
    if (rc != MQA_OK) return rc;
    rc = check_flags(p.flags);
    if (rc != MQA_OK) return rc;
    if (p.num_tokens < 0)
        return fail(MQA_ERR_INVALID_ARG, "num_tokens must be >= 0 (got %d)", p.num_tokens);
    if (fp8 ? p.num_kv_heads != 1 : p.num_kv_heads < 1)
        return fail(MQA_ERR_INVALID_ARG, "num_kv_heads must be %s (got %d)", fp8 ? "1" : ">= 1",
                    p.num_kv_heads);
    const int D = p.head_dim;
    if (!(D == 64 || D == 128 || (fp8 && D == 32)))
        return fail(MQA_ERR_UNSUPPORTED, "head_dim must be %s64 or 128 (got %d)", fp8 ? "32, " : "", D);
    if (p.dtype != MQA_DTYPE_BF16 && p.dtype != MQA_DTYPE_F16)
        return fail(MQA_ERR_INVALID_ARG, "dtype must be bf16 or f16 (got %d)", p.dtype);
    if ((int64_t)p.num_tokens * p.num_kv_heads * (D / 16) > INT32_MAX)
        return fail(MQA_ERR_UNSUPPORTED, "num_tokens * num_kv_heads * head_dim must be < 2^35");
    if (p.num_tokens == 0 || p.batch == 0) return MQA_OK;
    if (!row_offsets && p.num_tokens % p.batch)
        return fail(MQA_ERR_INVALID_ARG,
                    "without row_offsets num_tokens must be a multiple of batch (got %d, %d)",
                    p.num_tokens, p.batch);
    if (!k || !k_cache || !block_table || !context_lens)
        return fail(MQA_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if (!v != !v_cache) return fail(MQA_ERR_INVALID_ARG, "v and v_cache go together");
    if (!v && v_values) return fail(MQA_ERR_INVALID_ARG, "v_values without v");
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(k_values, 16) || !aligned(v_values, 16))
        return fail(MQA_ERR_INVALID_ARG, "tokens, caches and values must be 16-byte aligned");
    if (!aligned(block_table, 4) || !aligned(context_lens, 4) || !aligned(row_offsets, 4) ||
        !aligned(p.status, 4))
        return fail(MQA_ERR_INVALID_ARG, "int32 buffers must be 4-byte aligned");
    if (p.k_stride_t % 8 || p.k_stride_h % 8 || (v && (p.v_stride_t % 8 || p.v_stride_h % 8)))
        return fail(MQA_ERR_INVALID_ARG, "the tokens' strides must be multiples of 8 elements");
    const int64_t cache = (int64_t)p.num_pages * p.page_size * p.num_kv_heads * (fp8 ? D + 4 : D / 2 + D / 16);
    if (overlap({k_cache, cache}, {v_cache, cache}))
        return fail(MQA_ERR_INVALID_ARG, "k_cache and v_cache must be two buffers");
    const int64_t values = (int64_t)p.num_tokens * p.num_kv_heads * D * 2;
    const Buffer all[] = {{k_values, values}, {v_values, values}, {k_cache, cache}, {v_cache, cache}};
    if (any_overlap(all, 2))
        return fail(MQA_ERR_INVALID_ARG, "values must overlap neither each other nor the caches");
    uint32_t* lib_status = nullptr;
    rc = check_arch(nullptr, &lib_status);
    if (rc != MQA_OK) return rc;
    AppendArgs a{};
    a.x[0] = {k, k_cache, k_values, p.k_stride_t, p.k_stride_h};
    a.x[1] = {v, v_cache, v_values, p.v_stride_t, p.v_stride_h};
    a.block_table = block_table;
    a.context_lens = context_lens;
    a.row_offsets = row_offsets;
    a.status = {lib_status, p.status, with_env(p.flags)};
    a.batch = p.batch;
    a.num_tokens = p.num_tokens;
    a.per_row = row_offsets ? 0 : p.num_tokens / p.batch;
    a.heads = p.num_kv_heads;
    a.page_size = p.page_size;
    a.ps_shift = log2_of(p.page_size);
    a.num_pages = p.num_pages;
    a.max_pages = p.max_pages_per_row;
    const cudaError_t e = launch_append(fp8, D, p.dtype, a, v ? 2 : 1, stream,
                                        (p.flags & MQA_FLAG_NO_PDL) == 0);
    if (e != cudaSuccess) return cuda_fail(e, "append launch");
    return MQA_OK;
}

int mqa_cache_append_fp8(const void* x, void* kv_cache, const int32_t* block_table,
                         const int32_t* context_lens, const int32_t* row_offsets, void* values,
                         const mqa_append_params* params, void* stream) {
    return run_append(true, x, nullptr, kv_cache, nullptr, block_table, context_lens, row_offsets,
                      values, nullptr, params, stream);
}

int mqa_cache_append_fp4(const void* k, const void* v, void* k_cache, void* v_cache,
                         const int32_t* block_table, const int32_t* context_lens,
                         const int32_t* row_offsets, void* k_values, void* v_values,
                         const mqa_append_params* params, void* stream) {
    return run_append(false, k, v, k_cache, v_cache, block_table, context_lens, row_offsets,
                      k_values, v_values, params, stream);
}

static int check_pages(const mqa_pages_params* p, bool table) {
    using namespace mqa;
    if (!p) return fail(MQA_ERR_INVALID_ARG, "params is NULL");
    int rc = check_flags(p->flags);
    if (rc != MQA_OK) return rc;
    if (p->num_pages < 1) return fail(MQA_ERR_INVALID_ARG, "num_pages must be >= 1");
    if (!aligned(p->status, 4))
        return fail(MQA_ERR_INVALID_ARG, "status must be 4-byte aligned");
    if (!table) return MQA_OK;
    rc = check_pool(p->batch, p->page_size, 8, p->num_pages, p->max_pages_per_row);
    if (rc != MQA_OK) return rc;
    if (p->batch > kMaxBatch || p->out_batch < 0 || p->out_batch > kMaxBatch)
        return fail(MQA_ERR_INVALID_ARG, "batch and out_batch must be in 0..%d (got %d, %d)",
                    kMaxBatch, p->batch, p->out_batch);
    if ((int64_t)p->batch * (p->max_pages_per_row + 1ll) > INT32_MAX)
        return fail(MQA_ERR_UNSUPPORTED, "batch * max_pages_per_row must be < 2^31");
    return MQA_OK;
}

static mqa::PagesArgs pages_args(const mqa_pages_params& p, uint32_t* lib_status) {
    mqa::PagesArgs a{};
    a.status = {lib_status, p.status, mqa::with_env(p.flags)};
    a.batch = p.batch;
    a.out_batch = p.out_batch;
    a.max_pages = p.max_pages_per_row;
    a.num_pages = p.num_pages;
    a.page_size = p.page_size;
    a.ps_shift = mqa::log2_of(p.page_size);
    return a;
}

int mqa_pages_fork(const int32_t* block_table, const int32_t* context_lens,
                   const int32_t* parents, int32_t* page_refs, int32_t* out_table,
                   int32_t* out_lens, const mqa_pages_params* params, void* stream) {
    using namespace mqa;
    int rc = check_pages(params, true);
    if (rc != MQA_OK) return rc;
    const mqa_pages_params& p = *params;
    if (p.batch == 0 && p.out_batch == 0) return MQA_OK;
    if (!page_refs || (p.batch > 0 && (!block_table || !context_lens)) ||
        (p.out_batch > 0 && (!parents || !out_table || !out_lens)))
        return fail(MQA_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if (!aligned(block_table, 4) || !aligned(context_lens, 4) || !aligned(parents, 4) ||
        !aligned(page_refs, 4) || !aligned(out_table, 4) || !aligned(out_lens, 4))
        return fail(MQA_ERR_INVALID_ARG, "int32 buffers must be 4-byte aligned");
    const int64_t row = 4ll * p.max_pages_per_row;
    const Buffer all[] = {{out_table, row * p.out_batch}, {out_lens, 4ll * p.out_batch}, {page_refs, 4ll * p.num_pages},
                          {block_table, row * p.batch}, {context_lens, 4ll * p.batch}, {parents, 4ll * p.out_batch}};
    if (any_overlap(all, 3))
        return fail(MQA_ERR_INVALID_ARG, "out_table, out_lens and page_refs must not overlap each other or the inputs");
    uint32_t* lib_status = nullptr;
    rc = check_arch(nullptr, &lib_status);
    if (rc != MQA_OK) return rc;
    const cudaError_t e = launch_fork(block_table, context_lens, parents, page_refs, out_table,
                                      out_lens, pages_args(p, lib_status), stream,
                                      (p.flags & MQA_FLAG_NO_PDL) == 0);
    if (e != cudaSuccess) return cuda_fail(e, "fork launch");
    return MQA_OK;
}

int mqa_pages_resize(int32_t* block_table, int32_t* context_lens, const int32_t* new_lens,
                     int32_t* page_refs, int32_t* copy_src, int32_t* copy_dst,
                     const mqa_pages_params* params, void* stream) {
    using namespace mqa;
    int rc = check_pages(params, true);
    if (rc != MQA_OK) return rc;
    const mqa_pages_params& p = *params;
    if (p.batch == 0) return MQA_OK;
    if (!block_table || !context_lens || !new_lens || !page_refs || !copy_src || !copy_dst)
        return fail(MQA_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if (!aligned(block_table, 4) || !aligned(context_lens, 4) || !aligned(new_lens, 4) ||
        !aligned(page_refs, 4) || !aligned(copy_src, 4) || !aligned(copy_dst, 4))
        return fail(MQA_ERR_INVALID_ARG, "int32 buffers must be 4-byte aligned");
    const int64_t l = 4ll * p.batch;
    const Buffer all[] = {{block_table, l * p.max_pages_per_row}, {context_lens, l}, {page_refs, 4ll * p.num_pages},
                          {copy_src, l}, {copy_dst, l}, {new_lens, l}};
    if (any_overlap(all, 5)) return fail(MQA_ERR_INVALID_ARG, "the buffers must not overlap");
    int dev = 0;
    uint32_t* lib_status = nullptr;
    rc = check_arch(&dev, &lib_status);
    if (rc != MQA_OK) return rc;
    const cudaError_t e = launch_resize(dev, block_table, context_lens, new_lens, page_refs,
                                        copy_src, copy_dst, pages_args(p, lib_status), stream,
                                        (p.flags & MQA_FLAG_NO_PDL) == 0);
    if (e != cudaSuccess) return cuda_fail(e, "resize launch");
    return MQA_OK;
}

int mqa_pages_compact(int32_t* block_table, const int32_t* context_lens, int32_t* page_refs,
                      int32_t* copy_src, int32_t* copy_dst, int32_t* count, int32_t* page_map,
                      const mqa_pages_params* params, void* stream) {
    using namespace mqa;
    int rc = check_pages(params, true);
    if (rc != MQA_OK) return rc;
    const mqa_pages_params& p = *params;
    const bool lists = p.num_pages >= 2;
    if (!page_refs || !count || !page_map || (lists && (!copy_src || !copy_dst)) ||
        (p.batch > 0 && (!block_table || !context_lens)))
        return fail(MQA_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if (!aligned(block_table, 4) || !aligned(context_lens, 4) || !aligned(page_refs, 4) ||
        !aligned(copy_src, 4) || !aligned(copy_dst, 4) || !aligned(count, 4) || !aligned(page_map, 4))
        return fail(MQA_ERR_INVALID_ARG, "int32 buffers must be 4-byte aligned");
    const int64_t l = 4ll * p.batch, half = p.num_pages / 2 * 4ll;
    const Buffer all[] = {{block_table, l * p.max_pages_per_row}, {page_refs, 4ll * p.num_pages}, {copy_src, half},
                          {copy_dst, half}, {count, 4}, {page_map, 4ll * p.num_pages}, {context_lens, l}};
    if (any_overlap(all, 6)) return fail(MQA_ERR_INVALID_ARG, "the buffers must not overlap");
    uint32_t* lib_status = nullptr;
    rc = check_arch(nullptr, &lib_status);
    if (rc != MQA_OK) return rc;
    const cudaError_t e = launch_compact(block_table, context_lens, page_refs, copy_src, copy_dst,
                                         count, page_map, pages_args(p, lib_status), stream,
                                         (p.flags & MQA_FLAG_NO_PDL) == 0);
    if (e != cudaSuccess) return cuda_fail(e, "compact launch");
    return MQA_OK;
}

int mqa_pages_copy(void* const* caches, const int64_t* page_bytes, int32_t num_caches,
                   const int32_t* src, const int32_t* dst, int32_t n, const int32_t* count,
                   const mqa_pages_params* params, void* stream) {
    using namespace mqa;
    int rc = check_pages(params, false);
    if (rc != MQA_OK) return rc;
    if (n < 0) return fail(MQA_ERR_INVALID_ARG, "n must be >= 0 (got %d)", n);
    if (num_caches < 1 || num_caches > MQA_PAGES_MAX_CACHES)
        return fail(MQA_ERR_INVALID_ARG, "num_caches must be in 1..%d (got %d)",
                    MQA_PAGES_MAX_CACHES, num_caches);
    if (!caches || !page_bytes || (n > 0 && (!src || !dst)))
        return fail(MQA_ERR_INVALID_ARG, "a pointer is NULL");
    if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(count, 4))
        return fail(MQA_ERR_INVALID_ARG, "int32 buffers must be 4-byte aligned");
    CopyArgs a;
    for (int i = 0; i < num_caches; ++i) {
        if (!caches[i] || !aligned(caches[i], 16))
            return fail(MQA_ERR_INVALID_ARG, "cache %d must be a 16-byte aligned pointer", i);
        if (page_bytes[i] < 16 || page_bytes[i] % 16 || page_bytes[i] > (1ll << 30))
            return fail(MQA_ERR_INVALID_ARG,
                        "page_bytes[%d] must be a multiple of 16, at most 2^30 (got %lld)", i,
                        (long long)page_bytes[i]);
        a.cache[i] = caches[i];
        a.chunks[i] = (uint32_t)(page_bytes[i] / 16);
    }
    if (n == 0) return MQA_OK;
    uint32_t* lib_status = nullptr;
    rc = check_arch(nullptr, &lib_status);
    if (rc != MQA_OK) return rc;
    a.status = {lib_status, params->status, with_env(params->flags)};
    a.src = src;
    a.dst = dst;
    a.count = count;
    a.n = n;
    a.num_caches = num_caches;
    a.num_pages = params->num_pages;
    const cudaError_t e = launch_copy(a, stream, (params->flags & MQA_FLAG_NO_PDL) == 0);
    if (e != cudaSuccess) return cuda_fail(e, "copy launch");
    return MQA_OK;
}

}  // extern "C"
