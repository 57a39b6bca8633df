/*
 * mqa_cache.h -- the cache around the logits: writing new tokens into the paged
 * caches, softmax attention over a cache held in 4 bits (every cached token, or
 * the tokens that mqa_logits_topk selected), and the life of the pages
 * (forking, growing, freeing, compacting, copying).
 *
 * The conventions of mqa_logits.h hold: device pointers except the params
 * structs (and what is marked HOST), buffers owned by the caller, nothing
 * allocated, asynchronous on `stream`, capturable in a CUDA graph, MQA_OK or a
 * negative mqa_status with mqa_logits_last_error(), status bits instead of traps.
 * Every kernel bounds what it reads from the device (lengths, page numbers,
 * token lists): a bad value is clamped or skipped in every mode, and raises a
 * status bit in validate mode (MQA_FLAG_VALIDATE).
 *
 * The FP4 page format, per page and kv head: page_size rows of D e2m1 codes
 * packed two per byte (even element in the low nibble), then page_size rows of
 * D/16 e4m3 scales (one per 16 consecutive elements); value = code * scale. A
 * page holds its heads one after the other, so with one head it is exactly the
 * page that paged_mqa_logits_fp4 reads. The FP8 page format is that of
 * paged_mqa_logits_fp8.
 */
#ifndef MQA_CACHE_H_
#define MQA_CACHE_H_

#include "mqa_logits.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MQA_DTYPE_BF16 0
#define MQA_DTYPE_F16 1

/* ------------------------------------------------------------ attention */

typedef struct mqa_attention_params {
    int32_t batch;              /* B, 0..32768 */
    int32_t next_n;             /* query positions per row, 1..4 */
    int32_t num_heads;          /* H query heads */
    int32_t num_kv_heads;       /* Hk <= 4096, divides H; H / Hk * next_n <= 128 (topk > 0: H / Hk <= 128) */
    int32_t head_dim;           /* D: 64 or 128 */
    int32_t page_size;          /* a power of two, 16..256 */
    int32_t num_pages;          /* pages in each of k_cache and v_cache */
    int32_t max_pages_per_row;  /* row stride of block_table; times page_size <= 2^31 - 2^16 */
    int32_t topk;               /* 0: every cached token; else the length of the token lists, <= 2^31 - 2^16 */
    int32_t num_ctas;           /* topk == 0: the value given to mqa_logits_schedule */
    int32_t dtype;              /* MQA_DTYPE_* of q and out */
    uint32_t flags;             /* MQA_FLAG_VALIDATE, MQA_FLAG_NO_PDL */
    float softmax_scale;        /* multiplies q . k */
    int32_t reserved;           /* 0 */
    int64_t q_stride_b, q_stride_n, q_stride_h; /* of q, in elements; multiples of 8 */
    uint64_t workspace_bytes;   /* size of workspace */
    int32_t* status;            /* optional device int32 for MQA_STATUS_* bits; may be NULL */
} mqa_attention_params;

/*
 * Attention of next_n query positions a row over the paged cache:
 *
 *   out[b][n][h] = sum_t p_t v_t,  p = softmax over the visible t of softmax_scale * q[b][n][h] . k_t,
 *
 * with k_t, v_t of kv head h / (H / Hk). Visible are the tokens t < ctx_bn (as
 * for the logits), or with topk > 0 the entries of indices[b][n] with
 * 0 <= t < ctx_bn; other entries (-1 among them) may stand anywhere in the list
 * and are skipped, and a token listed twice counts twice. A position that sees
 * no token gets out = 0 and lse = -inf. What lies in slots that a position does
 * not see (NaN scales among it) never reaches its result.
 *
 * q:            device bf16 or f16 [B][next_n][H][D] with the strides of params
 *               (D contiguous), 16-byte aligned. The kernels multiply in f16:
 *               a bf16 row (b, n, h) is first scaled by a power of two, undone
 *               on the scores, so it is exact down to 2^-31 of the row's largest.
 *               Finite values are expected, and scores within +-2^26.
 * k_cache, v_cache: device bytes [num_pages][Hk][page_size * (D/2 + D/16)],
 *               16-byte aligned, FP4 pages; they may be the same buffer.
 * block_table, context_lens: as for paged_mqa_logits_fp4.
 * schedule:     topk == 0: device int32 [(num_ctas + 1) * 2] of
 *               mqa_logits_schedule for these context_lens (its reuse rule
 *               holds); else unused, may be NULL.
 * indices:      topk > 0: device int32 [B][next_n][topk]; else NULL.
 * out:          device, type of q, [B][next_n][H][D], 16-byte aligned, written whole.
 * lse:          NULL, or device fp32 [B][next_n][H]: the natural logarithm of
 *               sum_t exp(softmax_scale * q . k_t).
 * workspace:    device, 16-byte aligned, at least mqa_attention_workspace_size
 *               bytes: partial results of rows that several CTAs share. Its
 *               contents mean nothing between calls, but two calls that can run
 *               at the same time (two streams, two graphs) need one each.
 */
int paged_mqa_attention_fp4(const void* q, const void* k_cache, const void* v_cache,
                            const int32_t* block_table, const int32_t* context_lens,
                            const int32_t* schedule, const int32_t* indices, void* out,
                            float* lse, void* workspace, const mqa_attention_params* params,
                            void* stream);

/* Bytes of workspace that a call with these params, or with a smaller batch or
 * next_n, needs on the current device (HOST *bytes; workspace_bytes, strides,
 * status and flags are not looked at). */
int mqa_attention_workspace_size(const mqa_attention_params* params, uint64_t* bytes);

/* ------------------------------------------------------------ appending */

typedef struct mqa_append_params {
    int32_t batch;              /* B >= 0 */
    int32_t num_tokens;         /* T: rows of the new tokens' tensors */
    int32_t num_kv_heads;       /* Hk (fp8: 1) */
    int32_t head_dim;           /* D: fp8 32, 64 or 128; fp4 64 or 128 */
    int32_t page_size;          /* a power of two, 8..256 (fp4: 16..256) */
    int32_t num_pages;
    int32_t max_pages_per_row;
    int32_t dtype;              /* MQA_DTYPE_* of the tokens and of values */
    uint32_t flags;             /* MQA_FLAG_VALIDATE, MQA_FLAG_NO_PDL */
    int32_t reserved;           /* 0 */
    int64_t k_stride_t, k_stride_h, v_stride_t, v_stride_h; /* elements; multiples of 8 */
    int32_t* status;            /* optional, may be NULL */
} mqa_append_params;

/*
 * Quantises new tokens and writes them to the last positions of their rows: row
 * b's tokens are i = row_offsets[b] .. row_offsets[b+1]-1, and the last of them
 * becomes position context_lens[b] - 1 (context_lens counts the new tokens
 * already, as the logits and attention calls that follow expect). With
 * row_offsets NULL every row has T / B tokens (T a multiple of B). Tokens before
 * row_offsets[0] and at or behind row_offsets[B] (a slice of a batch's offsets, a
 * padded batch) belong to no row and are not written. A token whose
 * position is negative, behind the block table or on a page outside
 * [0, num_pages) is not written (validate mode: MQA_STATUS_BAD_CONTEXT /
 * _BAD_PAGE). Other slots keep their bytes. Two tokens must not have the same
 * slot (rows that share the page that they write to: see mqa_pages_resize).
 *
 * FP8 pages (x device [T][D] with stride k_stride_t): s = 2^e, the least with
 * max|x| / s <= 448 (1 for a zero token, at least 2^-126); codes e4m3 of x / s,
 * to nearest even. A power of two costs e4m3 no precision and makes x / s exact.
 *
 * FP4 pages (k, v device [T][Hk][D]): per 16 elements sc = e4m3 of max|x| / 6 to
 * nearest even, at most 448 and 2^-9 in the place of 0; codes e2m1 of x / sc to
 * nearest even, at most 6, zero without a sign. v and v_cache may both be NULL
 * (a cache of keys alone, as paged_mqa_logits_fp4 reads it).
 *
 * values, k_values, v_values: NULL, or device [T][Hk][D] contiguous of the
 * tokens' type: what the cache now holds for each written token (exact in bf16,
 * rounded to f16 where that is too narrow); other tokens' rows are left. Caches and
 * values are buffers of their own.
 * Tokens are expected finite.
 */
int mqa_cache_append_fp8(const void* x, void* kv_cache, const int32_t* block_table,
                         const int32_t* context_lens, const int32_t* row_offsets, void* values,
                         const mqa_append_params* params, void* stream);
int mqa_cache_append_fp4(const void* k, const void* v, void* k_cache, void* v_cache,
                         const int32_t* block_table, const int32_t* context_lens,
                         const int32_t* row_offsets, void* k_values, void* v_values,
                         const mqa_append_params* params, void* stream);

/* ------------------------------------------------------------ pages
 * A pool's pages are counted in page_refs, device int32 [num_pages]: how many
 * block-table entries (and other holders of the caller's) point at each; 0 is a
 * free page. Row b's pages are block_table[b][0 .. ceil(len_b / page_size) - 1],
 * lengths are clamped to [0, max_pages_per_row * page_size]. Table entries
 * outside [0, num_pages) are skipped (validate mode: MQA_STATUS_BAD_PAGE).
 * What a call writes may overlap none of its other buffers. Results do not
 * depend on the order in which threads run. */

typedef struct mqa_pages_params {
    int32_t batch;              /* rows of block_table, 0..32768 */
    int32_t out_batch;          /* mqa_pages_fork: rows of out_table, 0..32768; else 0 */
    int32_t max_pages_per_row;  /* row stride of the tables */
    int32_t num_pages;
    int32_t page_size;          /* tokens, a power of two, 8..256 */
    uint32_t flags;             /* MQA_FLAG_VALIDATE, MQA_FLAG_NO_PDL */
    int32_t* status;            /* optional, may be NULL */
} mqa_pages_params;

/*
 * Fork: row r of the new batch goes on from row parents[r] of the old one,
 * sharing all its pages; parents[r] outside [0, batch) makes an empty row. Writes
 * out_table [out_batch][max_pages_per_row] (-1 behind a row's pages) and out_lens
 * [out_batch] whole, and counts page_refs from the old table's references to the
 * new one's: what no row goes on from is freed. parents device int32 [out_batch].
 */
int mqa_pages_fork(const int32_t* block_table, const int32_t* context_lens,
                   const int32_t* parents, int32_t* page_refs, int32_t* out_table,
                   int32_t* out_lens, const mqa_pages_params* params, void* stream);

/*
 * Resize: every row gets the length new_lens[b], in place. A row that shrinks
 * gives its pages behind the new end back (their entries become -1; 0 frees the
 * row). A row that grows takes pages, and if its last page is partly filled and
 * shared, it takes a page in that one's place: copy_src[b], copy_dst[b] (device
 * int32 [batch], else -1) name the copy that mqa_pages_copy has to make before
 * the row is written to. Pages taken are the lowest that were free before the
 * call, in the order of the rows and of the pages in them; what the call frees
 * is free from the next call on. A row whose pages, with all rows' before it, are
 * more than were free keeps its length, table and pages, and MQA_STATUS_NO_PAGES
 * is raised. context_lens is set to the lengths that came about.
 */
int mqa_pages_resize(int32_t* block_table, int32_t* context_lens, const int32_t* new_lens,
                     int32_t* page_refs, int32_t* copy_src, int32_t* copy_dst,
                     const mqa_pages_params* params, void* stream);

/*
 * Compact: with N pages in use (page_refs > 0), those numbered N and above move
 * to the free ones below N, in ascending order: copy_src[i] -> copy_dst[i] for
 * i < *count (device int32 [num_pages / 2], -1 behind; count device int32 [1]),
 * which mqa_pages_copy has to copy. page_refs and block_table are set to the new
 * numbers, page_map (device int32 [num_pages]) gives each old page's new number,
 * -1 for a free page.
 */
int mqa_pages_compact(int32_t* block_table, const int32_t* context_lens, int32_t* page_refs,
                      int32_t* copy_src, int32_t* copy_dst, int32_t* count, int32_t* page_map,
                      const mqa_pages_params* params, void* stream);

#define MQA_PAGES_MAX_CACHES 256
/*
 * Copies pages src[i] -> dst[i], i < n, in each of num_caches pools: caches is a
 * HOST array of device pointers (16-byte aligned), page_bytes a HOST array of
 * their pages' sizes (multiples of 16). count: NULL, or device int32: only
 * i < *count. Pairs with either outside [0, num_pages) are skipped (where that is -1
 * silently, other numbers raise MQA_STATUS_BAD_PAGE in validate mode). A page must not be a
 * destination twice, nor source and destination in one call. params: num_pages,
 * flags and status are looked at.
 */
int mqa_pages_copy(void* const* caches, const int64_t* page_bytes, int32_t num_caches,
                   const int32_t* src, const int32_t* dst, int32_t n, const int32_t* count,
                   const mqa_pages_params* params, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MQA_CACHE_H_ */
