/*
 * dspark_paged.h -- the paged key-value cache around a speculative step, in
 * libdspark (one GB300 GPU, sm_103a).
 *
 * The scheduler (dspark.h) gives request r a verify length l_r, so the target
 * runs over l_r + 1 new tokens of the request. Between the scheduler and the
 * verification stand four calls, all on the device, in this order:
 *   dspark_pages_reserve    pages, slots and positions for the new tokens, and
 *                           the row offsets that dspark_verify reads;
 *   dspark_kv_append        the new tokens' keys and values into the cache;
 *   dspark_paged_attention  attention of the new tokens over the cache;
 *   dspark_pages_release    (after the verification) the pages that only
 *                           rejected tokens used, and those of finished
 *                           requests, back to the free pages.
 *
 * The cache is a pool of num_pages pages of page_size tokens. block_table[r][i]
 * names the page of request r's tokens i*page_size .. (i+1)*page_size - 1; the
 * ids that no request holds form a stack, free_pages[0 .. *free_count - 1]
 * (top last), in an array of num_pages entries. Keys (and values, in a buffer
 * of their own with the same strides) of token t of page p and head h start at
 * element p*page_stride + t*token_stride + h*head_stride, their D elements
 * contiguous; so both [pages][page_size][heads][D] and
 * [pages][heads][page_size][D] are such layouts.
 *
 * Conventions are those of dspark.h: caller-owned device pointers, no
 * allocation, no synchronisation, host errors as return codes before anything
 * is launched, data errors in *device_status, CUDA-graph capturable after one
 * call outside a capture. page_size is a power of two, 8..1024;
 * num_pages >= 1 and num_pages * page_size <= 2^31 - 1.
 */
#ifndef DSPARK_PAGED_H
#define DSPARK_PAGED_H

#include "dspark.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of keys, values, queries and attention outputs next to
   DSPARK_BF16: IEEE half precision (not a type of logits). */
#define DSPARK_F16 2
/* *device_status of dspark_pages_reserve: the free pages ran out. */
#define DSPARK_ERR_NO_PAGES 7

/* Query rows (new tokens x query heads per key head) that one pass over a
   request's keys serves, at most; more rows take more passes. */
#define DSPARK_PAGED_MAX_ROWS 160
/* Most CTAs that dspark_paged_attention launches. */
#define DSPARK_PAGED_MAX_CTAS 320

/* Rows of a partial result of dspark_paged_attention, at most. */
#define DSPARK_PAGED_ROWS(Hq, Hkv, max_new)                                        \
  (16u * DSPARK_CEILDIV((size_t)((Hq) / (Hkv)) * (size_t)(max_new), 16u) <         \
           DSPARK_PAGED_MAX_ROWS                                                   \
       ? 16u * DSPARK_CEILDIV((size_t)((Hq) / (Hkv)) * (size_t)(max_new), 16u)     \
       : (size_t)DSPARK_PAGED_MAX_ROWS)
/* Workspace of dspark_paged_attention, in bytes: one record per CTA, and for
   the two requests that a CTA may share with its neighbours a partial
   maximum, sum (8 bytes) and output row (D floats) per query row. */
#define DSPARK_PAGED_ATTENTION_WS_BYTES(Hq, Hkv, max_new, D)                       \
  (DSPARK_ALIGN256((size_t)DSPARK_PAGED_MAX_CTAS * 64u) +                          \
   2u * (size_t)DSPARK_PAGED_MAX_CTAS * DSPARK_PAGED_ROWS(Hq, Hkv, max_new) *      \
       ((size_t)(D) * 4u + 8u))

/*
 * dspark_pages_reserve -- pages, slots and row offsets for one step's new
 * tokens. Request r holds context_len[r] tokens in ceil(context_len[r] /
 * page_size) pages and gets n_r = new_len[r] + extra more (extra = 1 when
 * new_len is the scheduler's verify_len: the anchor comes first). Requests are
 * served in order; new pages are popped from the stack in order of (request,
 * position). The first request that does not fit (its tokens in max_tokens,
 * its pages in the free pages) and all requests after it get nothing, and
 * *device_status says why (DSPARK_ERR_TOO_LARGE, DSPARK_ERR_NO_PAGES).
 *
 * Arguments
 *   context_len   [B] int32 >= 0; new_len [B] int32; extra >= 0. A request with
 *                 new_len < 0, or whose context_len + n_r exceeds max_pages *
 *                 page_size, gets nothing (DSPARK_ERR_BAD_DATA), others do.
 *   block_table   [B][max_pages] int32, in/out, rows table_stride entries
 *                 apart: new entries are written, others left as they are.
 *   free_pages, free_count   the stack; read only (its top *free_count -
 *                 *free_count_out entries now belong to requests).
 *   max_tokens    rows of slot_map and positions, 0 .. 2^30.
 * Outputs
 *   context_out   [B] int32: context_len + n_r (context_len where nothing was
 *                 given). May be context_len itself.
 *   row_off       [B+1] int64: sum of the n before r: dspark_verify's
 *                 target_row_off when extra = 1, and the rows of the attention.
 *   draft_off     [B+1] int64 or NULL: sum of the new_len before r (of requests
 *                 that got theirs): dspark_verify's draft_row_off.
 *   slot_map      [max_tokens] int32: page * page_size + offset of each new
 *                 token, -1 past the last. A page id outside the pool (from the
 *                 stack or the table) gives num_pages * page_size, which the
 *                 other calls refuse, and DSPARK_ERR_BAD_DATA.
 *   positions     [max_tokens] int32 or NULL: each new token's position, -1
 *                 past the last.
 *   free_count_out [1] int32. May be free_count itself.
 *   device_status  [1] int32 (required).
 * Calling it again with the same inputs gives the same outputs (unless they
 * overwrite the inputs). No workspace; one launch, and a second one of one CTA where
 * an output is written over an input.
 */
int dspark_pages_reserve(const int32_t* context_len, const int32_t* new_len, int32_t extra,
                         int32_t B, int32_t page_size, int32_t num_pages, int32_t* block_table,
                         int64_t table_stride, int32_t max_pages, const int32_t* free_pages,
                         const int32_t* free_count, int32_t max_tokens, int32_t* context_out,
                         int64_t* row_off, int64_t* draft_off, int32_t* slot_map,
                         int32_t* positions, int32_t* free_count_out, int32_t* device_status,
                         struct CUstream_st* stream);

/*
 * dspark_pages_release -- after the verification: request r keeps
 * context_len[r] + kept_len[r] + extra of its reserved_len[r] tokens (kept_len
 * = accepted_len, extra = 1: the anchor and the accepted drafts), or none when
 * kept_len[r] = -1 (the request is finished). The pages past the kept tokens
 * are pushed on the stack in order of (request, position).
 *
 * Arguments
 *   context_len   [B] int32: tokens before the reservation (its input).
 *   reserved_len  [B] int32: tokens after it (its context_out). Where both are
 *                 equal (nothing was given), kept_len counts as -extra unless it
 *                 is -1.
 *   kept_len      [B] int32, -1 <= kept_len, kept_len + extra <= reserved_len -
 *                 context_len; else the request keeps everything and
 *                 *device_status is DSPARK_ERR_BAD_DATA.
 *   block_table   [B][max_pages] int32, read only. Page ids are pushed as they
 *                 are (dspark_pages_reserve judges them).
 *   free_pages    [num_pages] int32, in/out; free_count [1] int32. A push past
 *                 the array is dropped (DSPARK_ERR_BAD_DATA).
 * Outputs
 *   context_out   [B] int32: tokens kept. May be context_len or reserved_len.
 *   free_count_out [1] int32. May be free_count itself.
 * Calling it again with the same inputs gives the same outputs (unless they
 * overwrite the inputs). No workspace; one launch, and a second one of one CTA where
 * an output is written over an input.
 */
int dspark_pages_release(const int32_t* context_len, const int32_t* reserved_len,
                         const int32_t* kept_len, int32_t extra, int32_t B, int32_t page_size,
                         int32_t num_pages, const int32_t* block_table, int64_t table_stride,
                         int32_t max_pages, int32_t* free_pages, const int32_t* free_count,
                         int32_t* context_out, int32_t* free_count_out, int32_t* device_status,
                         struct CUstream_st* stream);

/*
 * dspark_kv_append -- keys and values of new tokens into the cache: row i of k
 * and v goes to slot slot_map[i] (page slot / page_size, token slot %
 * page_size); rows with a negative slot are skipped; a slot of num_pages *
 * page_size or more is skipped and sets DSPARK_ERR_BAD_DATA. Slots that occur
 * twice leave either row.
 *
 * Arguments
 *   k, v          dtype (DSPARK_BF16, DSPARK_F16): head h of row i at element
 *                 i*row_stride + h*in_head_stride, D contiguous; the same
 *                 strides for both.
 *   n >= 0 rows, Hkv >= 1 heads, D = 64 or 128.
 *   k_cache, v_cache, page_stride, token_stride, head_stride: the cache.
 *   All pointers 16-byte aligned, all strides multiples of 8 elements, >= 0.
 * No workspace; one launch.
 */
int dspark_kv_append(const void* k, const void* v, int64_t row_stride, int64_t in_head_stride,
                     const int32_t* slot_map, int32_t n, int32_t Hkv, int32_t D, int32_t dtype,
                     void* k_cache, void* v_cache, int64_t page_stride, int64_t token_stride,
                     int64_t head_stride, int32_t page_size, int32_t num_pages,
                     int32_t* device_status, struct CUstream_st* stream);

/*
 * dspark_paged_attention -- softmax attention of each request's newest tokens
 * over its pages. Request r has T = row_off[r+1] - row_off[r] new tokens (0 <= T
 * <= max_new), the last T of its context_len[r] cached ones (keys and values
 * already in the cache). New token t of query head h, with the key head h' =
 * h / (Hq / Hkv), sees the cached tokens u with
 *   u <= context_len - T + t, and u > context_len - T + t - window if window > 0,
 *   s_u = scale * <q, K[u][h']>,  out = sum_u e^{s_u} V[u][h'] / sum_u e^{s_u},
 *   lse = log sum_u e^{s_u}.
 * A row that sees no token (t < T - context_len) gives zeros and lse = -inf.
 * Cached values that a row does not see never reach it, whatever they hold
 * (infinities, NaN, memory that was never written).
 *
 * Products of 16-bit inputs are accumulated in binary32 on the tensor cores;
 * the maximum, the sum and the output are binary32; the weights e^{s - m} are
 * rounded to the inputs' type for the second product (their sum is not). m is near
 * the row's largest score: for half precision some nats below it, so that weights
 * keep their bits down to e^-16 of the largest (where scale * |s| is below 2^17);
 * for bf16 at or above it, so that no weight exceeds 1. The
 * output is rounded once. Results depend on the inputs alone, not on timing.
 *
 * Arguments
 *   q             [n_tokens][Hq][D] dtype (DSPARK_BF16, DSPARK_F16): strides
 *                 q_row_stride, q_head_stride in elements, D contiguous.
 *   k_cache, v_cache  dtype, the cache.
 *   block_table   [B][max_pages] int32, rows table_stride entries apart. An id
 *                 outside the pool where a visible token lies sets
 *                 DSPARK_ERR_BAD_DATA (that request's rows are unspecified).
 *   context_len   [B] int32, 0 .. max_pages * page_size.
 *   row_off       [B+1] int64, ascending from >= 0 to <= n_tokens. Rows outside
 *                 every request are not written.
 *   Hq, Hkv       Hq a multiple of Hkv; D = 64 or 128; max_new >= 1. A key head's
 *                 (Hq / Hkv) * max_new query rows are served in passes of up to
 *                 DSPARK_PAGED_MAX_ROWS, side by side, which share the device
 *                 evenly: long prompts belong in calls of their own, without
 *                 requests of few new tokens. More passes than the device has SMs,
 *                 or max_pages * page_size * Hkv past 2^37, are refused.
 *   scale         finite, > 0.
 *   window        visible tokens per new token, itself included; 0: all.
 * Outputs
 *   out           [n_tokens][Hq][D] dtype, contiguous.
 *   lse           [n_tokens][Hq] float32 or NULL (natural logarithm).
 *   device_status [1] int32 (required): DSPARK_OK or a data error;
 *                 DSPARK_ERR_TOO_LARGE (nothing computed) for a batch of 2^31
 *                 units or more (128 tokens of a key head each).
 *   workspace     at least DSPARK_PAGED_ATTENTION_WS_BYTES(Hq, Hkv, max_new, D)
 *                 bytes, 256-byte aligned; no initial contents needed.
 * q, k_cache, v_cache and out must be 16-byte aligned and all strides multiples
 * of 8 elements, >= 0 (tensor memory access); otherwise DSPARK_ERR_INVALID_ARG.
 */
int dspark_paged_attention(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                           const void* k_cache, const void* v_cache, int64_t page_stride,
                           int64_t token_stride, int64_t head_stride, int32_t page_size,
                           int32_t num_pages, const int32_t* block_table, int64_t table_stride,
                           int32_t max_pages, const int32_t* context_len,
                           const int64_t* row_off, int32_t B, int32_t n_tokens, int32_t Hq,
                           int32_t Hkv, int32_t D, int32_t max_new, float scale, int32_t window,
                           int32_t dtype, void* out, float* lse, int32_t* device_status,
                           void* workspace, size_t workspace_bytes, struct CUstream_st* stream);

#ifdef __cplusplus
}
#endif

#endif /* DSPARK_PAGED_H */
