/*
 * clef_cache.h — C ABI of the paged 4-bit memory cache on GB300 (sm_103a).
 *
 * The head's memory keys and values are its largest intermediate and its dominant cost
 * (clef_head.h: two routing layers of width 1024 make 8 KB of bf16 per memory row).  A
 * record's state comes before its schema in the prompt ("clef-flash-CoreAI
 * metadata.json" decision.prompt.layout) and the backbone is causal, so the rows of the
 * state do not change when another schema is asked of the same record.  The cache keeps
 * them between calls in 4 bits a value, in pages that the requests of a batch share out
 * among themselves: page accounts built on the GPU from request lengths, a store that
 * quantises rows into their slots, a read back, and attention straight over the 4-bit
 * pages.  clef_memory_store and clef_stream_finish_memory are the head's own path over it.
 *
 * Conventions are those of clef_head.h: caller-owned device memory, host-side validation
 * before any launch, a clef_status from every entry point, all work asynchronous on
 * `stream` of the current device, nothing allocated, every call capturable into a CUDA
 * graph.  Lengths, tables and slots are DEVICE memory, read by the kernels: a captured
 * call follows their contents at replay time.  `flags` is a device int32 that the caller
 * clears (or passes to clef_cache_status, which reads and clears it); kernels only set bits
 * in it.
 */
#ifndef CLEF_CACHE_H
#define CLEF_CACHE_H

#include "clef_head.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the keys, values and queries that go in and out. */
typedef enum clef_dtype {
    CLEF_BF16 = 0,
    CLEF_FP16 = 1,
    CLEF_FP32 = 2 /* clef_cache_read only */
} clef_dtype;

/* A cache: `n_pages` pages of `page` tokens (a power of two, 16 to 256) of `heads` key/value
 * heads (1 to 1024; the heads of several layers may lie side by side) of `head_dim` 64 or
 * 128 values.  Slot s is token s % page of page s / page; n_pages * page < 2^31.
 *
 * Stored form.  Each run of 64 values of a token's head is one group with a scale s and a
 * minimum m, in bf16, and 4-bit codes c; a value stands for s c + m.
 *   m = bf16(min x),  s = bf16(max(max x - m, 0) / 15),  c = clamp(rint((x - m) / s), 0, 15),
 * in fp32, roundings to nearest even, c = 0 where s = 0.  A group whose values or range are
 * not finite gets s = m = NaN and so reads back as NaN, alone: other groups are not
 * touched by it.  4.5 bits a value; an error of at most s / 2 plus the rounding of m and s.
 *
 * Layout of `data` (256-byte aligned, clef_cache_size bytes): piece [page][head][page / 16],
 * each 1152 * (head_dim / 64) bytes for 16 tokens: key codes, value codes (512 bytes each
 * per 64 values), then for each token and group four bf16: key scale, key minimum, value
 * scale, value minimum.  A byte holds the codes of values d (low four bits) and d + 8 of one
 * token, d in the lower half of a run of 16.  Within 512 bytes, key codes keep token
 * 8 hi + g, byte 8 ks + 2 t + e of the token's group at 64 g + 16 t + 4 ks + 2 e + hi;
 * value codes keep token 8 hi + 2 t + e, byte 8 ks + g at that place: the order in which a
 * warp's matrix instruction takes them, so that attention reads 16 bytes a lane and splits
 * them in registers.  A byte never holds two tokens. */
typedef struct clef_cache {
    void* data;
    int32_t n_pages;
    int32_t page;
    int32_t heads;
    int32_t head_dim;
} clef_cache;

/* Most requests (block-table rows) of one plan or attention call. */
#define CLEF_CACHE_MAX_REQUESTS 1024

/* Bytes of `data` for this cache (its `data` pointer is not looked at). */
CLEF_API int clef_cache_size(const clef_cache* cache, size_t* bytes);

/* Page accounts of a step: request lengths go from lengths[b] to want[b].
 *   lengths      int32 [B], in and out: tokens that request b holds.
 *   want         int32 [B]: tokens that it is to hold after the call.
 *   block_table  int32 [B][table_stride]: the pages of request b in order, in and out;
 *                entries past its last page are -1.  0 <= lengths, want <= table_stride * page.
 *   free_pages   int32 [n_pages], free_count int32 [1]: a stack of the pages that nobody
 *                holds, in and out; entries at and past the count are -1.
 *   cu_new       int32 [B + 1], out: running sum of the tokens that each request gained.
 *   slots        int32 [n_slots], out: the slot of every gained token, request by request
 *                (the row order of clef_cache_append); -1 behind the last one.
 * First every request that shrinks gives back its pages, the highest request and its last
 * page first; then the growing requests take pages from the top of the stack, the lowest
 * request and its next page first (so a step that is taken back leaves the stack as it
 * was).  When the pages run out, that request and all later ones that need a page keep
 * their old length (they gain no token), and the status is CLEF_ERR_NO_PAGES.  A length out
 * of range leaves its request as it is, and gained tokens past n_slots get no slot: both are
 * CLEF_ERR_DEVICE_BOUNDS.  One page must not be held twice; the kernels' accesses stay in
 * bounds whatever the tables hold.  The arrays must not overlap, and each starts on 4 bytes.
 * 1 <= B <= CLEF_CACHE_MAX_REQUESTS, 1 <= table_stride, table_stride * page <= 2^31 - 65536,
 * B * table_stride and n_slots at most 2^30. */
CLEF_API int clef_cache_plan(const clef_cache* cache, int32_t B, int32_t* lengths, const int32_t* want,
                             int32_t* block_table, int32_t table_stride, int32_t* free_pages, int32_t* free_count,
                             int32_t* cu_new, int32_t* slots, int32_t n_slots, int32_t* flags, void* stream);

/* Quantises key and value rows into the cache.
 *   k, v        [n_tokens][n_heads][head_dim] of `dtype` (bf16 or fp16), each with its own
 *               row and head strides in elements; values of a head are contiguous.  Rows and
 *               heads may start at any element (16-byte aligned ones load faster).
 *   slots       int32 [n_tokens]: slot of every row; a negative one skips the row, one past
 *               the cache is skipped and CLEF_ERR_DEVICE_BOUNDS.  No slot twice in one call
 *               (that token then holds a mixture of the rows).
 * The heads go to cache heads head0 .. head0 + n_heads - 1.  Tokens of other slots keep
 * their bits.  A captured or eager append may run beside reads of other slots, not of its
 * own. */
CLEF_API int clef_cache_append(const clef_cache* cache, int32_t n_tokens, int32_t head0, int32_t n_heads, int32_t dtype,
                               const void* k, int64_t k_row_stride, int64_t k_head_stride, const void* v,
                               int64_t v_row_stride, int64_t v_head_stride, const int32_t* slots, int32_t* flags,
                               void* stream);

/* The values that stored rows stand for: k, v [n_tokens][n_heads][head_dim], contiguous,
 * 16-byte aligned, of `dtype` (bf16, fp16 or fp32; one rounding from fp32; fp16 values past
 * its range become infinite), of slots[i].  A row whose slot is negative is set to zero;
 * one past the cache is too, and CLEF_ERR_DEVICE_BOUNDS. */
CLEF_API int clef_cache_read(const clef_cache* cache, int32_t n_tokens, int32_t head0, int32_t n_heads, int32_t dtype,
                             const int32_t* slots, void* k, void* v, int32_t* flags, void* stream);

/* Workspace bytes of clef_cache_attend for these sizes (0 when none is needed).
 * max_length is table_stride * page of the call. */
CLEF_API int clef_cache_attend_workspace(const clef_cache* cache, int32_t B, int32_t total_q, int32_t q_heads,
                                         int32_t max_length, size_t* bytes);

/* Attention of a ragged batch of queries over the cache:
 *   o = sum_j softmax_j(scale q . k_j) v_j,  lse = ln sum_j exp(scale q . k_j),
 * over the keys j of the query's request.
 *   q            [total_q][q_heads][head_dim] of `dtype` (bf16 or fp16), row stride
 *                q_row_stride and head stride q_head_stride in elements, both even and the
 *                base 4-byte aligned.  q_heads = kv_heads * a whole number; query head h
 *                reads cache head head0 + h / (q_heads / kv_heads).
 *   cu_q         int32 [B + 1], non-decreasing from 0: the query rows of request b are
 *                cu_q[b] .. cu_q[b + 1] - 1, at most max_q of them (from 0 on).
 *   block_table, table_stride, lengths: as clef_cache_plan leaves them.  Request b has keys
 *                0 .. lengths[b] - 1.
 *   causal       0: every query sees all keys of its request.  1: the queries are the last
 *                tokens of the request; query i of n sees keys 0 .. lengths[b] - n + i.
 *   out          [total_q][q_heads][head_dim] of `dtype`, contiguous, 4-byte aligned; lse
 *                fp32 [total_q][q_heads], or NULL.  Both lie apart from each other and from q,
 *                from its first value to its last.
 * A query that sees no key (an empty request, or one with fewer keys than queries) gets
 * out = 0, lse = -inf.  Rows at and behind cu_q[B] are left as they were.
 * Scores, softmax and sums are fp32.  For the product with the values, softmax weights are
 * rounded to 11 bits for bf16 queries and to 22 for fp16 ones, relative to the row's own
 * largest product of weight and value scale; for bf16 queries of requests of many rows (queries x
 * query heads a key/value head: over 32 at head_dim 64, over 16 at 128) the values are rounded to
 * 11 bits too, twice.  The output is rounded once.  A row's result depends on nothing but its
 * own request and the keys that it sees: not on the batch, nor on the width of the table, and
 * bit for bit the same from call to call.  Query values are below 2^118 in magnitude (larger
 * ones give scores that are too small), stored values below 2^108 (sums of larger ones may
 * overflow fp32).
 * A table entry outside the cache hides its tokens, a length or cu_q out of range is cut
 * to it, each with CLEF_ERR_DEVICE_BOUNDS.
 * workspace: clef_cache_attend_workspace bytes, 256-byte aligned (may be NULL when 0);
 * calls that overlap on the GPU need one each, captured graphs included.
 * 1 <= B <= CLEF_CACHE_MAX_REQUESTS; 0 <= max_q <= total_q, max_q * q_heads at most 2^31 - 65536 (and
 * so are the work items and partial rows of a call, else CLEF_ERR_UNSUPPORTED_CONFIG); scale finite. */
CLEF_API int clef_cache_attend(const clef_cache* cache, int32_t B, int32_t total_q, int32_t max_q, int32_t q_heads,
                               int32_t head0, int32_t kv_heads, int32_t dtype, const void* q, int64_t q_row_stride,
                               int64_t q_head_stride, const int32_t* cu_q, const int32_t* block_table,
                               int32_t table_stride, const int32_t* lengths, float scale, int32_t causal, void* out,
                               float* lse, int32_t* flags, void* workspace, size_t workspace_bytes, void* stream);

/* Waits for `stream`, then reads and clears `flags`: CLEF_OK, CLEF_ERR_DEVICE_TIMEOUT (a wait of a 4-bit
 * product, clef_fp4.h, ran out), CLEF_ERR_DEVICE_BOUNDS or CLEF_ERR_NO_PAGES (the first of these that happened). */
CLEF_API int clef_cache_status(int32_t* flags, void* stream);

/* ---- the head over kept memory.
 * The cache of a head has head_dim 64 and heads = n_route * cfg->heads: head l * cfg->heads
 * + h is head h of routing layer l.
 *
 * clef_memory_store quantises the K/V of rows [row0, row0 + n_rows) of record `record` of
 * every routing layer, as clef_stream_rows (same schema, workspace and stream) or
 * clef_head_forward left them in the workspace, into the cache's slots
 * slots[0 .. n_rows - 1] (device int32).  Errors as clef_stream_rows; a cache of another shape is
 * CLEF_ERR_INVALID_ARGUMENT. */
CLEF_API int clef_memory_store(const clef_config* cfg, const clef_schema* schema, int32_t record, int32_t row0,
                               int32_t n_rows, const void* workspace, size_t workspace_bytes, const clef_cache* cache,
                               const int32_t* slots, int32_t* flags, void* stream);

/* clef_stream_finish with the memory read from the cache: record b's rows 0 .. lengths[b] - 1
 * are the tokens of row b of block_table.  Only rows from first_row[b] on (host int32 [B],
 * 0 <= first_row[b] < lengths[b]) need have gone through clef_stream_rows on this workspace (with
 * clef_stream_begin before them): the kept rows before them are read from the cache alone.
 * Every question and option span must start at or behind first_row of its record
 * (pooling reads the statistics of those rows) else CLEF_ERR_INVALID_ARGUMENT; table_stride *
 * page must cover the longest record.  hidden_dtype: CLEF_BF16 or CLEF_FP16 rows, as they
 * were streamed.  attend_workspace: clef_cache_attend_workspace(cache, B, O, heads,
 * table_stride * page) bytes.  Outputs as clef_stream_finish, with the memory's keys and
 * values rounded to the cache's 4 bits. */
CLEF_API int clef_stream_finish_memory(const clef_config* cfg, const void* const* weights, const void* prepared,
                                       const clef_schema* schema, const int32_t* first_row, const void* hidden,
                                       int32_t hidden_dtype, const int32_t* token_ids, const uint16_t* lexical,
                                       float* logits, float* probs, float* q_value, float* q_conf, int32_t* q_argmax,
                                       void* workspace, size_t workspace_bytes, const clef_cache* cache,
                                       const int32_t* block_table, int32_t table_stride, int32_t* flags,
                                       void* attend_workspace, size_t attend_workspace_bytes,
                                       const clef_debug_outputs* debug, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CLEF_CACHE_H */
