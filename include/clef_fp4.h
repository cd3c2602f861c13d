/*
 * clef_fp4.h — C ABI of the microscaled 4-bit operators on GB300 (sm_103a).
 *
 * The memory K/V projection is four fifths of the head's time (clef_head.h).  Its rows and
 * weights can be kept in 4 bits with a scale for every few values, which the tensor cores
 * multiply at several times their bf16 rate and which take a quarter of the memory: rows
 * quantised (with the statistics that the memory LayerNorm needs, in the same pass), read
 * back, multiplied with the LayerNorm folded in, and the head's streamed rows over them
 * (clef_stream_rows_fp4).
 *
 * A row of `cols` values is cut into blocks (the last may be short).  A value is an e2m1
 * number (0, 0.5, 1, 1.5, 2, 3, 4, 6, signed) times its block's scale, nearest, ties to the
 * even code; the decisions are exact, so equal values give equal codes on any path.
 *   CLEF_MXFP4  blocks of 32, scale 2^(floor(log2 amax) - 2), not below 2^-127 (e8m0);
 *               quotients above 6 become 6
 *   CLEF_NVFP4  blocks of 16, scale r * e4m3(amax / (6 r)), where r = 2^(floor(log2 a) - 10),
 *               not below 2^-126, a the row's largest finite size: a row stands by itself,
 *               whatever other rows hold
 * An nvfp4 scale may round up, so that a row's largest value stands for up to 18 / 17 of itself: finite values that
 * close to a type's largest (65504 in fp16 stands for 67584) read back as infinity in that type.  The largest
 * number of an mxfp4 block is 1.5 times the power of two at or below its largest size, which every type holds.
 * A block that holds an infinity or a NaN reads as NaN, and so does every product of its row;
 * other rows and blocks are as without it.
 *
 * Layout.  codes: row-major, ceil(cols / 32) * 16 bytes a row; byte j holds value 2j in its
 * low four bits and 2j + 1 in the high ones (bit 3 the sign); values behind `cols` are 0.
 * scales: one byte a block, rows in groups of 128 and blocks in groups of 4; a group of both
 * is 512 contiguous bytes (byte (row % 32) * 16 + row % 128 / 32 * 4 + block % 4), the groups
 * of 128 rows lie one after the other with cols rounded up to 256; blocks behind `cols` are 0.
 * row_scale: r of every row (fp32; unused for CLEF_MXFP4).
 *
 * Conventions are those of clef_head.h: caller-owned device memory, host-side validation
 * before any launch, a clef_status from every entry point, all work asynchronous on
 * `stream` of the current device, nothing allocated, every call capturable into a CUDA
 * graph.  `flags` is a device int32 that the caller clears; kernels only set bits in it
 * (clef_cache_status reads and clears it).  Every wait of the products is bounded: where one
 * ran out it reports CLEF_ERR_DEVICE_TIMEOUT, and the outputs since it was last read are not to be used.
 */
#ifndef CLEF_FP4_H
#define CLEF_FP4_H

#include "clef_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum clef_fp4_format { CLEF_MXFP4 = 0, CLEF_NVFP4 = 1 } clef_fp4_format;

#define CLEF_FP4_MAX_COLS 16384

/* A matrix of rows kept in 4 bits.  codes and scales: 256-byte aligned device memory of the
 * sizes that clef_fp4_size gives; row_scale: [rows] fp32, NULL for CLEF_MXFP4.
 * 1 <= rows < 2^31 - 256, 1 <= cols <= CLEF_FP4_MAX_COLS. */
typedef struct clef_fp4 {
    void* codes;
    void* scales;
    float* row_scale;
    int32_t rows;
    int32_t cols;
    int32_t format;
} clef_fp4;

/* Bytes of codes and scales of a rows x cols matrix. */
CLEF_API int clef_fp4_size(int32_t format, int32_t rows, int32_t cols, size_t* codes_bytes, size_t* scales_bytes);

/* Rows x (dtype bf16, fp16 or fp32, `row_stride` elements apart, the values of a row
 * contiguous) into q.  Optional outputs ([rows] fp32, NULL: not wanted): mean and rstd, the
 * row's mean and 1 / sqrt(variance + 1e-5) of x itself; sums, the sum of what the row
 * stands for once kept.  They are fp32 sums: a row whose values add up past fp32's range has an infinite
 * mean, and one whose squared distances from the mean do by far (a spread of about 2^96 / sqrt(cols) and more) an rstd of 0. */
CLEF_API int clef_fp4_quantize(const clef_fp4* q, int32_t dtype, const void* x, int64_t row_stride, float* mean,
                               float* rstd, float* sums, void* stream);

/* What the rows of q stand for, rounded once to dtype (bf16, fp16 or fp32), into out. */
CLEF_API int clef_fp4_dequantize(const clef_fp4* q, int32_t dtype, void* out, int64_t row_stride, void* stream);

/* out[m, n] = sum over k of x[m, k] w[n, k] + bias[n], sums in fp32, rounded once to dtype
 * (bf16, fp16 or fp32).  x and w: of one format and one number of columns; bias: [w.rows]
 * fp32 or NULL.  With mean, rstd (of x's rows) and sums (of w's rows) all given, x's rows
 * are taken less their means and times their rstd: rstd[m] (x w^T - mean[m] sums[n]) + bias[n],
 * the layer behind a LayerNorm whose weight w holds already.  Sums meet w's row scale first and x's (and rstd)
 * then, in fp32: rows of w above about 2^90 pass its range on the way, whatever x is.  (Kept rows
 * are raw ones: a row whose mean is large against its spread spends its codes on the mean.)  out's rows are
 * `row_stride` elements apart (at least w.rows) and out lies apart from all inputs. */
CLEF_API int clef_fp4_product(const clef_fp4* x, const clef_fp4* w, const float* bias, const float* mean,
                              const float* rstd, const float* sums, int32_t dtype, void* out, int64_t row_stride,
                              int32_t* flags, void* stream);

/* Bytes of scratch to give clef_fp4_linear for `rows` rows of `cols` values of type x_dtype and `outs` rows of weights,
 * with sums (normalized) or without, whose rows all start on 16 bytes and have a multiple of 8 values (aligned; one
 * row: x does) or not, in a call by itself or in a captured graph (captured), whose launches cost the host nothing.
 * 0: the rows are few and best quantised inside the product, in one launch; give NULL.
 * Without `aligned` the size does for any call of so many rows. */
CLEF_API int clef_fp4_linear_scratch(int32_t format, int32_t x_dtype, int32_t rows, int32_t cols, int32_t outs,
                                     int32_t normalized, int32_t aligned, int32_t captured, size_t* bytes);

/* A layer with 4-bit weights: clef_fp4_quantize of the `rows` rows x in w's format, then clef_fp4_product with
 * w, the same numbers by one call.  With `sums` (of w's rows) the rows are normalized as there, and their
 * mean and rstd ([rows] fp32, both needed then) come back too; without, all three are NULL.
 * scratch: 256-byte aligned device memory of the call's own until it has run; NULL, for few aligned rows alone: one
 * launch, which needs none. */
CLEF_API int clef_fp4_linear(const clef_fp4* w, int32_t x_dtype, const void* x, int64_t x_stride, int32_t rows,
                             const float* bias, const float* sums, int32_t dtype, void* out, int64_t row_stride,
                             float* mean, float* rstd, void* scratch, size_t scratch_bytes, int32_t* flags,
                             void* stream);

/* Self-test of the products' wait limits: clef_fp4_linear without bias and sums whose product never loads the last
 * 256 columns (or fewer, where the row ends), so that the waits for them run out after limit_ns (1 us .. 100 ms)
 * each.  The kernels then report CLEF_ERR_DEVICE_TIMEOUT in `flags` and return; out is left as it was, or in part
 * written, and the context stays usable. */
CLEF_API int clef_fp4_selftest_timeout(const clef_fp4* w, int32_t x_dtype, const void* x, int64_t x_stride, int32_t rows,
                                       int32_t dtype, void* out, int64_t row_stride, void* scratch, size_t scratch_bytes,
                                       int64_t limit_ns, int32_t* flags, void* stream);

/* ---- the head with its memory K/V projection in 4 bits ---- */

/* The K/V weights of every routing layer (with the memory LayerNorm's weight, as clef_prepare_weights left
 * them in `prepared`) into w (2 * n_route * width rows of `hidden` values, of either format), and the sums
 * of w's rows (fp32). */
CLEF_API int clef_fp4_memory_weights(const clef_config* cfg, const void* prepared, const clef_fp4* w, float* sums,
                                     void* stream);

/* Bytes of scratch for n_rows streamed rows, and for a whole forward pass of the schema. */
CLEF_API int clef_stream_rows_fp4_scratch(const clef_config* cfg, int32_t format, int32_t n_rows, size_t* bytes);
CLEF_API int clef_head_forward_fp4_scratch(const clef_config* cfg, int32_t format, const clef_schema* schema,
                                           size_t* bytes);

/* clef_stream_rows with the rows and the weights in 4 bits: `hidden` is bf16 or fp16 (quantised as it is), w and
 * sums come from clef_fp4_memory_weights.  A row's keys and values depend on the row alone, up to the
 * order in which fp32 sums of other numbers of rows a call are added.  Chunks of a schema may mix
 * this call and the others; clef_stream_finish and its kin follow as ever. */
CLEF_API int clef_stream_rows_fp4(const clef_config* cfg, const void* prepared, const clef_fp4* w, const float* sums,
                                  const clef_schema* schema, const void* hidden, int32_t hidden_dtype, int32_t record,
                                  int32_t row0, int32_t n_rows, void* workspace, size_t workspace_bytes, void* scratch,
                                  size_t scratch_bytes, void* stream);

/* The forward pass over such a projection: clef_stream_begin, every record's rows, and the finish in one
 * call.  Records whose rows lie one after the other without a gap, here and in the workspace, are
 * projected together. */
CLEF_API int clef_head_forward_fp4(const clef_config* cfg, const void* const* weights, const void* prepared,
                                   const clef_fp4* w, const float* sums, const clef_schema* schema, const void* hidden,
                                   int32_t hidden_dtype, const int32_t* token_ids, const uint16_t* lexical, float* logits,
                                   float* probs, float* q_value, float* q_conf, int32_t* q_argmax, void* workspace,
                                   size_t workspace_bytes, void* scratch, size_t scratch_bytes,
                                   const clef_debug_outputs* debug, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* CLEF_FP4_H */
