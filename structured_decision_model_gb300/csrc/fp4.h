// Host-side launchers of the microscaled 4-bit kernels (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/clef_fp4.h"

namespace clef {

constexpr int kFp4Tile = 256;       // columns of one K tile: 128 bytes of codes
constexpr int kFp4RowGroup = 128;   // rows of one group of scales
constexpr int kFp4ScaleGroup = 512; // bytes of 128 rows x 4 scales

inline int fp4_block(int format) { return format == CLEF_MXFP4 ? 32 : 16; }
inline int64_t fp4_code_stride(int cols) { return int64_t(cols + 31) / 32 * 16; }
inline int fp4_ktiles(int cols) { return (cols + kFp4Tile - 1) / kFp4Tile; }
// 512-byte groups of scales of 128 rows: 2 (mxfp4) or 4 (nvfp4) a K tile
inline int fp4_kgroups(int format, int cols) { return fp4_ktiles(cols) * (format == CLEF_MXFP4 ? 2 : 4); }
inline int64_t fp4_row_groups(int64_t rows) { return (rows + kFp4RowGroup - 1) / kFp4RowGroup; }

struct Fp4QuantizeArgs {
    const void* x;
    int64_t row_stride;  // elements
    uint8_t* codes;
    uint8_t* scales;
    float* row_scale;    // NVFP4
    float* mean;         // optional
    float* rstd;         // with mean
    float* sums;         // optional
    int rows, cols;
    float inv_cols;      // 1 / cols
};
cudaError_t launch_fp4_quantize(const Fp4QuantizeArgs& a, int format, int dtype, cudaStream_t s);

struct Fp4DequantizeArgs {
    const uint8_t* codes;
    const uint8_t* scales;
    const float* row_scale;
    void* out;
    int64_t row_stride;
    int rows, cols;
};
cudaError_t launch_fp4_dequantize(const Fp4DequantizeArgs& a, int format, int dtype, cudaStream_t s);

struct Fp4ProductArgs {
    const float* x_scale;  // [M], null: 1
    const float* w_scale;  // [N], null: 1
    const float* bias;     // [N], null: 0
    const float* mean;     // [M], with rstd and sums: the LayerNorm fold
    const float* rstd;     // [M]
    const float* sums;     // [N]
    void* out;
    int64_t ldo;
    int* flags;
    int M, N;              // rows of x and of w
    int k64;               // columns in steps of 64 (one MMA)
    int kgroups;           // scale groups of a row group
    int splits;            // K parts of a tile (a cluster)
    int paired;            // 16-bit outputs: rows and columns allow stores of two values at a time
    const void* x;         // few rows as they come: rows x_stride elements apart, of `cols` values,
    int64_t x_stride;      // their statistics (with sums: the LayerNorm fold) going out
    float* mean_out;
    float* rstd_out;
    int cols;
    float inv_cols;
    int w_settled;         // no kernel that may still run on the stream writes w: it may be read ahead of them
    uint64_t wait_ns;      // limit of a wait
    int withheld;          // 1: the last K tile is never loaded, so that the waits for it run out (the self-test)
    int bulk;              // 16-bit outputs: rows start and end on 16 bytes, so that TMA can store them
};
cudaError_t launch_fp4_product(const clef_fp4& x, const clef_fp4& w, const Fp4ProductArgs& a, int dtype,
                               cudaStream_t s);


// Rows that the product quantises itself, in one launch: whether it can, whether that pays, and the launch (a.M rows
// of type x_dtype that start on 16 bytes, cols a multiple of 8).
constexpr int kFp4FewRows = 16;
bool fp4_few_rows(int format, int x_dtype, int rows, int cols, bool normalized);
bool fp4_few_pays(int format, int x_dtype, int rows, int cols, int outs, bool normalized, bool captured);
cudaError_t launch_fp4_few(const clef_fp4& w, const Fp4ProductArgs& a, int x_dtype, int dtype, cudaStream_t s);

// clef_fp4_linear; only the checks of its arguments; or with a product whose last K tile is withheld and whose waits end
// after starve_ns.
enum Fp4Call { kFp4Check, kFp4Run, kFp4Starve };
int fp4_linear(Fp4Call call, uint64_t starve_ns, const clef_fp4* w, int32_t x_dtype, const void* x, int64_t x_stride, int32_t rows,
               const float* bias, const float* sums, int32_t dtype, void* out, int64_t row_stride, float* mean, float* rstd,
               void* scratch, size_t scratch_bytes, int32_t* flags, void* stream);

}  // namespace clef
