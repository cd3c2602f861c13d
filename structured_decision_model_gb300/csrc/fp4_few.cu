// A layer of 4-bit weights on few rows that are not quantised yet: the tile kernel quantises them itself.
#include "fp4_tile.cuh"

namespace clef {

namespace {

template <int FMT, int DT>
cudaError_t launch_few(const clef_fp4& w, const Fp4ProductArgs& a, int dtype, cudaStream_t s) {
    if (dtype == CLEF_BF16) return launch_tile<FMT, 32, CLEF_BF16, DT>(nullptr, w, a, s);
    if (dtype == CLEF_FP16) return launch_tile<FMT, 32, CLEF_FP16, DT>(nullptr, w, a, s);
    return launch_tile<FMT, 32, CLEF_FP32, DT>(nullptr, w, a, s);
}

template <int FMT>
cudaError_t launch_few_of(const clef_fp4& w, const Fp4ProductArgs& a, int x_dtype, int dtype, cudaStream_t s) {
    if (x_dtype == CLEF_BF16) return launch_few<FMT, CLEF_BF16>(w, a, dtype, s);
    if (x_dtype == CLEF_FP16) return launch_few<FMT, CLEF_FP16>(w, a, dtype, s);
    return launch_few<FMT, CLEF_FP32>(w, a, dtype, s);
}

}  // namespace

// Every CTA reads its K range of the rows itself and, for row scales or statistics, all of them, a row a warp at a time.
// GPU time against the two launches' (graph, bf16; a call by itself is 5 us shorter in one launch):
//   4096 x 4096 mxfp4: 1 row 4.7, 5.4 us; 8: 5.2, 5.9; 16: 5.9, 6.3; 32: 7.6, 6.9     16384 columns, 8 rows: 9.6, 9.8; 16: 11.6, 10.1
//   4096 x 4096 nvfp4: 1 row 6.6, 5.8 us; 8: 7.2, 5.9; 16: 9.3, 6.2                   16384 columns, 1 row: 13.2, 10.3
bool fp4_few_rows(int format, int x_dtype, int rows, int cols, bool normalized) {
    const int64_t bytes = int64_t(cols) * (x_dtype == CLEF_FP32 ? 4 : 2);
    if (format == CLEF_NVFP4 || normalized) return rows <= 8 && bytes <= 12288;
    return (rows <= 8 && bytes <= 32768) || (rows <= kFp4FewRows && bytes <= 8192);
}

cudaError_t launch_fp4_few(const clef_fp4& w, const Fp4ProductArgs& a, int x_dtype, int dtype, cudaStream_t s) {
    return w.format == CLEF_MXFP4 ? launch_few_of<CLEF_MXFP4>(w, a, x_dtype, dtype, s)
                                  : launch_few_of<CLEF_NVFP4>(w, a, x_dtype, dtype, s);
}

}  // namespace clef
