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
bool fp4_few_rows(int format, int x_dtype, int rows, int cols, bool normalized) {
    if (cols % 8 != 0) return false;
    const int64_t bytes = int64_t(cols) * (x_dtype == CLEF_FP32 ? 4 : 2);
    if (format == CLEF_NVFP4 || normalized) return rows <= 8 && bytes <= 12288;
    return (rows <= 8 && bytes <= 32768) || (rows <= kFp4FewRows && bytes <= 8192);
}

// A call by itself is 5 us shorter in one launch (host time: 11 for 16 us, 15 for 20 normalized), so that it wins until
// the GPU has more to do than that: every 128 outputs have the rows quantised once more.  In a graph GPU time decides.
// One launch, two launches (us in a graph, bf16, columns x outputs):
//                  1024 x 4096  2048 x 8192  4096 x 4096  4096 x 16384  4096 x 32768  4096 x 131072
//   mxfp4,  1 row   3.4, 4.3     4.6, 5.8     4.5, 5.5     7.8, 8.6      8.9, 13.3     49.0, 47.7
//           8       3.8, 4.6     5.2, 6.0     4.9, 5.8     8.4, 8.5      9.9, 12.1     49.2, 49.1
//          16       4.3, 4.7     6.2, 6.0     5.6, 6.2    10.1, 8.5     12.4, 10.8     66.5, 49.2
//   nvfp4,  1       4.6, 4.6     5.7, 5.9     6.3, 5.8     9.1, 8.9     10.3, 13.7     52.3, 49.8
//           4       4.5, 4.8     6.1, 6.1     6.6, 5.9    10.0, 8.8     11.2, 13.9     55.2, 51.1
//           8       4.7, 4.8     6.7, 6.1     7.1, 6.0    10.8, 8.8     12.6, 12.4     58.7, 51.2
// mxfp4 with statistics goes as nvfp4 does: 8 rows 4.5, 4.7; 5.9, 5.9; 6.5, 5.8; 9.7, 8.5; 11.6, 12.1; 54.4, 49.1.
bool fp4_few_pays(int format, int x_dtype, int rows, int cols, int outs, bool normalized, bool captured) {
    if (outs > 32768) return false;
    if (!captured) return true;
    const int64_t bytes = int64_t(cols) * (x_dtype == CLEF_FP32 ? 4 : 2);
    if (format == CLEF_MXFP4 && !normalized) return rows * bytes <= 65536;
    // long rows are read through before the first code is made: worth it only where the two launches' tiles, more than
    // one an SM, have more to wait for
    return bytes <= 2048 || (rows <= 4 && outs > 128 * 152);
}

cudaError_t launch_fp4_few(const clef_fp4& w, const Fp4ProductArgs& a, int x_dtype, int dtype, cudaStream_t s) {
    return w.format == CLEF_MXFP4 ? launch_few_of<CLEF_MXFP4>(w, a, x_dtype, dtype, s)
                                  : launch_few_of<CLEF_NVFP4>(w, a, x_dtype, dtype, s);
}

}  // namespace clef
