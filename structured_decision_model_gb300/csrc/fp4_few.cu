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

bool fp4_few_rows(int rows, int cols, int x_dtype, const void* x, int64_t x_stride) {
    const int64_t size = x_dtype == CLEF_FP32 ? 4 : 2;
    return rows <= kFewRows && cols % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
           (rows == 1 || x_stride * size % 16 == 0);
}

cudaError_t launch_fp4_few(const clef_fp4& w, const Fp4ProductArgs& a, int x_dtype, int dtype, cudaStream_t s) {
    return w.format == CLEF_MXFP4 ? launch_few_of<CLEF_MXFP4>(w, a, x_dtype, dtype, s)
                                  : launch_few_of<CLEF_NVFP4>(w, a, x_dtype, dtype, s);
}

}  // namespace clef
