// C ABI of the microscaled 4-bit operators: argument checks and launches.
#include <initializer_list>

#include "common.cuh"
#include "fp4.h"

using namespace clef;

namespace {

constexpr int64_t kInt32 = int64_t(1) << 31;

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

bool bad_type(int dtype) { return dtype != CLEF_BF16 && dtype != CLEF_FP16 && dtype != CLEF_FP32; }

int64_t size_of(int dtype) { return dtype == CLEF_FP32 ? 4 : 2; }

// A run of bytes that a call reads or writes (empty where the pointer is null).
struct Run {
    uintptr_t at;
    uint64_t n;
    Run(const void* p, int64_t bytes) : at(reinterpret_cast<uintptr_t>(p)), n(p && bytes > 0 ? uint64_t(bytes) : 0) {}
    bool meets(const Run& o) const { return n && o.n && (at <= o.at ? o.at - at < n : at - o.at < o.n); }
};

// From the first value to the last of rows `stride` elements apart.
Run rows_run(const void* p, int64_t rows, int64_t stride, int64_t cols, int64_t size) {
    return Run(p, ((rows - 1) * stride + cols) * size);
}

int check_size(int32_t format, int32_t rows, int32_t cols) {
    if (format != CLEF_MXFP4 && format != CLEF_NVFP4) return CLEF_ERR_UNSUPPORTED_CONFIG;
    if (rows < 1 || rows >= kInt32 - 256 || cols < 1 || cols > CLEF_FP4_MAX_COLS) return CLEF_ERR_UNSUPPORTED_CONFIG;
    // scale groups are counted in 32 bits
    if (fp4_row_groups(rows) * fp4_kgroups(format, cols) >= kInt32) return CLEF_ERR_UNSUPPORTED_CONFIG;
    return CLEF_OK;
}

int64_t codes_bytes(const clef_fp4& q) { return q.rows * fp4_code_stride(q.cols); }
int64_t scales_bytes(const clef_fp4& q) {
    return fp4_row_groups(q.rows) * fp4_kgroups(q.format, q.cols) * kFp4ScaleGroup;
}

int check_matrix(const clef_fp4* q) {
    if (!q) return CLEF_ERR_INVALID_ARGUMENT;
    const int st = check_size(q->format, q->rows, q->cols);
    if (st != CLEF_OK) return st;
    if (!q->codes || !q->scales || misaligned(q->codes, 256) || misaligned(q->scales, 256) ||
        misaligned(q->row_scale, 4) || (q->format == CLEF_NVFP4 && !q->row_scale))
        return CLEF_ERR_INVALID_ARGUMENT;
    return CLEF_OK;
}

Run codes_run(const clef_fp4& q) { return Run(q.codes, codes_bytes(q)); }
Run scales_run(const clef_fp4& q) { return Run(q.scales, scales_bytes(q)); }
Run row_scale_run(const clef_fp4& q) { return Run(q.format == CLEF_NVFP4 ? q.row_scale : nullptr, int64_t(q.rows) * 4); }

// `rows` rows `stride` elements apart: aligned to the element, at least `least` apart, and no further from first to
// last than memory reaches.
bool bad_rows(const void* p, int dtype, int64_t rows, int64_t stride, int64_t least) {
    return !p || misaligned(p, uintptr_t(size_of(dtype))) || stride < least || stride > kInt32 ||
           (rows - 1) * stride > (int64_t(1) << 40);
}

int check_product(const clef_fp4& x, const clef_fp4& w, const float* bias, const float* mean, const float* rstd,
                  const float* sums, int dtype, const void* out, int64_t row_stride, const int32_t* flags) {
    // output tiles are counted in 32 bits
    if ((int64_t(x.rows) + 31) / 32 * ((int64_t(w.rows) + 127) / 128) >= kInt32 / 16) return CLEF_ERR_UNSUPPORTED_CONFIG;
    if (x.format != w.format || x.cols != w.cols || bad_type(dtype) || bad_rows(out, dtype, x.rows, row_stride, w.rows) ||
        !mean != !rstd || !mean != !sums || !flags)
        return CLEF_ERR_INVALID_ARGUMENT;
    for (const void* p : {static_cast<const void*>(bias), static_cast<const void*>(mean), static_cast<const void*>(rstd),
                          static_cast<const void*>(sums), static_cast<const void*>(flags)})
        if (misaligned(p, 4)) return CLEF_ERR_INVALID_ARGUMENT;
    const int64_t m4 = int64_t(x.rows) * 4, n4 = int64_t(w.rows) * 4;
    const Run to = rows_run(out, x.rows, row_stride, w.rows, size_of(dtype));
    for (const Run& r : {codes_run(x), scales_run(x), row_scale_run(x), codes_run(w), scales_run(w), row_scale_run(w),
                         Run(bias, n4), Run(mean, m4), Run(rstd, m4), Run(sums, n4), Run(flags, 4)})
        if (to.meets(r)) return CLEF_ERR_INVALID_ARGUMENT;
    return CLEF_OK;
}

// The arguments of a checked product.  `w_settled`: nothing that may still run on the stream writes w.
Fp4ProductArgs product_args(const clef_fp4& x, const clef_fp4& w, const float* bias, const float* mean, const float* rstd,
                            const float* sums, int dtype, void* out, int64_t row_stride, int32_t* flags, bool w_settled) {
    Fp4ProductArgs a{};
    a.x_scale = x.format == CLEF_NVFP4 ? x.row_scale : nullptr;
    a.w_scale = w.format == CLEF_NVFP4 ? w.row_scale : nullptr;
    a.bias = bias;
    a.mean = mean;
    a.rstd = rstd;
    a.sums = sums;
    a.out = out;
    a.ldo = row_stride;
    a.flags = flags;
    a.M = x.rows;
    a.N = w.rows;
    a.k64 = (x.cols + 63) / 64;
    a.kgroups = fp4_kgroups(x.format, x.cols);
    a.splits = 1;
    a.paired = dtype != CLEF_FP32 && row_stride % 2 == 0 && w.rows % 2 == 0 && !misaligned(out, 4);
    // TMA writes whole 16-byte pieces of a row, also where the row ends inside one
    a.bulk = dtype != CLEF_FP32 && row_stride % 8 == 0 && w.rows % 8 == 0 && !misaligned(out, 16);
    a.wait_ns = kWaitLimitNs;
    a.w_settled = w_settled;
    a.cols = x.cols;
    a.inv_cols = 1.f / float(x.cols);
    return a;
}

int status(cudaError_t e) { return e == cudaSuccess ? CLEF_OK : CLEF_ERR_CUDA; }

// Where the rows of a layer's call lie in its scratch.
struct Scratch {
    size_t scales, row_scale, total;
    Scratch(int format, int rows, int cols) {
        const clef_fp4 q{nullptr, nullptr, nullptr, rows, cols, format};
        scales = (size_t(codes_bytes(q)) + 255) / 256 * 256;
        row_scale = scales + (size_t(scales_bytes(q)) + 255) / 256 * 256;
        total = row_scale + (format == CLEF_NVFP4 ? size_t(rows) * 4 : 0);
    }
    clef_fp4 matrix(void* base, int format, int rows, int cols) const {
        uint8_t* b = static_cast<uint8_t*>(base);
        return clef_fp4{b, b + scales, format == CLEF_NVFP4 ? reinterpret_cast<float*>(b + row_scale) : nullptr, rows, cols,
                        format};
    }
};

}  // namespace

namespace clef {

int fp4_linear(Fp4Call call, uint64_t starve_ns, const clef_fp4* w, int32_t x_dtype, const void* x, int64_t x_stride, int32_t rows,
               const float* bias, const float* sums, int32_t dtype, void* out, int64_t row_stride, float* mean, float* rstd,
               void* scratch, size_t scratch_bytes, int32_t* flags, void* stream) {
    int st = check_matrix(w);
    if (st == CLEF_OK) st = check_size(w->format, rows, w->cols);
    if (st != CLEF_OK) return st;
    if (bad_type(x_dtype) || bad_rows(x, x_dtype, rows, x_stride, 0)) return CLEF_ERR_INVALID_ARGUMENT;
    const bool aligned = !misaligned(x, 16) && (rows == 1 || x_stride * size_of(x_dtype) % 16 == 0);
    const bool few = !scratch && aligned && fp4_few_rows(w->format, x_dtype, rows, w->cols, sums != nullptr);
    const Scratch S(w->format, rows, w->cols);
    clef_fp4 q{nullptr, nullptr, nullptr, rows, w->cols, w->format};
    if (!few) {
        if (!scratch || misaligned(scratch, 256)) return CLEF_ERR_INVALID_ARGUMENT;
        if (scratch_bytes < S.total) return CLEF_ERR_WORKSPACE_TOO_SMALL;
        q = S.matrix(scratch, w->format, rows, w->cols);
    }
    st = check_product(q, *w, bias, mean, rstd, sums, dtype, out, row_stride, flags);
    if (st != CLEF_OK) return st;
    // what is written: the scratch, the statistics and the output, apart from each other and from what is read
    const int64_t m4 = int64_t(rows) * 4, n4 = int64_t(w->rows) * 4;
    const Run space(few ? nullptr : scratch, int64_t(S.total)), in = rows_run(x, rows, x_stride, w->cols, size_of(x_dtype)),
        to = rows_run(out, rows, row_stride, w->rows, size_of(dtype));
    const Run reads[] = {in, codes_run(*w), scales_run(*w), row_scale_run(*w), Run(bias, n4), Run(sums, n4), Run(flags, 4)};
    for (const Run& r : reads)
        if (r.meets(space) || r.meets(Run(mean, m4)) || r.meets(Run(rstd, m4))) return CLEF_ERR_INVALID_ARGUMENT;
    if (to.meets(in) || to.meets(space) || space.meets(Run(mean, m4)) || space.meets(Run(rstd, m4)) ||
        Run(mean, m4).meets(Run(rstd, m4)))
        return CLEF_ERR_INVALID_ARGUMENT;
    if (call == kFp4Check) return CLEF_OK;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    Fp4ProductArgs p = product_args(q, *w, bias, mean, rstd, sums, dtype, out, row_stride, flags, true);
    if (call == kFp4Starve) {
        p.wait_ns = starve_ns;
        p.withheld = 1;
    }
    if (few) {  // one launch
        p.x = x;
        p.x_stride = x_stride;
        p.x_scale = p.mean = p.rstd = nullptr;
        p.mean_out = mean;
        p.rstd_out = rstd;
        p.w_settled = false;  // the kernel before this one may be w's
        return status(launch_fp4_few(*w, p, x_dtype, dtype, s));
    }
    const Fp4QuantizeArgs a{x, x_stride, static_cast<uint8_t*>(q.codes), static_cast<uint8_t*>(q.scales), q.row_scale,
                            mean, rstd, nullptr, rows, w->cols, 1.f / float(w->cols)};
    const int quantised = status(launch_fp4_quantize(a, w->format, x_dtype, s));
    return quantised == CLEF_OK ? status(launch_fp4_product(q, *w, p, dtype, s)) : quantised;
}

}  // namespace clef

extern "C" {

int clef_fp4_size(int32_t format, int32_t rows, int32_t cols, size_t* codes, size_t* scales) {
    if (!codes || !scales) return CLEF_ERR_INVALID_ARGUMENT;
    const int st = check_size(format, rows, cols);
    if (st != CLEF_OK) return st;
    const clef_fp4 q{nullptr, nullptr, nullptr, rows, cols, format};
    *codes = size_t(codes_bytes(q));
    *scales = size_t(scales_bytes(q));
    return CLEF_OK;
}

int clef_fp4_quantize(const clef_fp4* q, int32_t dtype, const void* x, int64_t row_stride, float* mean, float* rstd,
                      float* sums, void* stream) {
    const int st = check_matrix(q);
    if (st != CLEF_OK) return st;
    if (bad_type(dtype) || bad_rows(x, dtype, q->rows, row_stride, 0) || !mean != !rstd || misaligned(mean, 4) ||
        misaligned(rstd, 4) || misaligned(sums, 4))
        return CLEF_ERR_INVALID_ARGUMENT;
    const int64_t each = int64_t(q->rows) * 4;
    const Run out[] = {codes_run(*q), scales_run(*q), row_scale_run(*q), Run(mean, each), Run(rstd, each), Run(sums, each)};
    const Run in = rows_run(x, q->rows, row_stride, q->cols, size_of(dtype));
    for (int i = 0; i < 6; ++i) {
        if (out[i].meets(in)) return CLEF_ERR_INVALID_ARGUMENT;
        for (int j = 0; j < i; ++j)
            if (out[i].meets(out[j])) return CLEF_ERR_INVALID_ARGUMENT;
    }
    const Fp4QuantizeArgs a{x, row_stride, static_cast<uint8_t*>(q->codes), static_cast<uint8_t*>(q->scales),
                            q->row_scale, mean, rstd, sums, q->rows, q->cols, 1.f / float(q->cols)};
    return status(launch_fp4_quantize(a, q->format, dtype, static_cast<cudaStream_t>(stream)));
}

int clef_fp4_dequantize(const clef_fp4* q, int32_t dtype, void* out, int64_t row_stride, void* stream) {
    const int st = check_matrix(q);
    if (st != CLEF_OK) return st;
    if (bad_type(dtype) || bad_rows(out, dtype, q->rows, row_stride, q->cols)) return CLEF_ERR_INVALID_ARGUMENT;
    const Run to = rows_run(out, q->rows, row_stride, q->cols, size_of(dtype));
    if (to.meets(codes_run(*q)) || to.meets(scales_run(*q)) || to.meets(row_scale_run(*q)))
        return CLEF_ERR_INVALID_ARGUMENT;
    const Fp4DequantizeArgs a{static_cast<const uint8_t*>(q->codes), static_cast<const uint8_t*>(q->scales),
                              q->row_scale, out, row_stride, q->rows, q->cols};
    return status(launch_fp4_dequantize(a, q->format, dtype, static_cast<cudaStream_t>(stream)));
}

int clef_fp4_product(const clef_fp4* x, const clef_fp4* w, const float* bias, const float* mean, const float* rstd,
                     const float* sums, int32_t dtype, void* out, int64_t row_stride, int32_t* flags, void* stream) {
    int st = check_matrix(x);
    if (st == CLEF_OK) st = check_matrix(w);
    if (st == CLEF_OK) st = check_product(*x, *w, bias, mean, rstd, sums, dtype, out, row_stride, flags);
    if (st != CLEF_OK) return st;
    return status(launch_fp4_product(*x, *w, product_args(*x, *w, bias, mean, rstd, sums, dtype, out, row_stride, flags, false),
                                     dtype, static_cast<cudaStream_t>(stream)));
}

int clef_fp4_linear_scratch(int32_t format, int32_t x_dtype, int32_t rows, int32_t cols, int32_t outs, int32_t normalized,
                            int32_t aligned, int32_t captured, size_t* bytes) {
    if (!bytes || bad_type(x_dtype) || outs < 1) return CLEF_ERR_INVALID_ARGUMENT;
    const int st = check_size(format, rows, cols);
    if (st != CLEF_OK) return st;
    const bool few = aligned && fp4_few_rows(format, x_dtype, rows, cols, normalized != 0) &&
                     fp4_few_pays(format, x_dtype, rows, cols, outs, normalized != 0, captured != 0);
    *bytes = few ? 0 : Scratch(format, rows, cols).total;
    return CLEF_OK;
}

int clef_fp4_linear(const clef_fp4* w, int32_t x_dtype, const void* x, int64_t x_stride, int32_t rows, const float* bias,
                    const float* sums, int32_t dtype, void* out, int64_t row_stride, float* mean, float* rstd,
                    void* scratch, size_t scratch_bytes, int32_t* flags, void* stream) {
    return fp4_linear(kFp4Run, 0, w, x_dtype, x, x_stride, rows, bias, sums, dtype, out, row_stride, mean, rstd, scratch,
                      scratch_bytes, flags, stream);
}

int clef_fp4_selftest_timeout(const clef_fp4* w, int32_t x_dtype, const void* x, int64_t x_stride, int32_t rows,
                              int32_t dtype, void* out, int64_t row_stride, void* scratch, size_t scratch_bytes,
                              int64_t limit_ns, int32_t* flags, void* stream) {
    if (limit_ns < 1000 || limit_ns > 100000000) return CLEF_ERR_INVALID_ARGUMENT;
    return fp4_linear(kFp4Starve, uint64_t(limit_ns), w, x_dtype, x, x_stride, rows, nullptr, nullptr, dtype, out, row_stride,
                      nullptr, nullptr, scratch, scratch_bytes, flags, stream);
}

}  // extern "C"
