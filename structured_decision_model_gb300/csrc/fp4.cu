// Rows into microscaled 4-bit form and back.
//
// Quantise.  A row belongs to one or more whole warps and stays in their registers: its
// largest sizes, its mean and variance (two passes over registers, so exact to fp32
// rounding) and its codes come from one read of memory.  A lane holds 8 consecutive values of
// every 256-value tile (one 16-byte read, one 4-byte write: both whole lines a warp), so a
// block of 16 or 32 values is 2 or 4 neighbouring lanes.
//
// Exact decisions.  A code is right when the quotient x / scale falls on the right side of
// the midpoints of e2m1 (multiples of 1/4 up to 5), ties included.  The quotient by a
// rounded reciprocal is off by 2^-23 of itself; adding and taking off 384 rounds it to a
// multiple of 2^-15.  For bf16 and fp16 values a quotient that is no midpoint is at least
// 2^-13 away from one (the value has 11 bits, the midpoint times the scale at most 7), so
// the rounded quotient is on the true side, and a midpoint comes out as itself.  An fp32
// value may lie closer: what it has left over, x - q * scale, is exact in one fused
// multiply-add, and its sign moves the quotient off the midpoint to the true side.
#include "common.cuh"
#include "fp4.h"
#include "kernels.h"

namespace clef {

namespace {

constexpr int kThreads = 256;
constexpr float kGrid = 384.f;                 // fp32 numbers in [256, 512) are multiples of 2^-15
constexpr float kAside = 7.62939453125e-06f;   // 2^-17: less than the grid's step

__device__ __forceinline__ float pow2(int e) {  // e in [-126, 127]
    return __int_as_float((e + 127) << 23);
}

// Exponent of the power of two at or below x >= 0, -127 for zero and subnormal numbers.
__device__ __forceinline__ int exponent_of(float x) { return int(__float_as_uint(x) >> 23) - 127; }

// Eight codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t pack_e2m1(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Eight codes to their numbers, as four fp16 pairs.
__device__ __forceinline__ void unpack_e2m1(uint32_t codes, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
}

__device__ __forceinline__ uint32_t to_e4m3(float x) {  // x >= 0, in the low byte
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return r & 0xFFu;
}

__device__ __forceinline__ float from_e4m3(uint32_t b) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(b)));
    return __half2float(__ushort_as_half(uint16_t(h & 0xFFFFu)));
}

// t / 6 so that rounding it to few bits gives what rounding the true quotient gives: cut off,
// with the last bit set where something was cut (a number next to a border stays off it).
__device__ __forceinline__ float sixth(float t) {
    const float q = __fdiv_rz(t, 6.f);
    return fmaf(-q, 6.f, t) != 0.f ? __uint_as_float(__float_as_uint(q) | 1u) : q;
}

// The eight values of a lane as they lie in memory: 4 words of two, or 8 fp32.
template <int DT>
struct Raw {
    uint32_t w[DT == CLEF_FP32 ? 8 : 4];
    __device__ __forceinline__ float at(int j) const {
        if constexpr (DT == CLEF_FP32) return __uint_as_float(w[j]);
        else if constexpr (DT == CLEF_BF16) return j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
        else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j >> 1]));
            return j & 1 ? f.y : f.x;
        }
    }
    // the largest size; NaN if one is NaN
    __device__ __forceinline__ float top() const {
        if constexpr (DT == CLEF_FP32) {
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = fabsf(__uint_as_float(w[j]));
                m = v > m || v != v ? v : m;  // once NaN, `v > m` stays false: kept below
                if (m != m) return m;
            }
            return m;
        } else {
            // sizes of 16-bit floats order as their bits do, NaN above all
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
            const uint32_t t = max(m & 0xFFFFu, m >> 16);
            if constexpr (DT == CLEF_BF16) return __uint_as_float(t << 16);
            else return __half2float(__ushort_as_half(uint16_t(t)));
        }
    }
};

// VEC: every row starts on 16 bytes and has a multiple of 8 values, so a lane's eight are
// read as whole 16-byte pieces; otherwise value by value.
template <int DT, bool VEC>
__device__ __forceinline__ Raw<DT> load8(const void* x, int64_t row0, int col, int cols) {
    Raw<DT> r;
    constexpr int kWords = DT == CLEF_FP32 ? 8 : 4;
    if constexpr (VEC) {
        if (col < cols) {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x) +
                                                            (row0 + col) * (DT == CLEF_FP32 ? 4 : 2));
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 v = p[i];
                r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) r.w[i] = 0;
        }
    } else if constexpr (DT == CLEF_FP32) {
        const uint32_t* p = static_cast<const uint32_t*>(x) + row0;
#pragma unroll
        for (int j = 0; j < 8; ++j) r.w[j] = col + j < cols ? p[col + j] : 0u;
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(x) + row0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = col + 2 * j < cols ? p[col + 2 * j] : 0u;
            const uint32_t hi = col + 2 * j + 1 < cols ? p[col + 2 * j + 1] : 0u;
            r.w[j] = lo | hi << 16;
        }
    }
    return r;
}

// Sums (or maxima) of a row that W warps share, in one order whatever else the block does.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* red, int W, int warp) {
    v = MAX ? warp_max(v) : warp_sum(v);
    if (W == 1) return v;
    __syncthreads();  // red may still be read from the last call
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    const int w0 = warp / W * W;
    v = red[w0];
    for (int i = 1; i < W; ++i) v = MAX ? fmaxf(v, red[w0 + i]) : v + red[w0 + i];
    return v;
}

// TILES: 256-value tiles that a lane keeps 8 values of; W warps a row (a power of two), so
// a row has at most 256 * TILES * W values.
template <int FMT, int DT, bool VEC, int TILES>
__global__ void __launch_bounds__(kThreads) fp4_quantize_kernel(const Fp4QuantizeArgs a, int W) {
    constexpr bool NV = FMT == CLEF_NVFP4;
    __shared__ float red[kThreads / 32];
    griddep_wait();
    griddep_launch();  // behind the wait: whoever starts early may take what came before us as done
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = int64_t(blockIdx.x) * (kThreads / 32 / W) + warp / W;
    const bool mine = row < a.rows;  // warps behind the last row still meet the barriers
    const int part = warp % W;
    const int ktiles = (a.cols + kFp4Tile - 1) / kFp4Tile;
    const int64_t row0 = row * a.row_stride;

    Raw<DT> raw[TILES];
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
        const int col = ((i * W + part) * 32 + lane) * 8;
        if (mine) raw[i] = load8<DT, VEC>(a.x, row0, col, a.cols);
        else raw[i] = Raw<DT>{};
    }
    // the largest size of every block, and of the row's finite blocks
    float top[TILES], row_top = 0.f;
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
        // bits of sizes order as the sizes do, with infinity and NaN above every number
        uint32_t t = __float_as_uint(raw[i].top());
        t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
        if (!NV) t = max(t, __shfl_xor_sync(0xffffffffu, t, 2));
        top[i] = __uint_as_float(t);
    }
    float inv_r = 1.f, r = 1.f;
    bool tiny = false;
    if constexpr (NV) {
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            if (top[i] < INFINITY) row_top = fmaxf(row_top, top[i]);
            else {  // the largest finite size of a block that is not finite
                const int col = ((i * W + part) * 32 + lane) * 8;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v = fabsf(raw[i].at(j));
                    if (col + j < a.cols && v < INFINITY) row_top = fmaxf(row_top, v);
                }
            }
        }
        row_top = row_reduce<true>(row_top, red, W, warp);
        const int e = max(exponent_of(row_top) - 10, -126);
        r = pow2(e);
        inv_r = pow2(-e);
        tiny = e < -100;  // 1 / (block scale * r) may pass fp32's range: divide in two steps
        if (mine && part == 0 && lane == 0) a.row_scale[row] = r;
    }
    if (a.mean) {  // the same for every thread
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            float t = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) t += raw[i].at(j);
            s += t;
        }
        const float mean = row_reduce<false>(s, red, W, warp) / float(a.cols);
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            const int col = ((i * W + part) * 32 + lane) * 8;
            float t = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = col + j < a.cols ? raw[i].at(j) - mean : 0.f;
                t = fmaf(d, d, t);
            }
            q += t;
        }
        const float var = row_reduce<false>(q, red, W, warp) / float(a.cols);
        if (mine && part == 0 && lane == 0) {
            a.mean[row] = mean;
            a.rstd[row] = 1.f / sqrtf(var + 1e-5f);
        }
    }
    const int64_t code_stride = int64_t(a.cols + 31) / 32 * 16;
    uint8_t* codes = a.codes + row * code_stride;
    const int kgroups = ktiles * (NV ? 4 : 2);
    uint8_t* scales = a.scales + (row / kFp4RowGroup * kgroups) * kFp4ScaleGroup +
                      (row % 32) * 16 + (row % kFp4RowGroup) / 32 * 4;
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
        const int tile = i * W + part;
        if (tile >= ktiles || !mine) continue;  // the same for a whole warp
        const int chunk = tile * 32 + lane;
        uint32_t byte;    // the block's scale as stored
        float scale, inv; // what it stands for (without r) and its reciprocal
        const bool bad = !(top[i] < INFINITY);
        if constexpr (NV) {
            byte = bad ? 0x7Fu : to_e4m3(sixth(top[i] * inv_r));
            scale = from_e4m3(byte);
            inv = byte == 0 ? 0.f : __frcp_rn(scale);
        } else {
            const int e = max(exponent_of(top[i]) - 2, -127);
            byte = bad ? 0xFFu : uint32_t(e + 127);
            scale = __uint_as_float(e == -127 ? 0x00400000u : uint32_t(e + 127) << 23);
            inv = pow2(-e);
        }
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = raw[i].at(j);
        if constexpr (DT == CLEF_FP32) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = NV ? v[j] * inv_r : v[j] * inv;  // powers of two
                const float q = (NV ? fmaf(x, inv, kGrid) : x + kGrid) - kGrid;
                const float rest = NV ? fmaf(-q, scale, x) : x - q;
                v[j] = inv == 0.f ? 0.f : q + (rest > 0.f ? kAside : rest < 0.f ? -kAside : 0.f);
            }
        } else {
            float by = inv;
            if constexpr (NV) {
                if (tiny) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] *= inv_r;
                } else {
                    by *= inv_r;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = fmaf(v[j], by, kGrid) - kGrid;
        }
        uint32_t packed = pack_e2m1(v);
        if (bad) {  // any number: the scale makes it NaN; behind the row's end zeros as ever
            const int left = a.cols - chunk * 8;
            packed = left >= 8 ? 0x22222222u : left > 0 ? 0x22222222u >> (32 - 4 * left) : 0u;
        }
        if (chunk * 4 < code_stride) *reinterpret_cast<uint32_t*>(codes + chunk * 4) = packed;
        // four blocks' scales are one word, written by the first lane of theirs
        uint32_t word = byte << (8 * (NV ? lane >> 1 & 3 : lane >> 2 & 3));
        if constexpr (NV) {
            word |= __shfl_xor_sync(0xffffffffu, word, 2);
            word |= __shfl_xor_sync(0xffffffffu, word, 4);
            if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(scales + int64_t(chunk >> 3) * kFp4ScaleGroup) = word;
        } else {
            word |= __shfl_xor_sync(0xffffffffu, word, 4);
            word |= __shfl_xor_sync(0xffffffffu, word, 8);
            if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(scales + int64_t(chunk >> 4) * kFp4ScaleGroup) = word;
        }
        if (a.sums) {
            uint32_t h[4];
            unpack_e2m1(packed, h);
            float t = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
                t += f.x + f.y;
            }
            total = fmaf(t, bad ? __uint_as_float(0x7FC00000u) : scale, total);
        }
    }
    if (a.sums) {
        total = row_reduce<false>(total, red, W, warp);
        if (mine && part == 0 && lane == 0) a.sums[row] = total * r;
    }
}

template <int DT>
__device__ __forceinline__ void store8(void* out, int64_t at, const float (&v)[8], int n, bool vec) {
    if constexpr (DT == CLEF_FP32) {
        float* p = static_cast<float*>(out) + at;
        if (vec) {
            reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) p[j] = v[j];
        }
    } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (DT == CLEF_BF16) w[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
            else {
                const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        uint16_t* p = static_cast<uint16_t*>(out) + at;
        if (vec) {
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) p[j] = uint16_t(w[j >> 1] >> (16 * (j & 1)));
        }
    }
}

// Read back: a thread takes 8 values (4 bytes of codes, one scale).
template <int FMT, int DT>
__global__ void __launch_bounds__(kThreads) fp4_dequantize_kernel(const Fp4DequantizeArgs a, int chunks, int64_t total,
                                                                 int vec) {
    constexpr bool NV = FMT == CLEF_NVFP4;
    griddep_wait();
    griddep_launch();
    const int64_t code_stride = int64_t(a.cols + 31) / 32 * 16;
    const int kgroups = (a.cols + kFp4Tile - 1) / kFp4Tile * (NV ? 4 : 2);
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < total; i += int64_t(gridDim.x) * kThreads) {
        const int64_t row = i / chunks;
        const int chunk = int(i - row * chunks);
        const uint32_t codes = reinterpret_cast<const uint32_t*>(a.codes + row * code_stride)[chunk];
        const int block = NV ? chunk >> 1 : chunk >> 2;
        const uint32_t byte = a.scales[(row / kFp4RowGroup * kgroups + (block >> 2)) * kFp4ScaleGroup + (row % 32) * 16 +
                                       (row % kFp4RowGroup) / 32 * 4 + (block & 3)];
        float scale, r = 1.f;
        if constexpr (NV) {
            scale = from_e4m3(byte);
            r = a.row_scale[row];
        } else {
            scale = byte == 0xFFu ? __uint_as_float(0x7FC00000u)
                                  : __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
        }
        uint32_t h[4];
        unpack_e2m1(codes, h);
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
            v[2 * j] = f.x * scale * r;
            v[2 * j + 1] = f.y * scale * r;
        }
        store8<DT>(a.out, row * a.row_stride + chunk * 8, v, a.cols - chunk * 8, vec != 0);
    }
}

template <int FMT, int DT, bool VEC>
cudaError_t quantize_rows(const Fp4QuantizeArgs& a, cudaStream_t s) {
    // Few rows: as many warps a row as it has tiles, for latency.  Many: as few as hold the
    // row in registers (16 tiles of 16-bit values, 8 of fp32), so that more reads are in flight
    // and no barrier is met.
    const int ktiles = fp4_ktiles(a.cols);
    constexpr int kMost = DT == CLEF_FP32 ? 8 : 16;
    const int64_t warps = int64_t(num_sms()) * 16;
    int W = 1;
    while (W < 8 && W < ktiles && (ktiles > kMost * W || int64_t(a.rows) * W < warps)) W *= 2;
    const int tiles = (ktiles + W - 1) / W;
    const dim3 grid(unsigned((int64_t(a.rows) * W + kThreads / 32 - 1) / (kThreads / 32)));
    if (tiles <= 1) return launch_pdl(fp4_quantize_kernel<FMT, DT, VEC, 1>, grid, dim3(kThreads), 0, s, a, W);
    if (tiles <= 4) return launch_pdl(fp4_quantize_kernel<FMT, DT, VEC, 4>, grid, dim3(kThreads), 0, s, a, W);
    if (tiles <= 8) return launch_pdl(fp4_quantize_kernel<FMT, DT, VEC, 8>, grid, dim3(kThreads), 0, s, a, W);
    if constexpr (kMost == 16)
        if (tiles <= 16) return launch_pdl(fp4_quantize_kernel<FMT, DT, VEC, 16>, grid, dim3(kThreads), 0, s, a, W);
    return cudaErrorInvalidValue;
}

template <int FMT, int DT>
cudaError_t quantize_type(const Fp4QuantizeArgs& a, cudaStream_t s) {
    constexpr int size = DT == CLEF_FP32 ? 4 : 2;
    const bool vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.row_stride * size % 16 == 0 && a.cols % 8 == 0;
    return vec ? quantize_rows<FMT, DT, true>(a, s) : quantize_rows<FMT, DT, false>(a, s);
}

template <int FMT, int DT>
cudaError_t dequantize_type(const Fp4DequantizeArgs& a, cudaStream_t s) {
    constexpr int size = DT == CLEF_FP32 ? 4 : 2;
    const int vec = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.row_stride * size % 16 == 0 && a.cols % 8 == 0;
    const int chunks = (a.cols + 7) / 8;
    const int64_t total = int64_t(a.rows) * chunks;
    const int64_t blocks = (total + kThreads - 1) / kThreads, most = int64_t(num_sms()) * 32;
    return launch_pdl(fp4_dequantize_kernel<FMT, DT>, dim3(unsigned(blocks < most ? blocks : most)), dim3(kThreads), 0,
                      s, a, chunks, total, vec);
}

}  // namespace

cudaError_t launch_fp4_quantize(const Fp4QuantizeArgs& a, int format, int dtype, cudaStream_t s) {
    if (format == CLEF_MXFP4) {
        if (dtype == CLEF_BF16) return quantize_type<CLEF_MXFP4, CLEF_BF16>(a, s);
        if (dtype == CLEF_FP16) return quantize_type<CLEF_MXFP4, CLEF_FP16>(a, s);
        return quantize_type<CLEF_MXFP4, CLEF_FP32>(a, s);
    }
    if (dtype == CLEF_BF16) return quantize_type<CLEF_NVFP4, CLEF_BF16>(a, s);
    if (dtype == CLEF_FP16) return quantize_type<CLEF_NVFP4, CLEF_FP16>(a, s);
    return quantize_type<CLEF_NVFP4, CLEF_FP32>(a, s);
}

cudaError_t launch_fp4_dequantize(const Fp4DequantizeArgs& a, int format, int dtype, cudaStream_t s) {
    if (format == CLEF_MXFP4) {
        if (dtype == CLEF_BF16) return dequantize_type<CLEF_MXFP4, CLEF_BF16>(a, s);
        if (dtype == CLEF_FP16) return dequantize_type<CLEF_MXFP4, CLEF_FP16>(a, s);
        return dequantize_type<CLEF_MXFP4, CLEF_FP32>(a, s);
    }
    if (dtype == CLEF_BF16) return dequantize_type<CLEF_NVFP4, CLEF_BF16>(a, s);
    if (dtype == CLEF_FP16) return dequantize_type<CLEF_NVFP4, CLEF_FP16>(a, s);
    return dequantize_type<CLEF_NVFP4, CLEF_FP32>(a, s);
}

}  // namespace clef
