// Rows into microscaled 4-bit form and back.
//
// Quantise.  A row belongs to one or more whole warps and stays in their registers: its
// largest sizes, its mean and variance and its codes come from one read of memory.  A lane holds 8 consecutive values of
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
#include <type_traits>

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
__device__ __forceinline__ uint32_t pack_e2m1(const float* v) {
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
__device__ __forceinline__ void unpack_e2m1(uint32_t codes, uint32_t* h) {
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

// t / 6 so that rounding it to few bits gives what rounding the true quotient gives.  One residual
// correction gives the nearest fp32 number, which is the quotient itself where that is a border of
// e4m3; for 16-bit values (t has 11 bits at most) a quotient that is none is far from one.  An fp32
// value's may round to a border: it is cut off instead, with the last bit set where something was cut.
template <bool WIDE>
__device__ __forceinline__ float sixth(float t) {
    constexpr float kSixth = 1.f / 6.f;
    const float q0 = t * kSixth;
    const float q = fmaf(fmaf(-q0, 6.f, t), kSixth, q0);
    if constexpr (!WIDE) return q;
    const float rest = fmaf(-q, 6.f, t);
    const uint32_t b = __float_as_uint(q) - (rest < 0.f ? 1u : 0u);
    return __uint_as_float(rest != 0.f ? b | 1u : b);
}

__device__ __forceinline__ float reciprocal(float x) {  // to 1 ulp
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The larger size of each half of two words of 16-bit floats, NaN if one is; the signs are of no use.
template <int DT>
__device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b) {
    uint32_t m;
    if constexpr (DT == CLEF_BF16) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    else asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    return m;
}

// The 16 values of a lane as they lie in memory: 8 words of two, or 16 fp32.
template <int DT>
struct Raw {
    static constexpr int kWords = DT == CLEF_FP32 ? 16 : 8;
    uint32_t w[kWords];
    // values 2j and 2j + 1 as an fp32 pair
    __device__ __forceinline__ uint64_t two(int j) const {
        if constexpr (DT == CLEF_FP32) return pair_of(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
        else if constexpr (DT == CLEF_BF16) return pair_of(bf16_lo(w[j]), bf16_hi(w[j]));
        else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            return pair_of(f.x, f.y);
        }
    }
    __device__ __forceinline__ float at(int j) const {
        const float2 f = both_of(two(j >> 1));
        return j & 1 ? f.y : f.x;
    }
    // bits of the largest size, which order as the sizes do, with infinity and NaN above every number
    __device__ __forceinline__ uint32_t top() const {
        if constexpr (DT == CLEF_FP32) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 16; ++j) m = max(m, w[j] & 0x7FFFFFFFu);
            return m;
        } else {
            const uint32_t m = larger2<DT>(larger2<DT>(larger2<DT>(w[0], w[1]), larger2<DT>(w[2], w[3])),
                                           larger2<DT>(larger2<DT>(w[4], w[5]), larger2<DT>(w[6], w[7])));
            const uint32_t t = max(m & 0x7FFFu, m >> 16 & 0x7FFFu);
            if constexpr (DT == CLEF_BF16) return t << 16;
            else return __float_as_uint(__half2float(__ushort_as_half(uint16_t(t))));
        }
    }
};

// LANES lanes' 16 values each from column col0 of a row on, `lane` the one's place among them; what lies
// behind the row reads as 0.
// VEC: every row starts on 16 bytes and has a multiple of 8 values, so a lane's are read as
// whole 16-byte pieces.  Otherwise neighbours are read side by side and handed round
// through shared memory (3001 x 1111 fp16: 4.3 us; value by value in each lane 7.3).
template <int DT, bool VEC, int LANES>
__device__ __forceinline__ Raw<DT> load16(const void* x, int64_t row0, int col0, int cols, int lane, uint32_t* stage) {
    Raw<DT> r;
    if constexpr (VEC) {
        constexpr int kSize = DT == CLEF_FP32 ? 4 : 2;
        const int col = col0 + lane * 16;
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x) + (row0 + col) * kSize);
#pragma unroll
        for (int i = 0; i < Raw<DT>::kWords / 4; ++i) {
            const uint4 v = col + i * (16 / kSize) < cols ? p[i] : make_uint4(0, 0, 0, 0);
            r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
        }
    } else {
        using T = std::conditional_t<DT == CLEF_FP32, uint32_t, uint16_t>;
        const T* p = static_cast<const T*>(x) + row0 + col0;
        T* to = reinterpret_cast<T*>(stage);
        T v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = col0 + LANES * j + lane < cols ? p[LANES * j + lane] : T(0);
        __syncwarp();  // the last piece has been read
#pragma unroll
        for (int j = 0; j < 16; ++j) to[LANES * j + lane] = v[j];
        __syncwarp();
        const uint4* own = reinterpret_cast<const uint4*>(stage + lane * Raw<DT>::kWords);
#pragma unroll
        for (int i = 0; i < Raw<DT>::kWords / 4; ++i) {
            const uint4 u = own[i];
            r.w[4 * i] = u.x; r.w[4 * i + 1] = u.y; r.w[4 * i + 2] = u.z; r.w[4 * i + 3] = u.w;
        }
    }
    return r;
}

// Over the LANES lanes of an aligned group.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The largest of a row that W warps share (a half of a warp has W = 1).
template <int LANES>
__device__ __forceinline__ float row_max(float v, float* red, int W, int warp) {
    v = lanes_max<LANES>(v);
    if (LANES < 32 || W == 1) return v;
    __syncthreads();  // red may still be read from the last call
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    const int w0 = warp / W * W;
    for (int i = 0; i < W; ++i) v = fmaxf(v, red[w0 + i]);
    return v;
}

// Sums over a row of what its lanes have for each of its pieces: pieces in order, then lanes, so that a sum
// does not depend on how many warps share the row.  One warp (or a half) adds up as it goes; several
// leave what they have in shared memory.
template <int LANES>
struct RowSum {
    float (*all)[32];  // the row's pieces
    float own = 0.f;
    __device__ __forceinline__ void add(float v, int W, int piece, int lane) {
        if (LANES < 32 || W == 1) own += v;
        else all[piece][lane] = v;
    }
    __device__ __forceinline__ float get(int W, int pieces, int lane) {
        if (LANES == 32 && W > 1) {
            __syncthreads();
            own = 0.f;
            for (int i = 0; i < pieces; ++i) own += all[i][lane];
        }
        return lanes_sum<LANES>(own);
    }
};

// STEPS: 512-value pieces of a row that a warp keeps, 16 values a lane; W warps a row (a power of
// two), so a row has at most 512 * STEPS * W values.  LANES 16: rows of up to 256 values, two a warp.
// EXTRA: statistics or sums are asked for.  64 registers a thread, for 32 warps an SM: with 8 pieces a warp and half the warps 131072 x 4096 bf16 took 301 us
// instead of 252.
template <int FMT, int DT, bool VEC, int STEPS, int LANES, bool EXTRA>
__global__ void __launch_bounds__(kThreads, DT == CLEF_FP32 && STEPS == 4 ? 2 : 4) fp4_quantize_kernel(const Fp4QuantizeArgs a, int W) {
    constexpr bool NV = FMT == CLEF_NVFP4;
    __shared__ float red[kThreads / 32];
    __shared__ float partial[EXTRA ? 3 : 1][EXTRA ? kThreads / 32 * STEPS : 1][32];
    __shared__ __align__(16) uint32_t stage[VEC ? 1 : kThreads / 32][VEC ? 4 : 32 * Raw<DT>::kWords];
    griddep_wait();
    griddep_launch();  // behind the wait: whoever starts early may take what came before us as done
    static_assert(LANES == 32 || STEPS == 1, "a half of a warp keeps one tile of a row");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x % LANES;
    const int64_t row = LANES == 32 ? int64_t(blockIdx.x) * (kThreads / 32 / W) + warp / W
                                    : int64_t(blockIdx.x) * (kThreads / LANES) + threadIdx.x / LANES;
    const bool mine = row < a.rows;  // threads behind the last row still meet the barriers and shuffles
    const int part = LANES == 32 ? warp % W : 0;
    const int padded = mine ? (a.cols + kFp4Tile - 1) / kFp4Tile * kFp4Tile : 0;  // columns that have scales
    const bool stats = EXTRA && a.mean, sums = EXTRA && a.sums;  // the same for every thread
    const int64_t row0 = row * a.row_stride;

    Raw<DT> raw[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int col0 = (i * W + part) * 512;
        uint32_t* own = stage[VEC ? 0 : warp] + (VEC || LANES == 32 ? 0 : (threadIdx.x & 16) * Raw<DT>::kWords);
        if (LANES < 32 || col0 < padded)
            raw[i] = load16<DT, VEC, LANES>(a.x, mine ? row0 : 0, col0, mine ? a.cols : 0, lane, own);
        else raw[i] = Raw<DT>{};
    }
    // the largest size of every block and of the row's finite blocks
    float top[STEPS], row_top = 0.f;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        uint32_t t = raw[i].top();
        if (!NV) t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
        top[i] = __uint_as_float(t);
        if (NV) {
            if (top[i] < INFINITY) row_top = fmaxf(row_top, top[i]);
            else {  // the largest finite size of a block that is not finite
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float v = fabsf(raw[i].at(j));
                    if (v < INFINITY) row_top = fmaxf(row_top, v);
                }
            }
        }
    }
    float inv_r = 1.f, r = 1.f;
    bool tiny = false;
    if constexpr (NV) {
        row_top = row_max<LANES>(row_top, red, W, warp);
        const int e = max(exponent_of(row_top) - 10, -126);
        r = pow2(e);
        inv_r = pow2(-e);
        tiny = e < -100;  // 1 / (block scale * r) may pass fp32's range: divide in two steps
        if (mine && part == 0 && lane == 0) a.row_scale[row] = r;
    }
    const int64_t code_stride = int64_t(a.cols + 31) / 32 * 16;
    uint8_t* codes = a.codes + row * code_stride;
    uint8_t* scales = a.scales + (row / kFp4RowGroup * (padded >> (NV ? 6 : 7))) * kFp4ScaleGroup +
                      (row % 32) * 16 + (row % kFp4RowGroup) / 32 * 4;
    const int first = EXTRA ? warp / W * W * STEPS : 0;  // of the row's pieces among the block's
    RowSum<LANES> sum{partial[0] + first}, squares{partial[EXTRA ? 1 : 0] + first}, total{partial[EXTRA ? 2 : 0] + first};
    const int pieces = (a.cols + 511) / 512;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        if (LANES == 32 && (i * W + part) * 512 >= padded) continue;  // the same for a whole warp
        const int col = (i * W + part) * 512 + lane * 16;
        const int left = a.cols - col;  // values from the lane's first to the row's end
        uint32_t byte;    // the block's scale as stored
        float scale, inv; // what it stands for (without r) and its reciprocal
        const bool bad = !(top[i] < INFINITY);
        if constexpr (NV) {
            byte = bad ? 0x7Fu : to_e4m3(sixth<DT == CLEF_FP32>(top[i] * inv_r));
            scale = from_e4m3(byte);
            inv = byte == 0 ? 0.f : reciprocal(scale);
        } else {
            const int e = max(exponent_of(top[i]) - 2, -127);
            byte = bad ? 0xFFu : uint32_t(e + 127);
            scale = __uint_as_float(e == -127 ? 0x00400000u : uint32_t(e + 127) << 23);
            inv = pow2(-e);
        }
        uint64_t x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = raw[i].two(j);
        if (stats) {  // (what lies behind the row's end is 0)
            uint64_t t = x[0], u = mul2(x[0], x[0]);
#pragma unroll
            for (int j = 1; j < 8; ++j) {
                t = add2(t, x[j]);
                u = fma2(x[j], x[j], u);
            }
            const float2 t2 = both_of(t), u2 = both_of(u);
            sum.add(t2.x + t2.y, W, i * W + part, lane);
            squares.add(u2.x + u2.y, W, i * W + part, lane);
        }
        float v[16];
        if constexpr (DT == CLEF_FP32) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float y = raw[i].at(j) * (NV ? inv_r : inv);  // powers of two
                const float q = (NV ? fmaf(y, inv, kGrid) : y + kGrid) - kGrid;
                const float rest = NV ? fmaf(-q, scale, y) : y - q;
                v[j] = inv == 0.f ? 0.f : q + (rest > 0.f ? kAside : rest < 0.f ? -kAside : 0.f);
            }
        } else if constexpr (!NV) {  // by a power of two: exact
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 q = both_of(mul2(x[j], pair_of(inv, inv)));
                v[2 * j] = q.x;
                v[2 * j + 1] = q.y;
            }
        } else {
            const uint64_t grid = pair_of(kGrid, kGrid), back = pair_of(-kGrid, -kGrid);
            float by1 = inv;
            if (tiny) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = mul2(x[j], pair_of(inv_r, inv_r));
            } else {
                by1 *= inv_r;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 q = both_of(add2(fma2(x[j], pair_of(by1, by1), grid), back));
                v[2 * j] = q.x;
                v[2 * j + 1] = q.y;
            }
        }
        uint2 packed = make_uint2(pack_e2m1(v), pack_e2m1(v + 8));
        if (bad) {  // any number: the scale makes it NaN; behind the row's end zeros as ever
            packed.x = left >= 8 ? 0x22222222u : left > 0 ? 0x22222222u >> (32 - 4 * left) : 0u;
            packed.y = left >= 16 ? 0x22222222u : left > 8 ? 0x22222222u >> (64 - 4 * left) : 0u;
        }
        if (mine && col < 2 * code_stride) *reinterpret_cast<uint2*>(codes + col / 2) = packed;
        // four blocks' scales are one word, written by the first lane of theirs
        uint32_t word = byte << (8 * (NV ? lane & 3 : lane >> 1 & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, NV ? 1 : 2);
        word |= __shfl_xor_sync(0xffffffffu, word, NV ? 2 : 4);
        if ((lane & (NV ? 3 : 7)) == 0 && col < padded)
            *reinterpret_cast<uint32_t*>(scales + int64_t(col >> (NV ? 6 : 7)) * kFp4ScaleGroup) = word;
        if (sums) {
            uint32_t h[8];
            unpack_e2m1(packed.x, h);
            unpack_e2m1(packed.y, h + 4);
            float t = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
                t += f.x + f.y;
            }
            total.add(t * (bad ? __uint_as_float(0x7FC00000u) : scale), W, i * W + part, lane);
        }
    }
    if (stats) {
        const float mean = sum.get(W, pieces, lane) / float(a.cols);
        float var = squares.get(W, pieces, lane) / float(a.cols) - mean * mean;
        // A mean square less a mean's loses as many bits as the mean exceeds the spread: such rows (and those
        // whose squares pass fp32) are read once more and sum the squares of what is left behind the mean.
        const bool far = mine && !(mean * mean <= var);
        if (LANES < 32 || W == 1 ? __any_sync(0xffffffffu, far) : __syncthreads_or(far)) {
            const uint64_t less = pair_of(-mean, -mean);
            RowSum<LANES> apart{sum.all};  // every thread is past the sums' barriers, and has read them
#pragma unroll 1
            for (int i = 0; i < STEPS; ++i) {
                if (LANES == 32 && (i * W + part) * 512 >= padded) continue;
                const int col0 = (i * W + part) * 512;
                const int left = a.cols - (col0 + lane * 16);  // values from the lane's first to the row's end
                uint32_t* own = stage[VEC ? 0 : warp] + (VEC || LANES == 32 ? 0 : (threadIdx.x & 16) * Raw<DT>::kWords);
                const Raw<DT> again = load16<DT, VEC, LANES>(a.x, mine ? row0 : 0, col0, mine ? a.cols : 0, lane, own);
                float q = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 d = both_of(add2(again.two(j), less));
                    if (2 * j < left) q = fmaf(d.x, d.x, q);
                    if (2 * j + 1 < left) q = fmaf(d.y, d.y, q);
                }
                apart.add(q, W, i * W + part, lane);
            }
            const float v = apart.get(W, pieces, lane) / float(a.cols);
            if (far) var = v;
        }
        if (mine && part == 0 && lane == 0) {
            a.mean[row] = mean;
            a.rstd[row] = 1.f / sqrtf(var + 1e-5f);
        }
    }
    if (sums) {
        const float all = total.get(W, pieces, lane);
        if (mine && part == 0 && lane == 0) a.sums[row] = all * r;
    }
}

// Read back: a warp takes 1024 values of a row, 4 times 8 a lane (4 bytes of codes, one scale).  VEC: every row
// of the output starts on a multiple of 8 values' bytes and has a multiple of 8 values, so that a lane
// stores its 8 at once; otherwise the warp hands the values round and stores 32 neighbours at a time.
constexpr int kBack = 1024;

// SHORT (VEC only): rows of up to 256 values; a warp takes 128 neighbouring eights of any rows.
template <int FMT, int DT, bool VEC, bool SHORT>
__global__ void __launch_bounds__(kThreads) fp4_dequantize_kernel(const Fp4DequantizeArgs a) {
    constexpr bool NV = FMT == CLEF_NVFP4;
    __shared__ __align__(16) float stage[VEC ? 1 : kThreads / 32][VEC ? 4 : 256];
    griddep_wait();
    griddep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t item = uint64_t(blockIdx.x) * (kThreads / 32) + warp;
    const int64_t code_stride = int64_t(a.cols + 31) / 32 * 16;
    const int kgroups = (a.cols + kFp4Tile - 1) / kFp4Tile * (NV ? 4 : 2);
    int64_t row0;  // the warp's first row, and where in it
    int at0;       // (SHORT: in eights)
    const uint32_t per = SHORT ? uint32_t(a.cols) / 8 : uint32_t(a.cols + kBack - 1) / kBack;
    if constexpr (SHORT) {
        row0 = int64_t(item * 128 / per);
        at0 = int(item * 128 - uint64_t(row0) * per);
    } else {
        row0 = int64_t(item / per);
        at0 = int(item - uint64_t(row0) * per) * kBack;
    }
    if (row0 >= a.rows) return;
    int64_t rows[4];
    int cols[4];
    uint32_t packed[4], byte[4];
    float r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (SHORT) {
            const uint32_t t = uint32_t(at0) + i * 32 + lane;
            rows[i] = row0 + t / per;
            cols[i] = rows[i] < a.rows ? int(t % per) * 8 : a.cols;
        } else {
            rows[i] = row0;
            cols[i] = at0 + i * 256 + lane * 8;
        }
        const int64_t row = rows[i];
        const int block = NV ? cols[i] >> 4 : cols[i] >> 5;
        packed[i] = byte[i] = 0;
        r[i] = 1.f;
        if (cols[i] < a.cols) {
            packed[i] = *reinterpret_cast<const uint32_t*>(a.codes + row * code_stride + cols[i] / 2);
            byte[i] = a.scales[(row / kFp4RowGroup * kgroups + (block >> 2)) * kFp4ScaleGroup + (row % 32) * 16 +
                               (row % kFp4RowGroup) / 32 * 4 + (block & 3)];
            if (NV) r[i] = a.row_scale[row];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t row = rows[i];
        const int col = cols[i];
        if (!SHORT && at0 + i * 256 >= a.cols) break;  // the same for a whole warp
        float scale;
        if constexpr (NV) scale = from_e4m3(byte[i]);
        else scale = byte[i] == 0xFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte[i] == 0 ? 0x00400000u : byte[i] << 23);
        uint32_t h[4];
        unpack_e2m1(packed[i], h);
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
            v[2 * j] = f.x * scale * r[i];
            v[2 * j + 1] = f.y * scale * r[i];
        }
        if constexpr (VEC) {
            if (col >= a.cols) continue;
            uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) +
                                                  (row * a.row_stride + col) * (DT == CLEF_FP32 ? 4 : 2));
            if constexpr (DT == CLEF_FP32) {
                // one whole 32-byte sector a lane
                asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out), "f"(v[0]), "f"(v[1]),
                             "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                             : "memory");
            } else {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (DT == CLEF_BF16) w[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
                    else {
                        const __half2 p = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
                        w[j] = *reinterpret_cast<const uint32_t*>(&p);
                    }
                }
                *out = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
            float* to = stage[warp];
            __syncwarp();  // the last values have been read
            reinterpret_cast<float4*>(to)[2 * lane] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(to)[2 * lane + 1] = make_float4(v[4], v[5], v[6], v[7]);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = at0 + i * 256 + j * 32 + lane;
                if (c >= a.cols) continue;
                const float y = to[j * 32 + lane];
                const int64_t at = row * a.row_stride + c;
                if constexpr (DT == CLEF_FP32) static_cast<float*>(a.out)[at] = y;
                else if constexpr (DT == CLEF_BF16) static_cast<uint16_t*>(a.out)[at] = float_to_bf16(y);
                else static_cast<uint16_t*>(a.out)[at] = __half_as_ushort(__float2half_rn(y));
            }
        }
    }
}

template <int FMT, int DT, bool VEC, bool EXTRA>
cudaError_t quantize_rows(const Fp4QuantizeArgs& a, cudaStream_t s) {
    // Few rows: as many warps a row as it has pieces, for latency.  Many: as few as hold the row in
    // registers (4 pieces of 16-bit values, 2 of fp32).
    const int pieces = (a.cols + 511) / 512;
    constexpr int kMost = DT == CLEF_FP32 ? 2 : 4;
    const int64_t warps = int64_t(num_sms()) * 16;
    int W = 1;
    while (W < 8 && W < pieces && (pieces > kMost * W || int64_t(a.rows) * W < warps)) W *= 2;
    if (a.cols <= 256)
        return launch_pdl(fp4_quantize_kernel<FMT, DT, VEC, 1, 16, EXTRA>, dim3(unsigned((int64_t(a.rows) + 15) / 16)),
                          dim3(kThreads), 0, s, a, 1);
    const int steps = (pieces + W - 1) / W;
    const dim3 grid(unsigned((int64_t(a.rows) * W + kThreads / 32 - 1) / (kThreads / 32)));
    if (steps <= 1) return launch_pdl(fp4_quantize_kernel<FMT, DT, VEC, 1, 32, EXTRA>, grid, dim3(kThreads), 0, s, a, W);
    if (steps <= 2) return launch_pdl(fp4_quantize_kernel<FMT, DT, VEC, 2, 32, EXTRA>, grid, dim3(kThreads), 0, s, a, W);
    if (steps <= 4) return launch_pdl(fp4_quantize_kernel<FMT, DT, VEC, 4, 32, EXTRA>, grid, dim3(kThreads), 0, s, a, W);
    return cudaErrorInvalidValue;
}

template <int FMT, int DT>
cudaError_t quantize_type(const Fp4QuantizeArgs& a, cudaStream_t s) {
    constexpr int size = DT == CLEF_FP32 ? 4 : 2;
    const bool vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.row_stride * size % 16 == 0 && a.cols % 8 == 0;
    const bool extra = a.mean || a.sums;
    if (vec) return extra ? quantize_rows<FMT, DT, true, true>(a, s) : quantize_rows<FMT, DT, true, false>(a, s);
    return extra ? quantize_rows<FMT, DT, false, true>(a, s) : quantize_rows<FMT, DT, false, false>(a, s);
}

template <int FMT, int DT>
cudaError_t dequantize_type(const Fp4DequantizeArgs& a, cudaStream_t s) {
    constexpr int size = DT == CLEF_FP32 ? 4 : 2;
    constexpr int piece = 8 * size;
    const bool vec = reinterpret_cast<uintptr_t>(a.out) % piece == 0 && a.row_stride * size % piece == 0 && a.cols % 8 == 0;
    const bool brief = vec && a.cols <= 256;
    const int64_t items = brief ? (int64_t(a.rows) * (a.cols / 8) + 127) / 128
                                : int64_t(a.rows) * ((a.cols + kBack - 1) / kBack);
    const int64_t blocks = (items + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    return launch_pdl(brief ? fp4_dequantize_kernel<FMT, DT, true, true>
                      : vec ? fp4_dequantize_kernel<FMT, DT, true, false> : fp4_dequantize_kernel<FMT, DT, false, false>,
                      dim3(unsigned(blocks)), dim3(kThreads), 0, s, a);
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
