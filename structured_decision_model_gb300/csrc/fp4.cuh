// Rows into microscaled 4-bit form: what the kernels that quantise share.
//
// Exact decisions.  A code is right when the quotient x / scale falls on the right side of
// the midpoints of e2m1 (multiples of 1/4 up to 5), ties included.  The quotient by a
// rounded reciprocal is off by 2^-23 of itself; adding and taking off 384 rounds it to a
// multiple of 2^-15.  For bf16 and fp16 values a quotient that is no midpoint is at least
// 2^-13 away from one (the value has 11 bits, the midpoint times the scale at most 7), so
// the rounded quotient is on the true side, and a midpoint comes out as itself.  An fp32
// value may lie closer: what it has left over, x - q * scale, is exact in one fused
// multiply-add, and its sign moves the quotient off the midpoint to the true side.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "fp4.h"

namespace clef {

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

// Sixteen values of a row (a lane's; blocks of 32 are two neighbouring lanes') as codes and their block's scale.
struct Coded {
    uint2 codes;
    uint32_t byte;  // the scale as stored
    float scale;    // what it stands for, without the row's scale; NaN where the block holds no number
};

// `top`: the block's largest size, as it comes from Raw::top; inv_r: the row scale's reciprocal and tiny whether
// 1 / (block scale * row scale) may pass fp32's range (nvfp4); left: values from the first to the row's end.
template <int FMT, int DT>
__device__ __forceinline__ Coded encode16(uint64_t (&x)[8], float top, float inv_r, bool tiny, int left) {
    constexpr bool NV = FMT == CLEF_NVFP4;
    Coded c;
    float inv;
    const bool bad = !(top < INFINITY);
    if constexpr (NV) {
        c.byte = bad ? 0x7Fu : to_e4m3(sixth<DT == CLEF_FP32>(top * inv_r));
        c.scale = from_e4m3(c.byte);
        inv = c.byte == 0 ? 0.f : reciprocal(c.scale);
    } else {
        const int e = max(exponent_of(top) - 2, -127);
        c.byte = bad ? 0xFFu : uint32_t(e + 127);
        c.scale = __uint_as_float(bad ? 0x7FC00000u : e == -127 ? 0x00400000u : uint32_t(e + 127) << 23);
        inv = pow2(-e);
    }
    float v[16];
    if constexpr (DT == CLEF_FP32) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float2 f = both_of(x[j >> 1]);
            const float y = (j & 1 ? f.y : f.x) * (NV ? inv_r : inv);  // powers of two
            const float q = (NV ? fmaf(y, inv, kGrid) : y + kGrid) - kGrid;
            const float rest = NV ? fmaf(-q, c.scale, y) : y - q;
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
        if (tiny) {  // in two steps
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
    c.codes = make_uint2(pack_e2m1(v), pack_e2m1(v + 8));
    if (bad) {  // any number: the scale makes it NaN; behind the row's end zeros as ever
        c.codes.x = left >= 8 ? 0x22222222u : left > 0 ? 0x22222222u >> (32 - 4 * left) : 0u;
        c.codes.y = left >= 16 ? 0x22222222u : left > 8 ? 0x22222222u >> (64 - 4 * left) : 0u;
    }
    return c;
}

// Four blocks' scales as one word, in every lane of theirs; true in the one that writes it.
template <int FMT>
__device__ __forceinline__ bool scale_word(uint32_t byte, int lane, uint32_t* word) {
    constexpr bool NV = FMT == CLEF_NVFP4;
    uint32_t w = byte << (8 * (NV ? lane & 3 : lane >> 1 & 3));
    w |= __shfl_xor_sync(0xffffffffu, w, NV ? 1 : 2);
    w |= __shfl_xor_sync(0xffffffffu, w, NV ? 2 : 4);
    *word = w;
    return (lane & (NV ? 3 : 7)) == 0;
}

// The largest finite size among a lane's values, from their block's largest size.
template <int DT>
__device__ __forceinline__ float finite_top(const Raw<DT>& raw, float top) {
    if (top < INFINITY) return top;
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const float v = fabsf(raw.at(j));
        if (v < INFINITY) most = fmaxf(most, v);
    }
    return most;
}

// r of a row, its reciprocal, and whether dividing by it and a block's scale takes two steps.
struct RowScale {
    float r, inv;
    bool tiny;
};
__device__ __forceinline__ RowScale row_scale_of(float row_top) {
    const int e = max(exponent_of(row_top) - 10, -126);
    return RowScale{pow2(e), pow2(-e), e < -100};
}

// Sums of a lane's values and of their squares (what lies behind the row's end is 0).
__device__ __forceinline__ uint64_t moments16(const uint64_t (&x)[8]) {
    uint64_t t = x[0], u = mul2(x[0], x[0]);
#pragma unroll
    for (int j = 1; j < 8; ++j) {
        t = add2(t, x[j]);
        u = fma2(x[j], x[j], u);
    }
    const float2 a = both_of(t), b = both_of(u);
    return pair_of(a.x + a.y, b.x + b.y);
}

// How a row's variance is found from its distances from the mean, where the mean square less the mean's square does not
// give it.  `by` scales the distances, a power of two: where the mean square passes fp32's range, so may the distances'
// (those that count are above 2^30 there, steps of values near 2^57 and more).
struct Spread {
    float mean, by;
};
constexpr float kFar = 2.3283064365386963e-10f;  // 2^-32
__device__ __forceinline__ Spread spread_of(float mean, float var) { return Spread{mean, var < INFINITY ? 1.f : kFar}; }
__device__ __forceinline__ bool far_from_zero(float mean, float var) { return !(mean * mean <= var && var < INFINITY); }
__device__ __forceinline__ float rstd_of(float var, float by) { return rsqrtf(var + 1e-5f * by * by) * by; }

// Sums of a lane's scaled distances from the mean and of their squares; `left` as in encode16.
template <int DT>
__device__ __forceinline__ uint64_t moments_apart(const Raw<DT>& raw, const Spread& from, int left) {
    const uint64_t less = pair_of(-from.mean, -from.mean), by = pair_of(from.by, from.by);
    uint64_t t = 0, u = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float2 f = both_of(mul2(add2(raw.two(j), less), by));
        if (2 * j >= left) f.x = 0.f;
        if (2 * j + 1 >= left) f.y = 0.f;
        const uint64_t d = pair_of(f.x, f.y);
        t = add2(t, d);
        u = fma2(d, d, u);
    }
    const float2 a = both_of(t), b = both_of(u);
    return pair_of(a.x + a.y, b.x + b.y);
}

// What the distances' mean is corrects the first mean to within half a step, and the distances' mean square less its
// square is the variance, without the square of the first mean's rounding (0.008 at a mean of 10^5: more than 1e-5 in the
// variance of a constant row).  Where that square is most of it, distances from the corrected mean are taken: a row that
// is not constant spreads over at least a step, so that those lose a bit at most.
// (Means and variances that are no numbers stay as they are.)
__device__ __forceinline__ float corrected_mean(const Spread& from, float rest) {
    const float m = fmaf(rest, 1.f / from.by, from.mean);
    return fabsf(m) < INFINITY ? m : from.mean;
}
__device__ __forceinline__ float variance_apart(float rest, float square) {
    return square < INFINITY ? fmaxf(fmaf(-rest, rest, square), 0.f) : square;
}

__device__ __forceinline__ bool mostly_rounding(float rest, float square) { return !(4.f * rest * rest <= square); }

}  // namespace clef
