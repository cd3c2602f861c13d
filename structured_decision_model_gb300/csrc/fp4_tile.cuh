// The tile kernel of the 4-bit products and what it shares with the pair kernel.  See fp4_product.cu for the
// layout.
#pragma once

#include <algorithm>

#include "fp4.cuh"
#include "kernels.h"
#include "per_device.h"

namespace clef {

namespace {

constexpr int kAtomBytes = 128;             // codes of one row of a K tile
constexpr int kWRows = 128;                 // rows of w in a CTA's tile
constexpr int kWBytes = kWRows * kAtomBytes;

constexpr int groups_of(int fmt) { return fmt == CLEF_MXFP4 ? 2 : 4; }  // scale groups of a K tile

// Descriptor of the 32 x 16-byte rows of a scale group: four 8-row core matrices, 128 bytes
// apart, no swizzle.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= uint64_t((saddr >> 4) & 0x3FFFu);
    d |= uint64_t(128 >> 4) << 32;  // stride byte offset
    d |= uint64_t(1) << 46;         // descriptor version
    return d;
}

// Instruction descriptor: e2m1 A and B, K-major, M x N tile, K = 64; scales e8m0 or e4m3,
// `part` the byte of a scale word that the MMA's scales start at (mxfp4: 0 or 2).
__host__ __device__ constexpr uint32_t idesc_fp4(int fmt, int M, int N, int part) {
    return (uint32_t(part) << 4)                              // B's scales
           | (1u << 7)                                        // A format e2m1
           | (1u << 10)                                       // B format e2m1
           | (uint32_t(N >> 3) << 17)                         // N / 8
           | ((fmt == CLEF_MXFP4 ? 1u : 0u) << 23)            // scale format: e8m0 or e4m3
           | (uint32_t(M >> 4) << 24)                         // M / 16
           | (uint32_t(part) << 29);                          // A's scales
}

template <int FMT, bool PAIR>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                        uint32_t accumulate) {
#define CLEF_FP4_MMA(GROUP, VEC)                                                                        \
    asm volatile(                                                                                       \
        "{\n\t.reg .pred p;\n\t"                                                                        \
        "setp.ne.b32 p, %6, 0;\n\t"                                                                     \
        "tcgen05.mma.cta_group::" GROUP ".kind::mxf4nvf4.block_scale.scale_vec::" VEC                   \
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                                              \
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)                                   \
        : "memory")
    if constexpr (FMT == CLEF_MXFP4) {
        if constexpr (PAIR) CLEF_FP4_MMA("2", "2X");
        else CLEF_FP4_MMA("1", "2X");
    } else {
        if constexpr (PAIR) CLEF_FP4_MMA("2", "4X");
        else CLEF_FP4_MMA("1", "4X");
    }
#undef CLEF_FP4_MMA
}

// 32 rows x 16 bytes of shared memory to 4 TMEM columns, repeated in all four lane quarters.
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
    if constexpr (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

template <int OUT>
__device__ __forceinline__ void store_value(void* out, int64_t at, float v) {
    if constexpr (OUT == CLEF_FP32) static_cast<float*>(out)[at] = v;
    else if constexpr (OUT == CLEF_BF16) static_cast<uint16_t*>(out)[at] = float_to_bf16(v);
    else static_cast<uint16_t*>(out)[at] = __half_as_ushort(__float2half_rn(v));
}

// What an output column (a row of w) brings: y = acc * scale * f[m] + (h[m] * sum + bias).
struct ColumnTerms {
    float scale, sum, bias;
};
__device__ __forceinline__ ColumnTerms column_terms(const Fp4ProductArgs& a, int n) {
    ColumnTerms t{1.f, 0.f, 0.f};
    if (n < a.N) {
        if (a.w_scale) t.scale = a.w_scale[n];
        if (a.sums) t.sum = a.sums[n];
        if (a.bias) t.bias = a.bias[n];
    }
    return t;
}

// What an output row (a row of x) brings: f and h of the formula above, kept in shared memory as
// (f, f, h, h) of two rows, so that one read serves two columns of an accumulator.
__device__ __forceinline__ float2 row_terms(const Fp4ProductArgs& a, int m) {
    float2 t = make_float2(1.f, 0.f);
    if (m < a.M) {
        if (a.x_scale) t.x = a.x_scale[m];
        if (a.rstd) {
            const float rs = a.rstd[m];
            t.x *= rs;
            t.y = -a.mean[m] * rs;
        }
    }
    return t;
}
__device__ __forceinline__ void put_row_terms(float* terms, int j, float2 t) {
    float* p = terms + (j >> 1) * 4 + (j & 1);
    p[0] = t.x;
    p[2] = t.y;
}

constexpr int kEpilogue = 256;               // threads of the epilogue: two warps for every 32 TMEM lanes
constexpr int kThreads = 64 + kEpilogue;     // and one warp each for TMA and MMA

constexpr int kKept = -1;
static_assert(kFp4FewRows <= 32, "few rows are one tile");

// Two 16-bit values in one word, the first in its low half.
template <int OUT>
__device__ __forceinline__ uint32_t pack_two(float lo, float hi) {
    if constexpr (OUT == CLEF_FP16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        return pack_bf16(lo, hi);
    }
}

// An output from its accumulator; finish2: of one column and two rows.
__device__ __forceinline__ float finish(float acc, const ColumnTerms& c, float f, float h) {
    return fmaf(acc * c.scale, f, fmaf(h, c.sum, c.bias));
}

__device__ __forceinline__ float2 finish2(float acc0, float acc1, const ColumnTerms& c, const float4& t) {
    const uint64_t acc = mul2(pair_of(acc0, acc1), pair_of(c.scale, c.scale));
    const uint64_t add = fma2(pair_of(t.z, t.w), pair_of(c.sum, c.sum), pair_of(c.bias, c.bias));
    return both_of(fma2(acc, pair_of(t.x, t.y), add));
}

// True in one thread of a converged warp.  The warps that issue TMA and MMA stay converged and pick the
// issuing thread around each batch of instructions: addresses and descriptors then stay in uniform
// registers, where the instructions want them.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(p));
    return p != 0;
}

// A barrier of the epilogue warps, behind which all of them know whether all may go on.
__device__ __forceinline__ bool epilogue_agrees(int ok) {
    int all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.s32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, 256, p;\n\t"
        "selp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(ok)
        : "memory");
    return all != 0;
}

// NC accumulator columns (rows m0 .. of x, of which `rows` exist) of one TMEM lane (column n) out;
// `terms` at row m0.  16-bit values go out two a lane where a.paired says that they may:
// neighbouring lanes swap halves, so that an even lane has columns n, n + 1 of an even row and the
// odd one those of the row behind it.
template <int OUT, int NC>
__device__ __forceinline__ void emit(const Fp4ProductArgs& a, const uint32_t (&r)[NC], const ColumnTerms& col,
                                     const float* terms, int m0, int rows, int n, int lane) {
    const float4* t4 = reinterpret_cast<const float4*>(terms);
    if (OUT != CLEF_FP32 && a.paired) {
        const int odd = lane & 1;
        const uint32_t pick = odd ? 0x3276u : 0x5410u;  // odd: (other's high, own high); even: (own low, other's low)
        uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + int64_t(m0 + odd) * a.ldo + (n - odd));
        const int64_t step = a.ldo;  // two rows, in words
        // rows of this lane, as a count of pairs: all of them in every tile but the last
        const int most = n < a.N ? (min(rows, NC) + 1 - odd) >> 1 : 0;
#pragma unroll
        for (int j = 0; j < NC / 2; ++j) {
            const float2 v = finish2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]), col, t4[j]);
            const uint32_t w = pack_two<OUT>(v.x, v.y);
            const uint32_t other = __shfl_xor_sync(0xffffffffu, w, 1);
            if (j < most) *out = __byte_perm(w, other, pick);
            out += step;
        }
    } else {
        const int most = n < a.N ? rows : 0;
        int64_t at = int64_t(m0) * a.ldo + n;
#pragma unroll
        for (int j = 0; j < NC / 2; ++j) {
            const float2 v = finish2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]), col, t4[j]);
            if (2 * j < most) store_value<OUT>(a.out, at, v.x);
            at += a.ldo;
            if (2 * j + 1 < most) store_value<OUT>(a.out, at, v.y);
            at += a.ldo;
        }
    }
}

// 16 accumulator columns (rows of x) of 32 TMEM lanes (columns of the output) as 16-bit values into a
// staged tile [16 rows][64 columns] of 128-byte swizzled rows; `saddr` is what this lane addresses in it for
// stmatrix.  lo and hi hold lanes 0..15 and 16..31 as tmem_ld16x64 gives them, from register FROM on; a
// thread's values belong to four columns and, of every 8 rows, two: one read of row terms serves
// eight values (a read a pair, with a whole lane's columns in one thread, kept shared memory busy:
// 19.8 against 12.3 us of 4864 x 4096 x 1024 without any output).
template <int OUT, int FROM>
__device__ __forceinline__ void stage16(uint32_t saddr, const uint32_t (&lo)[32], const uint32_t (&hi)[32],
                                        const ColumnTerms (&col)[4], const float* terms, int lane) {
    const float4* t4 = reinterpret_cast<const float4*>(terms) + (lane & 3);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const float4 t = t4[4 * g];
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t* r = (i < 2 ? lo : hi) + FROM + 4 * g + 2 * (i & 1);
            const float2 v = finish2(__uint_as_float(r[0]), __uint_as_float(r[1]), col[i], t);
            w[i] = pack_two<OUT>(v.x, v.y);
        }
        stmatrix_x4_trans(saddr + g * 1024, w);
    }
}

// A barrier of the four warps of one half of the epilogue.
__device__ __forceinline__ void half_sync(int half) {
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(2 + half) : "memory");
}

template <int NC>
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[NC]) {
    if constexpr (NC == 16) tmem_ld16(taddr, r);
    else tmem_ld32(taddr, r);
}

// --------------------------------------------------------- one CTA, one tile
// 128 rows of w x BN rows of x.  Few rows of x leave few tiles, so the K range of a tile is
// cut among the CTAs of a cluster, which stage their fp32 tiles in their own shared memory
// and add them in order through distributed shared memory.  Latency bounds it: 4096 x 4096 takes 4.0 us for one
// row (weights 1.4 us at the copy rate), 5.3 for 64, 6.8 for 128, 7.4 for 256; 16384 x 4096, 24 rows, 6.9 us.
template <int FMT, int BN>
struct TileCfg {
    static constexpr int GROUPS = groups_of(FMT);
    static constexpr int X_BYTES = BN * kAtomBytes;
    static constexpr int S_BYTES = GROUPS * kFp4ScaleGroup;  // of 128 rows of one side
    static constexpr int STAGE = kWBytes + X_BYTES + 2 * S_BYTES;
    static constexpr int STAGES = BN == 32 ? 4 : 3;  // two CTAs an SM
    static constexpr int SMEM = STAGES * STAGE + 1024 /*align*/ + BN * 8 /*row terms*/ + 128 /*barriers*/;
    static constexpr uint32_t S_COLS = 4 * GROUPS;  // TMEM columns of one side's scales
    static constexpr uint32_t TMEM_COLS = BN == 32 ? 64 : 2 * BN;
    static constexpr int LD = kWRows + 4;  // row stride (floats) of a staged tile [BN][128]
    static_assert(BN + 2 * S_COLS <= TMEM_COLS, "accumulator and scales fit");
    static_assert(BN * LD * 4 <= STAGES * STAGE, "a staged tile fits the operand stages");
    static_assert(STAGE % 1024 == 0 && X_BYTES % 1024 == 0, "swizzle atoms start on 1024 bytes");
};


// The S parts of a tile, staged [rows][LD] at `staged` in every CTA of the cluster, added up in order: CTA sp
// finishes rows sp, sp + S, ..., a warp a row, four columns a lane, with 8 remote reads under way at
// once (a column a thread and a row at a time, this took longer than the products: 128 rows x 4096
// x 4096 in two parts 12.5 us, now 8.3).
template <int OUT, int S, int LD>
__device__ __forceinline__ void join_parts(const Fp4ProductArgs& args, uint32_t staged, const float* terms, int m0,
                                           int rows, int n_tile, int sp, int warp, int lane) {
    constexpr int Q = 8 / S;
    const int step = S * (kEpilogue / 32), n0 = n_tile + lane * 4;
    ColumnTerms col[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) col[e] = column_terms(args, n0 + e);
    for (int j0 = sp + S * warp; j0 < rows; j0 += Q * step) {
        float4 v[Q][S];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            // rows past the tile's last are read from where the last is
            const uint32_t at = staged + uint32_t(lane * 16 + min(j0 + q * step, rows - 1) * LD * 4);
#pragma unroll
            for (int i = 0; i < S; ++i) v[q][i] = ld_cluster_f4(cluster_map(at, uint32_t(i)));
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int j = j0 + q * step;
            if (j >= rows) break;
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < S; ++i) {
                acc[0] += v[q][i].x; acc[1] += v[q][i].y;
                acc[2] += v[q][i].z; acc[3] += v[q][i].w;
            }
            const float* t = terms + (j >> 1) * 4 + (j & 1);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = finish(acc[e], col[e], t[0], t[2]);
            const int64_t at = int64_t(m0 + j) * args.ldo + n0;
            if (OUT != CLEF_FP32 && args.paired) {
                uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(args.out) + at);
                if (n0 < args.N) out[0] = pack_two<OUT>(acc[0], acc[1]);
                if (n0 + 2 < args.N) out[1] = pack_two<OUT>(acc[2], acc[3]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n0 + e < args.N) store_value<OUT>(args.out, at + e, acc[e]);
            }
        }
    }
}

// Few rows of x by the epilogue's warps, rows warp, warp + 8, ... each: a row's scale and statistics from all of
// it (its terms go to `terms`, its largest size to `tops`), then the rows' codes and scales of K tiles
// kt0 .. kt1 - 1 into the operand stages, as TMA would have laid them.  The numbers are those of the
// kernel that quantises many rows, in the same order.
template <int FMT, int DT, typename C>
__device__ __forceinline__ void few_rows(const Fp4ProductArgs& args, uint8_t* smem, float* terms, float* tops,
                                         uint64_t* full, uint64_t* empty, int kt0, int kt1, int warp, int lane,
                                         volatile int* abort_flag) {
    constexpr bool NV = FMT == CLEF_NVFP4;
    const int cols = args.cols;
#pragma unroll 1
    for (int m = warp; m < args.M; m += kEpilogue / 32) {
        const int64_t row0 = int64_t(m) * args.x_stride;
        float2 f = make_float2(1.f, 0.f);
        if (NV || args.mean_out) {
            float row_top = 0.f, sum = 0.f, squares = 0.f;
#pragma unroll 4
            for (int c = 0; c < cols; c += 512) {
                const Raw<DT> raw = load16<DT, true, 32>(args.x, row0, c, cols, lane, nullptr);
                if (NV) row_top = fmaxf(row_top, finite_top<DT>(raw, __uint_as_float(raw.top())));
                if (args.mean_out) {
                    uint64_t x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = raw.two(j);
                    const float2 v = both_of(moments16(x));
                    sum += v.x;
                    squares += v.y;
                }
            }
            if (NV) {
                row_top = warp_max(row_top);
                f.x = row_scale_of(row_top).r;
                if (lane == 0) tops[m] = row_top;
            }
            if (args.mean_out) {
                float mean = warp_sum(sum) * args.inv_cols;
                float var = warp_sum(squares) * args.inv_cols - mean * mean;
                Spread from = spread_of(mean, var);
                if (far_from_zero(mean, var)) {  // see the kernel for many rows
#pragma unroll 1
                    for (int turn = 0; turn < 2; ++turn) {
                        float d = 0.f, q = 0.f;
                        for (int c = 0; c < cols; c += 512) {
                            const Raw<DT> raw = load16<DT, true, 32>(args.x, row0, c, cols, lane, nullptr);
                            const float2 v = both_of(moments_apart<DT>(raw, from, cols - (c + lane * 16)));
                            d += v.x;
                            q += v.y;
                        }
                        const float rest = warp_sum(d) * args.inv_cols, square = warp_sum(q) * args.inv_cols;
                        var = variance_apart(rest, square);
                        if (turn == 0) mean = from.mean = corrected_mean(from, rest);
                        if (!mostly_rounding(rest, square)) break;
                    }
                }
                const float rstd = rstd_of(var, from.by);
                f.x *= rstd;
                f.y = -mean * rstd;
                if (blockIdx.x == 0 && lane == 0) {
                    args.mean_out[m] = mean;
                    args.rstd_out[m] = rstd;
                }
            }
        }
        if (lane == 0) put_row_terms(terms, m, f);
    }
    __syncwarp();  // tops
    // two K tiles at a time, 16 values a lane
    int s = 0;
    uint32_t phase = 1;
    for (int kt = kt0; kt < kt1; kt += 2) {
        const int tiles = min(2, kt1 - kt), which = lane >> 4, col = kt * kFp4Tile + lane * 16;
        const int s1 = s + 1 == C::STAGES ? 0 : s + 1;
        const uint32_t phase1 = s1 == 0 ? phase ^ 1u : phase;
        bool ok = mbar_wait_bounded(&empty[s], phase, abort_flag, args.flags, args.wait_ns);
        if (tiles == 2) ok = mbar_wait_bounded(&empty[s1], phase1, abort_flag, args.flags, args.wait_ns) && ok;
        if (!__all_sync(0xffffffffu, ok)) break;
        uint8_t* st = smem + (which ? s1 : s) * C::STAGE + kWBytes;
        const int v = (lane & 15) * 16;  // the first value's place in its K tile
        auto load = [&](int m) {         // (a row behind the last reads as zeros)
            return load16<DT, true, 32>(args.x, int64_t(m) * args.x_stride, kt * kFp4Tile,
                                        m < args.M ? min(cols, (kt + tiles) * kFp4Tile) : 0, lane, nullptr);
        };
        Raw<DT> next = load(warp);
#pragma unroll 1
        for (int m = warp; m < args.M; m += kEpilogue / 32) {
            const Raw<DT> raw = next;
            next = load(m + kEpilogue / 32);  // while this one is worked on
            const RowScale rs = NV ? row_scale_of(tops[m]) : RowScale{1.f, 1.f, false};
            uint32_t t = raw.top();
            if (!NV) t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
            uint64_t x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = raw.two(j);
            const Coded c = encode16<FMT, DT>(x, __uint_as_float(t), rs.inv, rs.tiny, cols - col);
            uint32_t word;
            const bool writes = scale_word<FMT>(c.byte, lane, &word);
            if (which < tiles) {
                // 16-byte pieces of a row's 128 bytes, swizzled by the row
                *reinterpret_cast<uint2*>(st + m * kAtomBytes + (((v >> 5) ^ (m & 7)) << 4) + (v >> 4 & 1) * 8) = c.codes;
                if (writes)
                    *reinterpret_cast<uint32_t*>(st + C::X_BYTES + C::S_BYTES + (v >> (NV ? 6 : 7)) * kFp4ScaleGroup + m * 16) = word;
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&full[s]);
            if (tiles == 2) mbar_arrive(&full[s1]);
        }
        s = tiles == 2 ? (s1 + 1 == C::STAGES ? 0 : s1 + 1) : s1;
        phase = s1 == 0 || (tiles == 2 && s == 0) ? phase ^ 1u : phase;
    }
}

// XT: x's type.  kKept: x is a 4-bit matrix that TMA loads.  Otherwise rows as they come (at most
// kFp4FewRows, 16-byte pieces): the epilogue's warps, idle until the products are done, quantise them
// straight into the operand stages.  Such a call takes one launch and no scratch.
template <int FMT, int BN, int OUT, int XT>
__global__ void __launch_bounds__(kThreads, 2) fp4_tile_kernel(const __grid_constant__ CUtensorMap tmW,
                                                                const __grid_constant__ CUtensorMap tmX,
                                                                const __grid_constant__ CUtensorMap tmSW,
                                                                const __grid_constant__ CUtensorMap tmSX,
                                                                const Fp4ProductArgs args) {
    using C = TileCfg<FMT, BN>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ float tops[XT == kKept ? 1 : kFp4FewRows];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* terms = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE);
    uint64_t* full = reinterpret_cast<uint64_t*>(terms + 2 * BN);
    uint64_t* empty = full + C::STAGES;
    uint64_t* done = empty + C::STAGES;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], XT == kKept ? 1 : 1 + kEpilogue / 32);  // the copies, and the warps that write x
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmX);
        prefetch_tensormap(&tmSW);
        prefetch_tensormap(&tmSX);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int S = args.splits;
    const int sp = int(blockIdx.x) % S, tile = int(blockIdx.x) / S;
    const int n_wt = (args.N + kWRows - 1) / kWRows;
    const int wt = tile % n_wt, xt = tile / n_wt;  // w's tiles next to each other share x's rows
    const int ktiles = (args.k64 + 3) / 4;
    const int kt0 = int(int64_t(sp) * ktiles / S), kt1 = int(int64_t(sp + 1) * ktiles / S);
    if (warp == 0) {
        // what does not come from the kernel before this one is asked for while that still runs
        constexpr int kLoaded = XT == kKept ? C::STAGE : kWBytes + C::S_BYTES;
        auto load_w = [&](int kt, int s) {
            uint8_t* st = smem + s * C::STAGE;
            mbar_arrive_expect_tx(&full[s], kLoaded);
            tma_load_2d(st, &tmW, kt * kAtomBytes, wt * kWRows, &full[s]);
            tma_load_2d(st + kWBytes + C::X_BYTES, &tmSW, 0, wt * args.kgroups + kt * C::GROUPS, &full[s]);
        };
        auto load_x = [&](int kt, int s) {
            if constexpr (XT == kKept) {
                uint8_t* st = smem + s * C::STAGE + kWBytes;
                tma_load_2d(st, &tmX, kt * kAtomBytes, xt * BN, &full[s]);
                // x's scales of the 128-row group that the tile lies in (tiles of fewer rows: the first)
                tma_load_2d(st + C::X_BYTES + C::S_BYTES, &tmSX, 0, xt * BN / kFp4RowGroup * args.kgroups + kt * C::GROUPS, &full[s]);
            }
        };
        // The first K tiles' stages wait for nobody: their copies are asked for under one election.  Converged, the warp
        // keeps addresses in uniform registers (511 rows x 4096 x 16384 23.9 -> 22.9 us, 511 x 2560 x 640 4.6 -> 4.5;
        // an election for each of the first K tiles as well: 23.2 and 4.6).
        const int last = kt1 - args.withheld;  // the K tiles that are loaded end here
        const int free = min(C::STAGES, last - kt0);
        if (elect_one() && args.w_settled) {
            for (int k = 0; k < free; ++k) load_w(kt0 + k, k);
        }
        griddep_wait();
        griddep_launch();
        if (elect_one()) {
            for (int k = 0; k < free; ++k) {
                if (!args.w_settled) load_w(kt0 + k, k);
                load_x(kt0 + k, k);
            }
        }
        __syncwarp();
        bool ok = true;
        int i = free, s = 0;  // stages filled so far, and the next one
        uint32_t phase = 0;
        for (int kt = kt0 + free; kt < last; ++kt, ++i) {
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&empty[s], phase, abort_flag, args.flags, args.wait_ns));
            if (!ok) break;
            if (elect_one()) {
                load_w(kt, s);
                load_x(kt, s);
            }
            __syncwarp();
            if (++s == C::STAGES) {
                s = 0;
                phase ^= 1u;
            }
        }
        if (!ok) {  // let every copy that was asked for land before the CTA goes
            for (int j = i < C::STAGES ? 0 : i - C::STAGES; j < i; ++j)
                mbar_wait_bounded(&full[j % C::STAGES], uint32_t(j / C::STAGES & 1), nullptr, nullptr);
        }
        __syncwarp();
    } else if (warp == 1) {
        griddep_wait();  // the time that the kernel before takes does not count against this warp's waits
        const uint32_t sw = tmem + BN, sx = sw + C::S_COLS;
        const uint64_t d0 = smem_desc_sw128(smem_u32(smem)), c0 = scale_desc(smem_u32(smem) + kWBytes + C::X_BYTES);
        bool ok = true;
        int s = 0;
        uint32_t phase = 0;
        for (int kt = kt0; kt < kt1; ++kt) {
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[s], phase, abort_flag, args.flags, args.wait_ns));
            if (!ok) break;
            tc_fence_after();
            const uint64_t da = d0 + uint64_t(s * (C::STAGE >> 4)), db = da + (kWBytes >> 4);
            const uint64_t dc = c0 + uint64_t(s * (C::STAGE >> 4));
            const int nk = min(4, args.k64 - 4 * kt);
            if (elect_one()) {
#pragma unroll
                for (int g = 0; g < C::GROUPS; ++g) {
                    copy_scales<false>(sw + 4 * g, dc + g * (kFp4ScaleGroup >> 4));
                    copy_scales<false>(sx + 4 * g, dc + (C::GROUPS + g) * (kFp4ScaleGroup >> 4));
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k >= nk) break;
                    constexpr bool MX = FMT == CLEF_MXFP4;
                    const uint32_t g = 4 * (MX ? k / 2 : k);  // mxfp4: a word holds two MMAs' scales
                    mma_fp4<FMT, false>(tmem, da + uint64_t(2 * k), db + uint64_t(2 * k),
                                        idesc_fp4(FMT, kWRows, BN, MX ? (k & 1) * 2 : 0), sw + g, sx + g,
                                        kt > kt0 || k > 0 ? 1u : 0u);
                }
                tc_commit(&empty[s]);
            }
            __syncwarp();
            if (++s == C::STAGES) {
                s = 0;
                phase ^= 1u;
            }
        }
        // on every path: what was issued completes before TMEM is freed
        if (elect_one()) tc_commit(done);
        __syncwarp();
        if (!mbar_wait_bounded(done, 0, nullptr, args.flags) || !ok) *abort_flag = 1;
        __syncwarp();
    } else {
        griddep_wait();  // the row terms may come from the kernel before
        const int t = int(threadIdx.x) - 64;
        const int quarter = warp & 3, half = t >> 7;  // TMEM lanes that this warp may read; its half of the columns
        const int row = quarter * 32 + lane, n = wt * kWRows + row;
        const ColumnTerms col = column_terms(args, n);
        if constexpr (XT == kKept) {
            if (t < BN) put_row_terms(terms, t, row_terms(args, xt * BN + t));
        } else {
            few_rows<FMT, XT, C>(args, smem, terms, tops, full, empty, kt0, kt1, warp - 2, lane, abort_flag);
        }
        bool ok = mbar_wait_bounded(done, 0, abort_flag, args.flags, args.wait_ns) && !*abort_flag;
        ok = epilogue_agrees(ok);  // the row terms are there too
        tc_fence_after();
        const int rows = min(BN, args.M - xt * BN);
        constexpr int NC = BN == 32 ? 16 : 32;
        if (ok) {
            float* red = reinterpret_cast<float*>(smem);  // idle: every MMA that read the stages is done
#pragma unroll 1
            for (int c = half * (BN / 2); c < min(rows, (half + 1) * (BN / 2)); c += NC) {
                uint32_t r[NC];
                tmem_load<NC>(tmem + uint32_t(c) + (uint32_t(quarter * 32) << 16), r);
                tmem_ld_wait();
                if (S == 1) {
                    emit<OUT, NC>(args, r, col, terms + 2 * c, xt * BN + c, rows - c, n, lane);
                } else {
#pragma unroll
                    for (int j = 0; j < NC; ++j) red[(c + j) * C::LD + row] = __uint_as_float(r[j]);
                }
            }
        }
        tc_fence_before();
    }
    if (S > 1) {
        cluster_sync();  // every thread of every CTA of the cluster, on every path
        if (warp >= 2 && !*abort_flag) {
            const int rows = min(BN, args.M - xt * BN);
            if (S == 2) join_parts<OUT, 2, C::LD>(args, smem_u32(smem), terms, xt * BN, rows, wt * kWRows, sp, warp - 2, lane);
            else if (S == 4) join_parts<OUT, 4, C::LD>(args, smem_u32(smem), terms, xt * BN, rows, wt * kWRows, sp, warp - 2, lane);
            else join_parts<OUT, 8, C::LD>(args, smem_u32(smem), terms, xt * BN, rows, wt * kWRows, sp, warp - 2, lane);
        }
        cluster_sync();  // no CTA leaves while another may still read its shared memory
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// ----------------------------------------------------------------- host side

// Codes [rows][stride bytes], boxes of 128 bytes x `box` rows, 128-byte swizzle; what lies
// outside reads as zeros.
bool codes_map(CUtensorMap* map, const clef_fp4& q, int box) {
    const uint64_t stride = uint64_t(fp4_code_stride(q.cols));
    return make_tma_2d(map, q.codes, 1, stride, uint64_t(q.rows), stride, kAtomBytes, uint32_t(box), true);
}

// Scale groups [groups][512 bytes, as words], boxes of the groups of one K tile.
bool scales_map(CUtensorMap* map, const clef_fp4& q) {
    const uint64_t groups = uint64_t(fp4_row_groups(q.rows)) * uint64_t(fp4_kgroups(q.format, q.cols));
    return make_tma_2d(map, q.scales, 4, kFp4ScaleGroup / 4, groups, kFp4ScaleGroup, kFp4ScaleGroup / 4,
                       uint32_t(groups_of(q.format)), false);
}

// The kernel's shared memory, opted into once for every device.
template <typename K>
cudaError_t set_up(PerDevice<int>* ready, K kernel, int bytes) {
    int device = 0, set = 0;
    const cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    return cudaError_t(ready->get(device, &set, [&](int* v) {
        *v = 1;
        return int(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    }));
}

template <int N, typename K>
cudaError_t launch_clusters(K kernel, int grid, int cluster, int threads, size_t smem, cudaStream_t s,
                            const CUtensorMap (&maps)[N], const Fp4ProductArgs& a) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if constexpr (N == 5) return counted(cudaLaunchKernelEx(&cfg, kernel, maps[0], maps[1], maps[2], maps[3], maps[4], a));
    else return counted(cudaLaunchKernelEx(&cfg, kernel, maps[0], maps[1], maps[2], maps[3], a));
}

// K parts of a tile.  A K tile takes a CTA about 0.29 us, joining the parts 0.5 us for one row and 1.3 to 1.5
// us for more, however many parts; CTAs beyond one an SM gain nothing (4096 x 4096, one row: 6.8, 5.2, 4.2,
// 4.7 us in 1, 2, 4, 8 parts; 4096 x 1024, 32 rows: 3.4, 4.0, 4.3 us in 1, 2, 4), nor do more than 4 parts of
// tiles of 128 rows (1024 x 4096, 256 rows: 6.4 us in 4, 8.6 in 8).
inline int tile_splits(int M, int tiles, int ktiles, int most) {
    const double join = M == 1 ? 0.5 : M <= 32 ? 1.3 : 1.5;
    double best = ktiles * 0.29;
    int splits = 1;
    for (int S = 2; S <= most && S <= ktiles && tiles * S <= num_sms(); S *= 2) {
        const double t = (ktiles + S - 1) / S * 0.29 + join;
        if (t < best) {
            best = t;
            splits = S;
        }
    }
    return splits;
}

// x is read through its maps (kKept) or, in few rows, through a.x.
template <int FMT, int BN, int OUT, int XT>
cudaError_t launch_tile(const clef_fp4* x, const clef_fp4& w, Fp4ProductArgs a, cudaStream_t s) {
    using C = TileCfg<FMT, BN>;
    static PerDevice<int> ready;
    const cudaError_t e = set_up(&ready, fp4_tile_kernel<FMT, BN, OUT, XT>, C::SMEM);
    if (e != cudaSuccess) return e;
    CUtensorMap maps[4];
    if (!codes_map(&maps[0], w, kWRows) || !scales_map(&maps[2], w)) return cudaErrorInvalidValue;
    if constexpr (XT == kKept) {
        if (!codes_map(&maps[1], *x, BN) || !scales_map(&maps[3], *x)) return cudaErrorInvalidValue;
    } else {
        maps[1] = maps[3] = maps[0];  // never used
    }
    const int tiles = (a.N + kWRows - 1) / kWRows * ((a.M + BN - 1) / BN);
    a.splits = tile_splits(a.M, tiles, fp4_ktiles(w.cols), BN == 128 ? 4 : 8);
    return launch_clusters(fp4_tile_kernel<FMT, BN, OUT, XT>, tiles * a.splits, a.splits, kThreads, C::SMEM, s, maps, a);
}

}  // namespace

}  // namespace clef
