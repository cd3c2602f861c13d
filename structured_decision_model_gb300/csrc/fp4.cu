// Rows into microscaled 4-bit form and back.
//
// Quantise.  A row belongs to a half, one or more warps and stays in their registers: its largest
// sizes, its mean and variance and its codes come from one read of memory.  A lane holds 16
// consecutive values of every 512: a block of 16 is one lane's and one of 32 two neighbours', so
// that a scale is worked out once or twice, and the codes' arithmetic runs on pairs (fma.rn.f32x2).
// Memory bounds it, and with statistics issue slots: 131072 x 4096 bf16 takes 206 us to nvfp4 (6.6 TB/s),
// 188 to mxfp4 (7.2 TB/s; a plain copy 6.8), 256 and 216 with statistics, 271 and 228 with sums.  Eight values a lane took 409, 324 and
// 470 (nvfp4 with statistics); rows of a block tied together by block-wide barriers, and indexes by division, 224, 195
// and 306; sums and squares apart, and asked for at run time, 294 with statistics.
#include "fp4.cuh"
#include "kernels.h"

namespace clef {

namespace {

constexpr int kThreads = 256;

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

// The 2^shift warps that share a row, and which row of the block and which of its warps this one is.
struct Share {
    int shift, slot, part;
    __device__ __forceinline__ bool alone() const { return shift == 0; }
};

// Barriers of warps that share a row, so that the block's other rows go their own way; row_any: whether `p` holds
// in one of their threads.
__device__ __forceinline__ void row_sync(const Share& w) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + w.slot), "r"(32 << w.shift) : "memory");
}
__device__ __forceinline__ bool row_any(bool p, const Share& w) {
    int any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.s32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
        "selp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(int(p)), "r"(1 + w.slot), "r"(32 << w.shift)
        : "memory");
    return any != 0;
}

// The largest of a row (a half of a warp is alone).
template <int LANES>
__device__ __forceinline__ float row_max(float v, float* red, const Share& w) {
    v = lanes_max<LANES>(v);
    if (LANES < 32 || w.alone()) return v;
    float* mine = red + (w.slot << w.shift);
    if ((threadIdx.x & 31) == 0) mine[w.part] = v;
    row_sync(w);
    for (int i = 0; i < 1 << w.shift; ++i) v = fmaxf(v, mine[i]);
    return v;
}

// Sums over a row of what its lanes have for each of its pieces: pieces in order, then lanes, so that a sum
// does not depend on how many warps share the row.  One warp (or a half) adds up as it goes; several
// leave what they have in shared memory.
template <int LANES>
struct RowSum {
    float (*all)[32];  // the row's pieces
    float own = 0.f;
    __device__ __forceinline__ void add(float v, const Share& w, int piece, int lane) {
        if (LANES < 32 || w.alone()) own += v;
        else all[piece][lane] = v;
    }
    __device__ __forceinline__ float get(const Share& w, int pieces, int lane) {
        if (LANES == 32 && !w.alone()) {  // behind a barrier
            own = 0.f;
#pragma unroll 4
            for (int i = 0; i < pieces; ++i) own += all[i][lane];
        }
        return lanes_sum<LANES>(own);
    }
};

// Two such sums, side by side; each half of the lanes adds up one of them.
template <int LANES>
struct RowSums {
    uint64_t (*all)[32];
    uint64_t own = 0;
    __device__ __forceinline__ void add(uint64_t v, const Share& w, int piece, int lane) {
        if (LANES < 32 || w.alone()) own = add2(own, v);
        else all[piece][lane] = v;
    }
    __device__ __forceinline__ float2 get(const Share& w, int pieces, int lane) {
        if (LANES == 32 && !w.alone()) {  // behind a barrier
            own = 0;
#pragma unroll 4
            for (int i = 0; i < pieces; ++i) own = add2(own, all[i][lane]);
        }
        const float2 f = both_of(own);
        const bool low = (lane & LANES / 2) == 0;
        float v = (low ? f.x : f.y) + __shfl_xor_sync(0xffffffffu, low ? f.y : f.x, LANES / 2);
#pragma unroll
        for (int o = LANES / 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        const float apart = __shfl_xor_sync(0xffffffffu, v, LANES / 2);
        return low ? make_float2(v, apart) : make_float2(apart, v);
    }
};

// Mean and 1 / sqrt(variance + eps) of a row from its distances, where its first mean and variance (of part 0) want them
// (of two rows in a warp, maybe one does).  `spread` holds the first mean for the warps that share the row; the sums in `all`
// have been read.  Rare and long: kept out of the kernel, which has no register to spare (131072 x 4096 bf16 to nvfp4 with
// statistics: 256 us, 271 with this within it; where every row wants it 413).
template <int DT, bool VEC, int STEPS, int LANES>
__device__ __noinline__ float2 statistics_apart(const void* x, int64_t row0, int cols, float inv_cols, Share w, int lane,
                                                uint64_t (*all)[32], Spread* spread, uint32_t* own, float2 first) {
    const bool shared = LANES == 32 && !w.alone(), far = w.part == 0 && far_from_zero(first.x, first.y);
    const int pieces = (cols + 511) / 512;
    RowSums<LANES> apart{all};
    Spread from = spread_of(first.x, first.y);
    bool wanted = far;  // of the row's first warp
#pragma unroll 1
    for (int turn = 0; turn < 2; ++turn) {
        if (shared) from = *spread;  // behind a barrier
        apart.own = 0;
#pragma unroll 1
        for (int i = 0; i < STEPS; ++i) {
            const int piece = (i << w.shift) + w.part, col0 = piece * 512;
            if (LANES == 32 && col0 >= cols) continue;
            const Raw<DT> again = load16<DT, VEC, LANES>(x, row0, col0, cols, lane, own);
            apart.add(moments_apart<DT>(again, from, cols - (col0 + lane * 16)), w, piece, lane);
        }
        if (shared) row_sync(w);
        if (w.part == 0) {
            const float2 f = apart.get(w, pieces, lane);
            const float rest = f.x * inv_cols, square = f.y * inv_cols;
            if (wanted) {
                first.y = variance_apart(rest, square);
                if (turn == 0) first.x = from.mean = corrected_mean(from, rest);
            }
            wanted = wanted && mostly_rounding(rest, square);
            if (shared && lane == 0) *spread = from;
        }
        if (turn == 0 && !(shared ? row_any(wanted, w) : __any_sync(0xffffffffu, wanted))) break;
    }
    return make_float2(first.x, rstd_of(first.y, from.by));
}

// What else is asked for: the statistics; sums of what is kept, and maybe the statistics.
enum { kNothing, kStats, kSums };

// STEPS: 512-value pieces of a row that a warp keeps, 16 values a lane; W = 2^shift warps a row, so that a row has at
// most 512 * STEPS * W values.  LANES 16: rows of up to 256 values, two a warp.  64 registers a thread, for 32 warps
// an SM: with 8 pieces a warp and half the warps 131072 x 4096 bf16 took 301 us instead of 252.
template <int FMT, int DT, bool VEC, int STEPS, int LANES, int EXTRA>
__global__ void __launch_bounds__(kThreads, DT == CLEF_FP32 && STEPS == 4 ? 2 : 4)
    fp4_quantize_kernel(const Fp4QuantizeArgs a, int shift) {
    constexpr bool NV = FMT == CLEF_NVFP4;
    __shared__ float red[kThreads / 32];
    __shared__ Spread spreads[EXTRA ? kThreads / 32 : 1];
    constexpr int kPieces = kThreads / 32 * STEPS;
    __shared__ uint64_t moments[EXTRA ? kPieces : 1][32];
    __shared__ float totals[EXTRA == kSums ? kPieces : 1][32];
    __shared__ __align__(16) uint32_t stage[VEC ? 1 : kThreads / 32][VEC ? 4 : 32 * Raw<DT>::kWords];
    griddep_wait();
    griddep_launch();  // behind the wait: whoever starts early may take what came before us as done
    static_assert(LANES == 32 || STEPS == 1, "a half of a warp keeps one tile of a row");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x % LANES;
    const Share w{shift, LANES == 32 ? warp >> shift : 0, LANES == 32 ? warp & ((1 << shift) - 1) : 0};
    const uint32_t row = LANES == 32 ? blockIdx.x * uint32_t(kThreads / 32 >> shift) + uint32_t(w.slot)
                                     : blockIdx.x * uint32_t(kThreads / LANES) + threadIdx.x / LANES;
    const bool mine = row < uint32_t(a.rows);  // threads behind the last row still meet their row's barriers and shuffles
    const int part = w.part;
    const int padded = mine ? (a.cols + kFp4Tile - 1) / kFp4Tile * kFp4Tile : 0;  // columns that have scales
    const bool stats = EXTRA == kStats || (EXTRA == kSums && a.mean);  // the same for every thread
    constexpr bool sums = EXTRA == kSums;
    const int64_t row0 = int64_t(row) * a.row_stride;

    Raw<DT> raw[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int col0 = ((i << shift) + part) * 512;
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
        if (NV) row_top = fmaxf(row_top, finite_top<DT>(raw[i], top[i]));
    }
    RowScale rs{1.f, 1.f, false};
    if constexpr (NV) {
        rs = row_scale_of(row_max<LANES>(row_top, red, w));
        if (mine && part == 0 && lane == 0) a.row_scale[row] = rs.r;
    }
    const uint32_t code_stride = uint32_t(a.cols + 31) / 32 * 16;
    uint8_t* codes = a.codes + uint64_t(row) * code_stride;
    uint8_t* scales = a.scales + uint64_t(row / kFp4RowGroup) * uint32_t(padded >> (NV ? 6 : 7)) * kFp4ScaleGroup +
                      (row % 32) * 16 + row % kFp4RowGroup / 32 * 4;
    const int first = EXTRA ? (w.slot << shift) * STEPS : 0;  // of the row's pieces among the block's
    RowSums<LANES> both{moments + first};
    RowSum<LANES> total{totals + (sums ? first : 0)};
    const int pieces = (a.cols + 511) / 512;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        if (LANES == 32 && ((i << shift) + part) * 512 >= padded) continue;  // the same for a whole warp
        const int col = ((i << shift) + part) * 512 + lane * 16;
        const int left = a.cols - col;  // values from the lane's first to the row's end
        uint64_t x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = raw[i].two(j);
        if (stats) both.add(moments16(x), w, (i << shift) + part, lane);
        const Coded c = encode16<FMT, DT>(x, top[i], rs.inv, rs.tiny, left);
        if (mine && col < int(2 * code_stride)) *reinterpret_cast<uint2*>(codes + col / 2) = c.codes;
        uint32_t word;
        if (scale_word<FMT>(c.byte, lane, &word) && col < padded)
            *reinterpret_cast<uint32_t*>(scales + uint32_t(col >> (NV ? 6 : 7)) * kFp4ScaleGroup) = word;
        if (sums) {
            uint32_t h[8];
            unpack_e2m1(c.codes.x, h);
            unpack_e2m1(c.codes.y, h + 4);
            float t = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
                t += f.x + f.y;
            }
            total.add(t * c.scale, w, (i << shift) + part, lane);
        }
    }
    if (stats) {
        // The row's first warp adds up; the others wait for what it finds only where that is far from zero.
        if (LANES == 32 && !w.alone()) row_sync(w);
        float2 found = make_float2(0.f, 0.f);  // mean and variance, then mean and 1 / sqrt(variance + eps)
        if (part == 0) {
            const float2 f = both.get(w, pieces, lane);
            found.x = f.x * a.inv_cols;
            found.y = f.y * a.inv_cols - found.x * found.x;
            if (LANES == 32 && !w.alone() && lane == 0) spreads[warp] = spread_of(found.x, found.y);
        }
        // A mean square less a mean's loses as many bits as the mean exceeds the spread: such rows, and those
        // whose squares pass fp32, are read once or twice more.
        const bool far = mine && part == 0 && far_from_zero(found.x, found.y);
        if (LANES < 32 || w.alone() ? __any_sync(0xffffffffu, far) : row_any(far, w)) {
            uint32_t* own = stage[VEC ? 0 : warp] + (VEC || LANES == 32 ? 0 : (threadIdx.x & 16) * Raw<DT>::kWords);
            found = statistics_apart<DT, VEC, STEPS, LANES>(a.x, mine ? row0 : 0, mine ? a.cols : 0, a.inv_cols, w, lane, both.all,
                                                            &spreads[LANES == 32 ? w.slot << shift : 0], own, found);
        } else {
            found.y = rstd_of(found.y, 1.f);
        }
        if (mine && part == 0 && lane == 0) {
            a.mean[row] = found.x;
            a.rstd[row] = found.y;
        }
    }
    if (sums) {
        if (LANES == 32 && !w.alone()) row_sync(w);
        const float all = part == 0 ? total.get(w, pieces, lane) : 0.f;
        if (mine && part == 0 && lane == 0) a.sums[row] = all * rs.r;
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

template <int FMT, int DT, bool VEC, int EXTRA>
cudaError_t quantize_rows(const Fp4QuantizeArgs& a, cudaStream_t s) {
    // Few rows: as many warps a row as it has pieces, for latency.  Many: as few as hold the row in
    // registers (4 pieces of 16-bit values, 2 of fp32).
    const int pieces = (a.cols + 511) / 512;
    constexpr int kMost = DT == CLEF_FP32 ? 2 : 4;
    const int64_t warps = int64_t(num_sms()) * 16;
    int W = 1, shift = 0;
    for (; W < 8 && W < pieces && (pieces > kMost * W || int64_t(a.rows) * W < warps); ++shift) W *= 2;
    if (a.cols <= 256)
        return launch_pdl(fp4_quantize_kernel<FMT, DT, VEC, 1, 16, EXTRA>, dim3(unsigned((int64_t(a.rows) + 15) / 16)),
                          dim3(kThreads), 0, s, a, 0);
    const int steps = (pieces + W - 1) / W;
    const dim3 grid(unsigned((int64_t(a.rows) * W + kThreads / 32 - 1) / (kThreads / 32)));
    if (steps <= 1) return launch_pdl(fp4_quantize_kernel<FMT, DT, VEC, 1, 32, EXTRA>, grid, dim3(kThreads), 0, s, a, shift);
    if (steps <= 2) return launch_pdl(fp4_quantize_kernel<FMT, DT, VEC, 2, 32, EXTRA>, grid, dim3(kThreads), 0, s, a, shift);
    if (steps <= 4) return launch_pdl(fp4_quantize_kernel<FMT, DT, VEC, 4, 32, EXTRA>, grid, dim3(kThreads), 0, s, a, shift);
    return cudaErrorInvalidValue;
}

template <int FMT, int DT>
cudaError_t quantize_type(const Fp4QuantizeArgs& a, cudaStream_t s) {
    constexpr int size = DT == CLEF_FP32 ? 4 : 2;
    const bool vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.row_stride * size % 16 == 0 && a.cols % 8 == 0;
    if (vec) {
        if (a.sums) return quantize_rows<FMT, DT, true, kSums>(a, s);
        return a.mean ? quantize_rows<FMT, DT, true, kStats>(a, s) : quantize_rows<FMT, DT, true, kNothing>(a, s);
    }
    if (a.sums) return quantize_rows<FMT, DT, false, kSums>(a, s);
    return a.mean ? quantize_rows<FMT, DT, false, kStats>(a, s) : quantize_rows<FMT, DT, false, kNothing>(a, s);
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
