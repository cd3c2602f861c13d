// Attention over the paged 4-bit memory cache for requests of many query rows: options over a
// record's memory, prompts in chunks.  (cache_attend.cu has the few-rows kernel, the formulas
// of the codes and the launch.)
//
// A CTA of four warps takes a split of a request's keys, one key/value head and 64 query rows,
// 16 a warp.  Here the queries are the M dimension, S = Q K^T and O += P V, and most of what the
// codes cost is paid once for 64 rows: in a step of 64 keys each warp turns the values of one
// 16-token piece into fp16 operands in shared memory, in the order in which the lanes take them
// as the B operand, and its keys' scales into fp32; then all four pieces meet all rows.  The key
// codes stay packed and each warp splits them itself (20 instructions a piece, while operands
// of four times the bytes would run into shared memory's rate).  Two buffers: a step's pieces
// are expanded while the step before is multiplied, one barrier a step.
//   Keys stay exact: codes as fp16 subnormals, and scores s_t (q . c_t) + m_t (sum q) in fp32,
// where s_t comes with the scale of the softmax and of the queries' power of two on it.
//   Values are rounded to fp16, (c - 8) s' + m' with s' = s 2^-e and m' = (m + 8 s) 2^-e, where 2^e
// is the size of the token's group: its largest magnitude comes to [1, 2).  The middle m' and
// the value are rounded by half a step of 11 bits each.  The size goes to the weights, p_t 2^e_t,
// which are rounded to 11 bits too, after the row's power of two (move_weights in
// cache_attend.cuh); the denominator sums p_t in fp32.  A token's values and a row's weights
// are thus scaled by themselves, whatever their neighbours hold.
//   fp16 outputs (FINE) keep as many digits as that, so for them the value operand is the centred code
// c - 8, exact; the weights p_t s_t are multiplied in two fp16 parts (22 bits), and the middles' sum
// p_t (m_t + 8 s_t) goes by itself in fp32 (options of 8 records of 16384 rows: 252 us, bf16 193).
// The softmax reference of a row moves only when a score exceeds it by 2^8.
//   64 queries x 8 requests x 16384 keys x 16 heads of 64: 193 us with the merge, 178 TFLOP/s.
// What bounds it: the instructions around the products (about 197 for 16 keys x 16 rows, 16 of
// them matrix instructions) at half of the issue slots; the matrix pipe is 35 % busy, shared
// memory 57 %.  Scaling each token's values by itself costs 20 of them and 10 us.  Before that, at
// 183 us, these were tried and slower: 32 rows a warp (265 us, out of registers), key operands
// expanded in shared memory (188), products of two or four pieces side by side (same), the next
// item requested ahead (191, out of registers).
#include "cache_attend.cuh"

namespace clef {

namespace {

constexpr int kRowsItem = 16 * kAttendWarps;  // query rows of an item
constexpr int kRowsStep = 16 * kAttendWarps;  // keys of a step

// Of an expanded piece: the tokens whose values are no numbers (a bit each, by group of 64
// values), and whether it is there at all.
struct PieceInfo {
    int bad0, bad1, absent;
};

template <int G, bool FINE>
struct RowsSmem {
    static constexpr int kStages = 3;                               // raw pieces a warp
    static constexpr int kRaw = kAttendWarps * kStages * kPiece * G;
    // an expanded piece: key codes, values in fp16, scale and minimum of its keys and the sizes of its
    // values in fp32
    static constexpr int kValuesAt = 512 * G;
    static constexpr int kScalesAt = kValuesAt + 2048 * G;
    static constexpr int kSizesAt = kScalesAt + 16 * 8 * G;
    static constexpr int kMiddlesAt = kSizesAt + 16 * 4 * G;  // FINE
    static constexpr int kExpanded = kMiddlesAt + (FINE ? 16 * 4 * G : 0);
    static constexpr int kBytes = kRaw + 2 * kAttendWarps * kExpanded;
};

__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
    const __half2 d = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                              *reinterpret_cast<const __half2*>(&c));
    return *reinterpret_cast<const uint32_t*>(&d);
}

}  // namespace

template <int G, bool FINE>
__global__ void __launch_bounds__(kAttendThreads, G == 1 ? (FINE ? 3 : 4) : 2) cache_attend_rows_kernel(const CacheAttendArgs a) {
    using Smem = RowsSmem<G, FINE>;
    constexpr int ST = Smem::kStages;
    constexpr int kBytes = kPiece * G;
    constexpr int kMaxPages = kAttendMaxChunk / 16;
    griddep_wait();
    griddep_launch();
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t* expanded = smem + Smem::kRaw;  // [buffer][piece]{keys, values, scales}
    const Requests s_req(reinterpret_cast<int*>(smem + Smem::kBytes), a.B);
    __shared__ const uint8_t* s_page[kMaxPages];
    __shared__ PieceInfo s_info[2][kAttendWarps];
    __shared__ int s_exp[kAttendWarps];
    __shared__ Item s_item;
    const int n_items = scan_requests<G, true>(a, s_req, kRowsItem);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, tq = lane & 3;
    const int page_mask = a.c.page - 1;
    uint8_t* raw = smem + warp * (ST * kBytes);

    for (int turn = 0; item_of_turn(turn) < n_items; ++turn) {
        __syncthreads();  // nothing of the item before this one is needed any more
        if (threadIdx.x == 0) s_item = item_of<kRowsItem>(a, s_req, item_of_turn(turn));
        __syncthreads();
        const Item& me = s_item;
        const int t0 = me.t0, t1 = me.t1, ahead = me.ahead;
        // ---- the split's pages, and the queries of the warp's rows g and g + 8
        for (int i = threadIdx.x; i < kMaxPages; i += kAttendThreads) {
            const uint8_t* at = nullptr;
            if ((int64_t(me.p0 + i) << a.c.page_shift) < t1) {
                const int id = a.table[int64_t(me.b) * a.width + me.p0 + i];
                if (id < 0 || id >= a.c.n_pages)
                    atomicOr(a.flags, kFlagBounds);
                else
                    at = a.c.data + ((int64_t(id) * a.c.heads + a.head0 + me.h) << (a.c.page_shift - 4)) * kBytes;
            }
            s_page[i] = at;
        }
        uint32_t qw[2][G][8];
        float top[2], qsum[2][G];
        const int r0 = warp * 16 + g;  // the lane's rows of the item: r0 and r0 + 8
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const bool live = r0 + 8 * r < me.rows;
            const int row = live ? me.row0 + r0 + 8 * r : 0, qi = a.by_share(row), qh = me.h * a.share + row - qi * a.share;
            const uint16_t* q = static_cast<const uint16_t*>(a.q) + (s_req.q0[me.b] + qi) * a.q_row + qh * a.q_head + 2 * tq;
            top[r] = 0.f;
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    qw[r][gr][i] = live ? __ldg(reinterpret_cast<const uint32_t*>(q + gr * 64 + i * 8)) : 0u;
                    const float2 x = unpack2(qw[r][gr][i], a.dtype);
                    sum += x.x + x.y;
                    top[r] = fmaxf(top[r], fmaxf(fabsf(x.x), fabsf(x.y)));
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                qsum[r][gr] = sum;
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], o));
        }
        // One power of two for all rows of the item puts the largest value in [2^14, 2^15); rows
        // that are far smaller (or no numbers) are scaled by themselves, and their scores by
        // what is between.
        int e[2], least = 1000;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int field = int(__float_as_uint(top[r]) >> 23);
            e[r] = top[r] > 0.f ? min(14 - (field - 127), 120) : 120;
            if (top[r] > 0.f && field < 255) least = min(least, e[r]);
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
        if (lane == 0) s_exp[warp] = least;
        __syncthreads();
        int common = 1000;
#pragma unroll
        for (int i = 0; i < kAttendWarps; ++i) common = min(common, s_exp[i]);
        if (common == 1000) common = 0;
        float rowmul[2];
        bool apart = false;
        uint32_t qa[G][4][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const bool own = top[r] > 0.f && (e[r] - common > 10 || e[r] < common);
            const int mine = own ? e[r] : common;
            rowmul[r] = pow2i(common - mine);
            apart |= own;
            const float up = pow2i(mine);
#pragma unroll
            for (int gr = 0; gr < G; ++gr)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float f = (i & 1) ? up * 0.0625f : up;
                    const float2 x = unpack2(qw[r][gr][i], a.dtype);
                    qa[gr][i >> 1][(i & 1) * 2 + r] = pack_f16(x.x * f, x.y * f);
                }
        }
        apart = __any_sync(0xffffffffu, apart);
        const float score_mul = a.scale_log2 * pow2i(24 - common);

        float acc[G][8][4];  // O: rows g (0, 1) and g + 8 (2, 3), values 8 n + 2 tq, + 1
        float l[2] = {0.f, 0.f}, ref[2] = {0.f, 0.f}, none[2][G];
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
            none[0][gr] = none[1][gr] = 0.f;
#pragma unroll
            for (int n = 0; n < 8; ++n) acc[gr][n][0] = acc[gr][n][1] = acc[gr][n][2] = acc[gr][n][3] = 0.f;
        }
        float mul[2][G];  // the weights' powers of two
        float z[2][G];    // FINE: sum of p (m + 8 s)
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
            mul[0][gr] = mul[1][gr] = 1.f;
            z[0][gr] = z[1][gr] = 0.f;
        }
        bool first = true;

        auto page_at = [&](int t) { return t < t1 ? s_page[(t >> a.c.page_shift) - me.p0] : nullptr; };
        auto request = [&](int t, int stage) {  // the warp's piece of the step at t
            const uint8_t* page = page_at(t + 16 * warp);
            if (page) {
                const uint8_t* src = page + (((t + 16 * warp) & page_mask) >> 4) * kBytes + lane * 16;
                uint8_t* dst = raw + stage * kBytes + lane * 16;
#pragma unroll
                for (int i = 0; i < kBytes; i += 512)
                    if (i + lane * 16 < kBytes) cp_async16(dst + i, src + i, true);
            }
            cp_async_commit();
        };
        // The warp's raw piece of the step at t becomes operands in buffer `buf`.
        auto expand = [&](int t, int stage, int buf) {
            const int tk = t + 16 * warp;
            const uint8_t* src = raw + stage * kBytes;
            uint8_t* dst = expanded + (buf * kAttendWarps + warp) * Smem::kExpanded;
            const bool there = page_at(tk) != nullptr;
            // scales: lane i looks after key i (lane i + 16 too)
            const int key = lane & 15;
            const bool real = there && tk + key < t1;
            float vs[G], vm[G], up[G];
            uint32_t bad[2] = {0u, 0u};
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                uint2 sm = *reinterpret_cast<const uint2*>(src + G * 1024 + (key * G + gr) * 8);
                if (!real) sm = make_uint2(0u, 0u);
                if (lane < 16)
                    *reinterpret_cast<float2*>(dst + Smem::kScalesAt + (gr * 16 + key) * 8) =
                        make_float2(bf16_lo(sm.x) * score_mul, bf16_hi(sm.x) * a.scale_log2);
                vs[gr] = bf16_lo(sm.y);
                vm[gr] = bf16_hi(sm.y);
                const bool odd = !(fabsf(vs[gr]) < INFINITY && fabsf(vm[gr]) < INFINITY);
                bad[gr] = __ballot_sync(0xffffffffu, odd) & 0xffffu;
                if (odd) vs[gr] = vm[gr] = 0.f;
                if (FINE) {
                    // the size is the scale itself (2^119 and more gives no fp16 number), the middle goes by itself
                    if (lane < 16) {
                        *reinterpret_cast<float*>(dst + Smem::kSizesAt + (gr * 16 + key) * 4) = fminf(vs[gr], 0x1p119f);
                        *reinterpret_cast<float*>(dst + Smem::kMiddlesAt + (gr * 16 + key) * 4) = fmaf(8.f, vs[gr], vm[gr]);
                    }
                    continue;
                }
                // 2^e, the size of the token's values: its largest is put in [1, 2)
                const int e = min(max(exponent_of(fmaxf(fabsf(vm[gr]), fabsf(fmaf(15.f, vs[gr], vm[gr])))), -126), 119);
                up[gr] = pow2i(-e);
                if (lane < 16)
                    *reinterpret_cast<float*>(dst + Smem::kSizesAt + (gr * 16 + key) * 4) =
                        vs[gr] == 0.f && vm[gr] == 0.f ? 0.f : pow2i(e);
            }
            if (lane == 0) s_info[buf][warp] = PieceInfo{int(bad[0]), int(bad[1]), there ? 0 : 1};
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                const uint4 kw = reinterpret_cast<const uint4*>(src + gr * 512)[lane];
                const uint4 vw = reinterpret_cast<const uint4*>(src + (G + gr) * 512)[lane];
                const uint32_t vws[4] = {vw.x, vw.y, vw.z, vw.w};
                // value scale and middle of the lane's key, then those of keys 2 tq, 2 tq + 1 (low,
                // high half) and of both + 8
                const uint32_t own = FINE ? 0u : pack_f16(vs[gr] * up[gr], fmaf(8.f, vs[gr], vm[gr]) * up[gr]);
                uint32_t s2[2], m2[2];
#pragma unroll
                for (int h = 0; h < (FINE ? 0 : 2); ++h) {
                    const uint32_t x = __shfl_sync(0xffffffffu, own, 8 * h + 2 * tq);
                    const uint32_t y = __shfl_sync(0xffffffffu, own, 8 * h + 2 * tq + 1);
                    s2[h] = __byte_perm(x, y, 0x5410);
                    m2[h] = __byte_perm(x, y, 0x7632);
                }
                reinterpret_cast<uint4*>(dst + gr * 512)[lane] = kw;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t x = vws[i], y = x >> 8;
                    // c - 8 of keys 2 tq, 2 tq + 1, and of both + 8: values d, then d + 8
                    uint32_t a0 = centred_low(x);
                    uint32_t a1 = centred_high(x);
                    uint32_t a2 = centred_low(y);
                    uint32_t a3 = centred_high(y);
                    if (!FINE) {
                        a0 = fma_f16x2(a0, s2[0], m2[0]);
                        a1 = fma_f16x2(a1, s2[0], m2[0]);
                        a2 = fma_f16x2(a2, s2[1], m2[1]);
                        a3 = fma_f16x2(a3, s2[1], m2[1]);
                    }
                    reinterpret_cast<uint4*>(dst + Smem::kValuesAt + gr * 2048)[i * 32 + lane] = make_uint4(a0, a2, a1, a3);
                }
            }
        };
        const int see0 = ahead + a.by_share(me.row0 + r0) + 1, see1 = ahead + a.by_share(me.row0 + r0 + 8) + 1;
        const int full = a.causal ? ahead + a.by_share(me.row0) + 1 : t1;  // keys that every row sees

        // The step at t, expanded in buffer `buf`, meets the warp's rows.
        auto multiply = [&](int t, int buf) {
            const uint8_t* base = expanded + buf * kAttendWarps * Smem::kExpanded;
            float p[kAttendWarps][2][4];  // piece, keys 0-7 / 8-15: (row g: key 2 tq, + 1; row g + 8: the same)
            bool odd = t + kRowsStep > t1 || t + kRowsStep > full;
#pragma unroll
            for (int i = 0; i < kAttendWarps; ++i) {
                const PieceInfo info = s_info[buf][i];
                odd |= (info.bad0 | info.bad1 | info.absent) != 0;
            }
            // of keys 2 tq and 2 tq + 1 (n = 1: + 8) of piece i: the sizes of their values, their middles
            auto pair_at = [&](int i, int at, int gr, int n) {
                return *reinterpret_cast<const float2*>(base + i * Smem::kExpanded + at + (gr * 16 + n * 8 + 2 * tq) * 4);
            };
            auto sizes_of = [&](int i, int gr, int n) { return pair_at(i, Smem::kSizesAt, gr, n); };
            float most = -INFINITY;
#pragma unroll
            for (int i = 0; i < kAttendWarps; ++i) {
                const uint8_t* piece = base + i * Smem::kExpanded;
                float s[G][2][4];
#pragma unroll
                for (int gr = 0; gr < G; ++gr) {
                    const uint4 kq = reinterpret_cast<const uint4*>(piece + gr * 512)[lane];
                    const uint32_t words[4] = {kq.x, kq.y, kq.z, kq.w};
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint32_t x = words[ks], y = x >> 8;
                        if (ks == 0) {
                            mma_f16_16816_first(s[gr][0], qa[gr][ks], x & 0x000F000Fu, x & 0x00F000F0u);
                            mma_f16_16816_first(s[gr][1], qa[gr][ks], y & 0x000F000Fu, y & 0x00F000F0u);
                        } else {
                            mma_f16_16816(s[gr][0], qa[gr][ks], x & 0x000F000Fu, x & 0x00F000F0u);
                            mma_f16_16816(s[gr][1], qa[gr][ks], y & 0x000F000Fu, y & 0x00F000F0u);
                        }
                    }
                }
                if (apart) {
#pragma unroll
                    for (int gr = 0; gr < G; ++gr)
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int c = 0; c < 4; ++c) s[gr][n][c] *= rowmul[c >> 1];
                }
#pragma unroll
                for (int n = 0; n < 2; ++n) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) p[i][n][c] = -ref[c >> 1];
#pragma unroll
                    for (int gr = 0; gr < G; ++gr) {
                        // {scale, minimum} of keys 2 tq and 2 tq + 1
                        const float4 k =
                            *reinterpret_cast<const float4*>(piece + Smem::kScalesAt + (gr * 16 + n * 8 + 2 * tq) * 8);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            p[i][n][c] = fmaf(s[gr][n][c], (c & 1) ? k.z : k.x,
                                              fmaf(qsum[c >> 1][gr], (c & 1) ? k.w : k.y, p[i][n][c]));
                    }
                    most = fmax3(most, p[i][n][0], p[i][n][1]);
                    most = fmax3(most, p[i][n][2], p[i][n][3]);
                }
            }
            if (odd) {  // keys that are not there or that a causal row does not see, values that are no numbers
                most = -INFINITY;
                bool any = false;
#pragma unroll
                for (int i = 0; i < kAttendWarps; ++i) {
                    const PieceInfo info = s_info[buf][i];
                    const int end = info.absent ? 0 : t1;
                    any |= !info.absent;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int key = n * 8 + 2 * tq + (c & 1), at = t + 16 * i + key;
                            const int sees = a.causal ? min(end, c < 2 ? see0 : see1) : end;
                            if (at >= sees) {
                                p[i][n][c] = -INFINITY;
                            } else {
                                if (info.bad0 >> key & 1) none[c >> 1][0] = NAN;
                                if (G == 2 && (info.bad1 >> key & 1)) none[c >> 1][G - 1] = NAN;
                            }
                            most = fmaxf(most, p[i][n][c]);
                        }
                }
                if (first && !any) return;  // nothing there: the references are still to be set
            }
            if (__any_sync(0xffffffffu, first || most > 8.f)) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int i = 0; i < kAttendWarps; ++i)
#pragma unroll
                        for (int n = 0; n < 2; ++n) mx = fmax3(mx, p[i][n][2 * r], p[i][n][2 * r + 1]);
#pragma unroll
                    for (int o = 1; o < 4; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    // mx is relative to the reference (0 in the first step, whatever is seen)
                    const bool moved = first ? mx > -INFINITY : mx > 8.f;
                    Decay d;
                    if (moved) {
                        if (!first) d.set(mx);
                        ref[r] += mx;
                        l[r] *= d.corr;
#pragma unroll
                        for (int i = 0; i < kAttendWarps; ++i)
#pragma unroll
                            for (int n = 0; n < 2; ++n) {
                                p[i][n][2 * r] -= mx;
                                p[i][n][2 * r + 1] -= mx;
                            }
                    }
#pragma unroll
                    for (int gr = 0; gr < G; ++gr) {
                        float x = 0.f, big = 0.f;
#pragma unroll
                        for (int i = 0; i < kAttendWarps; ++i)
#pragma unroll
                            for (int n = 0; n < 2; ++n) {
                                const float2 f = sizes_of(i, gr, n);
                                x = fmax3(x, ex2_approx(p[i][n][2 * r]) * f.x, ex2_approx(p[i][n][2 * r + 1]) * f.y);
                            }
#pragma unroll
                        for (int n = 0; n < 8; ++n)
                            big = fmax3(big, fabsf(acc[gr][n][2 * r]), fabsf(acc[gr][n][2 * r + 1]));
#pragma unroll
                        for (int o = 1; o < 4; o <<= 1) {
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                        }
                        if (moved) {
                            const float f = move_weights(mul[r][gr], x, big, d);
                            if (FINE) z[r][gr] *= d.corr;
#pragma unroll
                            for (int n = 0; n < 8; ++n) {
                                acc[gr][n][2 * r] *= f;
                                acc[gr][n][2 * r + 1] *= f;
                            }
                        }
                    }
                }
                first = false;
            }
#pragma unroll
            for (int i = 0; i < kAttendWarps; ++i)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        p[i][n][c] = ex2_approx(p[i][n][c]);
                        l[c >> 1] += p[i][n][c];
                    }
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                float w[kAttendWarps][2][4], x[2] = {0.f, 0.f};  // weights, still without the row's factor
#pragma unroll
                for (int i = 0; i < kAttendWarps; ++i)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const float2 f = sizes_of(i, gr, n);
#pragma unroll
                        for (int c = 0; c < 4; ++c) w[i][n][c] = p[i][n][c] * ((c & 1) ? f.y : f.x);
                        if (FINE) {
                            const float2 m = pair_at(i, Smem::kMiddlesAt, gr, n);
#pragma unroll
                            for (int c = 0; c < 4; ++c) z[c >> 1][gr] = fmaf(p[i][n][c], (c & 1) ? m.y : m.x, z[c >> 1][gr]);
                        }
                        x[0] = fmax3(x[0], w[i][n][0], w[i][n][1]);
                        x[1] = fmax3(x[1], w[i][n][2], w[i][n][3]);
                    }
                // larger values than the rows have used before
                if (__any_sync(0xffffffffu, fmaxf(x[0] * mul[0][gr], x[1] * mul[1][gr]) > kMostWeight)) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
#pragma unroll
                        for (int o = 1; o < 4; o <<= 1) x[r] = fmaxf(x[r], __shfl_xor_sync(0xffffffffu, x[r], o));
                        if (x[r] * mul[r][gr] > kMostWeight) {
                            const float f = move_weights(mul[r][gr], x[r], 0.f, Decay());
#pragma unroll
                            for (int n = 0; n < 8; ++n) {
                                acc[gr][n][2 * r] *= f;
                                acc[gr][n][2 * r + 1] *= f;
                            }
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < kAttendWarps; ++i) {
                    uint32_t pa[4], pl[4];  // FINE: pl holds what rounding left of pa
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float w0 = w[i][n][2 * r] * mul[r][gr], w1 = w[i][n][2 * r + 1] * mul[r][gr];
                            pa[2 * n + r] = pack_f16(w0, w1);
                            if (FINE) pl[2 * n + r] = rest_f16(pa[2 * n + r], w0, w1);
                        }
                    const uint8_t* values = base + i * Smem::kExpanded + Smem::kValuesAt + gr * 2048;
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt) {
                        const uint4 f = reinterpret_cast<const uint4*>(values)[mt * 32 + lane];
                        mma_f16_16816(acc[gr][2 * mt], pa, f.x, f.y);
                        mma_f16_16816(acc[gr][2 * mt + 1], pa, f.z, f.w);
                        if (FINE) {
                            mma_f16_16816(acc[gr][2 * mt], pl, f.x, f.y);
                            mma_f16_16816(acc[gr][2 * mt + 1], pl, f.z, f.w);
                        }
                    }
                }
            }
        };

#pragma unroll
        for (int s = 0; s < ST - 1; ++s) request(t0 + s * kRowsStep, s);
        cp_async_wait<ST - 2>();
        __syncwarp();
        expand(t0, 0, 0);
        __syncthreads();
        const bool busy = warp * 16 < me.rows;  // the warp has rows
        int stage = 0, buf = 0;
        for (int t = t0; t < t1; t += kRowsStep) {
            // the raw piece at `stage` has been expanded; the one after it is about to be
            const int next = stage == ST - 1 ? 0 : stage + 1, free_stage = stage == 0 ? ST - 1 : stage - 1;
            request(t + (ST - 1) * kRowsStep, free_stage);
            cp_async_wait<ST - 2>();
            __syncwarp();
            if (t + kRowsStep < t1) expand(t + kRowsStep, next, buf ^ 1);
            if (busy) multiply(t, buf);
            __syncthreads();
            stage = next;
            buf ^= 1;
        }
        cp_async_wait<0>();

        // ---- the warp's rows: normalised, with the logarithm (base 2) of the sum
        const bool whole = s_req.len[me.b] <= a.chunk;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float sum = l[r];
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
            for (int gr = 0; gr < G; ++gr)
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    none[r][gr] += __shfl_xor_sync(0xffffffffu, none[r][gr], o);
                    if (FINE) z[r][gr] += __shfl_xor_sync(0xffffffffu, z[r][gr], o);
                }
            const int rr = r0 + 8 * r;
            if (rr >= me.rows) continue;
            const int qi = a.by_share(me.row0 + rr), qh = me.h * a.share + me.row0 + rr - qi * a.share;
            const int64_t row = whole ? int64_t(s_req.q0[me.b] + qi) * a.q_heads + qh
                                      : (me.b ? s_req.parts[me.b - 1] : 0) +
                                            (int64_t(me.split) * s_req.nq[me.b] + qi) * a.q_heads + qh;
            // (query rows of requests that overlap, which cu_q must not have, could make more
            // partial rows than the workspace holds)
            if (!whole && (row < 0 || row >= a.part_rows)) {
                if (tq == 0) atomicOr(a.flags, kFlagBounds);
                continue;
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            if (tq == 0) {
                const float lse2 = sum == 0.f ? -INFINITY : ref[r] + log2f(sum);
                if (!whole)
                    a.part_lse[row] = lse2;
                else if (a.lse)
                    a.lse[row] = lse2 * 0.6931471805599453f;
            }
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                const float back = 1.f / mul[r][gr];
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const float x = fmaf(fmaf(acc[gr][n][2 * r], back, z[r][gr]), inv, none[r][gr]);
                    const float y = fmaf(fmaf(acc[gr][n][2 * r + 1], back, z[r][gr]), inv, none[r][gr]);
                    const int64_t at = row * (64 * G) + gr * 64 + n * 8 + 2 * tq;
                    if (!whole)
                        *reinterpret_cast<float2*>(a.part_o + at) = make_float2(x, y);
                    else
                        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at) =
                            a.dtype == 0 ? pack_bf16(x, y) : pack_f16(x, y);
                }
            }
        }
    }
}

namespace {

template <int G, bool FINE>
cudaError_t launch_rows(const CacheAttendArgs& a, cudaStream_t s) {
    constexpr int kBytes = RowsSmem<G, FINE>::kBytes, kEach = Requests::kInts * 4;
    static PerDevice<int> state;
    int ctas = 0;
    const cudaError_t e =
        resident_ctas(state, cache_attend_rows_kernel<G, FINE>, kBytes + kCacheMaxRequests * kEach, kBytes + 64 * kEach, &ctas);
    if (e != cudaSuccess) return e;
    return launch_pdl(cache_attend_rows_kernel<G, FINE>, dim3(unsigned(ctas)), dim3(kAttendThreads), size_t(kBytes + a.B * kEach), s, a);
}

}  // namespace

cudaError_t launch_cache_attend_rows(const CacheAttendArgs& a, cudaStream_t s) {
    if (a.dtype == 1) return a.c.groups == 1 ? launch_rows<1, true>(a, s) : launch_rows<2, true>(a, s);
    return a.c.groups == 1 ? launch_rows<1, false>(a, s) : launch_rows<2, false>(a, s);
}

}  // namespace clef
