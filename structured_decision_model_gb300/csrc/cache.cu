// Kernels of the paged 4-bit memory cache: page accounts, store, read back.  The stored
// form and its byte layout are described in clef_cache.h.
#include "cache.h"
#include "common.cuh"
#include "kernels.h"

namespace clef {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanFused = 8 * kPlanThreads;  // slots that the plan kernel itself fills

// Inclusive sum over the block's threads (1024), in thread order; `tmp` holds 32 values.
__device__ __forceinline__ int block_scan(int x, int* tmp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // tmp may still be read by the previous scan
    if (lane == 31) tmp[warp] = x;
    __syncthreads();
    int t = tmp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += y;
    }
    const int before = __shfl_sync(0xffffffffu, t, warp > 0 ? warp - 1 : 0);
    return x + (warp > 0 ? before : 0);
}

// Number of entries of the non-decreasing `ends` (n of them) that are <= i.
__device__ __forceinline__ int upper(const int* ends, int n, int i) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] <= i)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

// Slots of gained tokens [first, end) in steps of `step`; `cu` holds the B + 1 running sums
// and `lengths` the new lengths, so that token t of request b is at position
// lengths[b] - (cu[b + 1] - cu[b]) + t - cu[b].
__device__ __forceinline__ void fill_slots(const CachePlanArgs& a, const int* cu, int first, int end, int step) {
    const int total = cu[a.B];
    for (int t = first; t < end; t += step) {
        int slot = -1;
        if (t < total) {
            const int b = min(upper(cu + 1, a.B, t), a.B - 1);
            const int pos = a.lengths[b] - cu[b + 1] + t;
            const int col = pos >> a.page_shift;
            const int id = pos >= 0 && col < a.width ? a.table[int64_t(b) * a.width + col] : -1;
            if (id < 0 || id >= a.n_pages)
                atomicOr(a.flags, kFlagBounds);
            else
                slot = (id << a.page_shift) | (pos & ((1 << a.page_shift) - 1));
        }
        a.slots[t] = slot;
    }
}

}  // namespace

// One CTA, one thread a request: what each request gives back and needs, three scans over
// the requests, then the page moves spread evenly over the threads (a search in the scans
// finds the request of each page).  Bound by its chain of dependent steps, not by bytes.
__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const CachePlanArgs a, int fill) {
    griddep_wait();
    griddep_launch();
    __shared__ int tmp[32];
    __shared__ int s_rel[kPlanThreads], s_more[kPlanThreads], s_have[kPlanThreads], s_cu[kPlanThreads + 1];
    __shared__ int s_grant;
    const int t = threadIdx.x;
    const int page = 1 << a.page_shift;
    const int64_t cap = int64_t(a.width) << a.page_shift;
    int old = 0, want = 0, have = 0, need = 0;
    if (t < a.B) {
        old = a.lengths[t];
        want = a.want[t];
        const bool bad_old = old < 0 || old > cap;
        if (bad_old || want < 0 || want > cap) {
            atomicOr(a.flags, kFlagBounds);
            want = old;  // left as it is
        }
        if (!bad_old) {
            have = int((int64_t(old) + page - 1) >> a.page_shift);
            need = int((int64_t(want) + page - 1) >> a.page_shift);
        }
    }
    int count = *a.free_count;
    if (count < 0 || count > a.n_pages) {
        if (t == 0) atomicOr(a.flags, kFlagBounds);
        count = count < 0 ? 0 : a.n_pages;
    }
    const int rel = max(have - need, 0), more = max(need - have, 0);
    const int rel_end = block_scan(rel, tmp);
    const int more_end = block_scan(more, tmp);
    s_rel[t] = rel_end;
    s_more[t] = more_end;
    s_have[t] = have;
    __syncthreads();
    const int n_rel = s_rel[kPlanThreads - 1];
    // give back: ascending index i of (request, page) pairs; the stack takes them in descending order
    for (int i = t; i < n_rel; i += kPlanThreads) {
        const int b = upper(s_rel, a.B, i);
        const int last = s_have[b] - 1, j = s_rel[b] - 1 - i;  // j-th page from the request's end
        const int64_t at = int64_t(b) * a.width + last - j;
        const int pos = count + n_rel - 1 - i;
        const int id = a.table[at];
        a.table[at] = -1;
        if (pos < a.n_pages)
            a.free_pages[pos] = id;
        else
            atomicOr(a.flags, kFlagBounds);  // more pages came back than there are
    }
    const int top = min(count + n_rel, a.n_pages);
    const bool fits = more == 0 || more_end <= top;
    if (t == 0) s_grant = 0;
    __syncthreads();
    if (fits && more > 0) atomicMax(&s_grant, more_end);
    const int gain_end = block_scan(fits ? max(want - old, 0) : 0, tmp);
    s_cu[t + 1] = gain_end;
    if (t == 0) s_cu[0] = 0;
    __syncthreads();
    const int grant = s_grant;  // requests fit in order, so the granted pages are the first ones
    for (int i = t; i < grant; i += kPlanThreads) {
        const int b = upper(s_more, a.B, i);
        const int first = b > 0 ? s_more[b - 1] : 0;
        const int pos = top - 1 - i;
        a.table[int64_t(b) * a.width + s_have[b] + i - first] = a.free_pages[pos];
        a.free_pages[pos] = -1;
    }
    if (t < a.B) {
        if (fits)
            a.lengths[t] = want;
        else
            atomicOr(a.flags, kFlagPages);
    }
    if (t <= a.B) a.cu[t] = s_cu[t];
    if (t == 0) {
        if (a.B == kPlanThreads) a.cu[a.B] = s_cu[a.B];
        *a.free_count = top - grant;
        if (s_cu[a.B] > a.n_slots) atomicOr(a.flags, kFlagBounds);
    }
    if (fill) {
        __syncthreads();
        fill_slots(a, s_cu, t, a.n_slots, kPlanThreads);
    }
}

// Slots of a large step, after the plan kernel.
__global__ void __launch_bounds__(256) cache_slots_kernel(const CachePlanArgs a) {
    griddep_wait();
    griddep_launch();
    __shared__ int s_cu[kCacheMaxRequests + 1];
    for (int i = threadIdx.x; i <= a.B; i += 256) s_cu[i] = a.cu[i];
    __syncthreads();
    const int64_t first = int64_t(blockIdx.x) * 1024;
    fill_slots(a, s_cu, int(first) + threadIdx.x, int(min(int64_t(a.n_slots), first + 1024)), 256);
}

cudaError_t launch_cache_plan(const CachePlanArgs& a, cudaStream_t s) {
    const bool fused = a.n_slots <= kPlanFused;
    cudaError_t e = launch_pdl(cache_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a, fused ? 1 : 0);
    if (e != cudaSuccess || fused) return e;
    return launch_pdl(cache_slots_kernel, dim3(unsigned((a.n_slots + 1023) / 1024)), dim3(256), 0, s, a);
}

// ------------------------------------------------------------------- rows
//
// A warp takes 16 consecutive rows of one head.  Four lanes hold the 64 values of a row's
// group, 16 each (lane / 4 is the row of eight, lane % 4 the run of 16 values): a lane owns
// the eight code bytes of its run, and a row's minimum and maximum cost two exchanges.

namespace {

constexpr int kRowsWarps = 8;

// Byte j of a token's 32 code bytes (one group) inside the 512 bytes of a 16-token piece.
__device__ __forceinline__ int key_byte(int r, int j) {
    return (r & 7) * 64 + (j & 7) / 2 * 16 + (j >> 3) * 4 + (j & 1) * 2 + (r >> 3);
}
__device__ __forceinline__ int value_byte(int r, int j) {
    return (j & 7) * 64 + (r & 7) / 2 * 16 + (j >> 3) * 4 + (r & 1) * 2 + (r >> 3);
}

// Start of the piece that holds a slot, for cache head `head`.
__device__ __forceinline__ uint8_t* piece_of(const CacheView& c, int slot, int head) {
    return c.data + (((int64_t(slot >> c.page_shift) * c.heads + head) << (c.page_shift - 4)) +
                     ((slot & (c.page - 1)) >> 4)) * (kPiece * c.groups);
}

// The slots around a warp's rows i0 .. i0 + 15: bit p of a mask stands for row i0 - 16 + p.
struct Window {
    uint64_t runs;   // rows that start 16 consecutive slots filling a piece
    uint32_t alone;  // rows of the window (bit k: row i0 + k) with a slot of their own outside such a run
    int slot;        // of row i0 + (lane & 15), negative where there is none
};

__device__ __forceinline__ Window window_of(const int32_t* slots, int64_t i0, int n, int total, int32_t* flags) {
    const int lane = threadIdx.x & 31;
    const int64_t ia = i0 - 16 + lane, ib = i0 + 16 + lane;
    int sa = ia >= 0 && ia < n ? slots[ia] : -2;
    int sb = lane < 15 && ib < n ? slots[ib] : -2;
    if (sa >= total) {  // (the row's own warp reports it)
        if (lane >= 16) atomicOr(flags, kFlagBounds);
        sa = -2;
    }
    if (sb >= total) sb = -2;
    int after_a = __shfl_down_sync(0xffffffffu, sa, 1);
    const int first_b = __shfl_sync(0xffffffffu, sb, 0);
    if (lane == 31) after_a = first_b;
    const int after_b = __shfl_down_sync(0xffffffffu, sb, 1);
    const uint32_t ma = __ballot_sync(0xffffffffu, sa >= 0 && after_a == sa + 1);
    const uint32_t mb = __ballot_sync(0xffffffffu, sb >= 0 && lane < 14 && after_b == sb + 1);
    const uint32_t za = __ballot_sync(0xffffffffu, sa >= 0 && (sa & 15) == 0);
    uint64_t m = ma | uint64_t(mb) << 32;  // bit p: the next row has the next slot
    m &= m >> 1;
    m &= m >> 2;
    m &= m >> 4;
    m &= m >> 7;  // 15 in a row
    Window w;
    w.runs = m & za;
    uint64_t c = w.runs;
    c |= c << 1;
    c |= c << 2;
    c |= c << 4;
    c |= c << 8;  // every row of a run
    const uint32_t live = __ballot_sync(0xffffffffu, sa >= 0);
    w.alone = (live >> 16) & ~uint32_t(c >> 16) & 0xffffu;
    w.slot = __shfl_sync(0xffffffffu, sa, 16 + (lane & 15));
    return w;
}

// 16 values of a row as eight words of two.
__device__ __forceinline__ void load16(uint32_t (&x)[8], const uint16_t* p, bool aligned) {
    if (aligned) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(p)), v = __ldg(reinterpret_cast<const uint4*>(p) + 1);
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
        x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = uint32_t(__ldg(p + 2 * i)) | uint32_t(__ldg(p + 2 * i + 1)) << 16;
    }
}

// Minimum / maximum of two pairs of values; a NaN stays one.
template <int T>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t d;
    if (T == 0)
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
template <int T>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    if (T == 0)
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
template <int T>
__device__ __forceinline__ float half_of(uint32_t w, int hi) {
    if (T == 0) return hi ? bf16_hi(w) : bf16_lo(w);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return hi ? f.y : f.x;
}
// A 16-bit value less an fp32 one, in one rounding.
template <int T>
__device__ __forceinline__ float less(uint32_t w, int hi, float m) {
    const uint16_t h = uint16_t(hi ? w >> 16 : w & 0xffffu);
    float d;
    if (T == 0)
        asm("sub.f32.bf16 %0, %1, %2;" : "=f"(d) : "h"(h), "f"(m));
    else
        asm("sub.f32.f16 %0, %1, %2;" : "=f"(d) : "h"(h), "f"(m));
    return d;
}

// Quantises the 64 values that four neighbouring lanes hold.  code: the lane's eight bytes;
// the group's scale and minimum (bf16, low and high half) are returned.
//   A code is the fp32 quotient (x - m) / s rounded to an integer, where quotients half-way
// between two integers are common (s has 8 bits, x - m a few more), so the quotient has to
// be exact there.  One residual correction of a s^-1 makes it so: with r = s^-1 (1 + e1) and
// q = a r (1 + e2), the residual a - q s is exact in one fused operation, and q + residual r
// is a / s to 2^-46 before its rounding, so a quotient of few bits comes out as itself.
template <int T>
__device__ __forceinline__ uint32_t quantise(const uint32_t (&x)[8], uint2* code) {
    uint32_t lo2 = x[0], hi2 = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo2 = min2<T>(lo2, x[i]);
        hi2 = max2<T>(hi2, x[i]);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        lo2 = min2<T>(lo2, __shfl_xor_sync(0xffffffffu, lo2, o));
        hi2 = max2<T>(hi2, __shfl_xor_sync(0xffffffffu, hi2, o));
    }
    lo2 = min2<T>(lo2, lo2 >> 16 | lo2 << 16);
    hi2 = max2<T>(hi2, hi2 >> 16 | hi2 << 16);
    const float lo = half_of<T>(lo2, 0), hi = half_of<T>(hi2, 0);
    const uint16_t mb = float_to_bf16(lo);
    const float m = bf16_to_float(mb), range = fmaxf(hi - m, 0.f);
    const uint16_t sb = float_to_bf16(__fdiv_rn(range, 15.f));
    const float s = bf16_to_float(sb);
    const bool bad = !(s < INFINITY && fabsf(m) < INFINITY);
    const bool flat = bad || s == 0.f;
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: a small number added to it is rounded to an integer
    uint32_t t[16];
    // tiny scales, and ranges that rounding took out of [0, 15 s], go the plain way
    if (!flat && (s < 0x1p-100f || lo < m || range > 15.4f * s)) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            t[i] = uint32_t(fminf(fmaxf(rintf(__fdiv_rn(less<T>(x[i >> 1], i & 1, m), s)), 0.f), 15.f));
    } else {
        const float r = flat ? 0.f : __frcp_rn(s);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float a = less<T>(x[i >> 1], i & 1, m);
            const float q = a * r;
            t[i] = __float_as_uint(fmaf(fmaf(-q, s, a), r, q) + kMagic);
        }
    }
    uint32_t y[8];  // low byte: code of value j, and of value j + 8 above it
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = t[j] + t[j + 8] * 16u;
    const uint32_t w0 = __byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040), 0x5410);
    const uint32_t w1 = __byte_perm(__byte_perm(y[4], y[5], 0x0040), __byte_perm(y[6], y[7], 0x0040), 0x5410);
    *code = flat ? make_uint2(0u, 0u) : make_uint2(w0, w1);
    return bad ? 0x7FC07FC0u : uint32_t(sb) | uint32_t(mb) << 16;
}

}  // namespace

template <int T>
__global__ void __launch_bounds__(32 * kRowsWarps) cache_append_kernel(const CacheRowsArgs a) {
    griddep_wait();
    griddep_launch();
    __shared__ __align__(16) uint32_t s_piece[kRowsWarps][2 * kPiece / 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = blockIdx.y * kRowsWarps + warp;
    if (head >= a.n_heads) return;
    const int64_t i0 = int64_t(blockIdx.x) * 16;
    const int G = a.c.groups;
    const Window win = window_of(a.slots, i0, a.n_tokens, a.c.n_pages << a.c.page_shift, a.flags);
    const int r8 = lane >> 2, run = lane & 3;
    const uint16_t* k0 = static_cast<const uint16_t*>(a.k) + head * a.k_head + run * 16;
    const uint16_t* v0 = static_cast<const uint16_t*>(a.v) + head * a.v_head + run * 16;

    const uint32_t start = uint32_t(win.runs >> 16) & 0xffffu;
    if (start) {
        // a whole piece (a window holds the start of one at most): codes laid out in shared
        // memory, then 16 bytes a lane
        const int at = __ffs(start) - 1;
        uint32_t* piece = s_piece[warp];
        const int64_t row = i0 + at + r8;
        for (int gr = 0; gr < G; ++gr) {
            uint32_t x[4][8];  // keys of rows r8 and r8 + 8, values of the same
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                load16(x[half], k0 + (row + 8 * half) * a.k_row + gr * 64, a.aligned);
                load16(x[2 + half], v0 + (row + 8 * half) * a.v_row + gr * 64, a.aligned);
            }
            uint2 c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t sm = quantise<T>(x[i], &c[i]);
                if (run == 0) piece[G * 256 + ((r8 + 8 * (i & 1)) * G + gr) * 2 + (i >> 1)] = sm;
            }
            // keys: word 16 g + 4 t + run holds bytes 2 t, 2 t + 1 of rows g and g + 8
            uint32_t* kc = piece + gr * 128 + r8 * 16 + run;
            kc[0] = __byte_perm(c[0].x, c[1].x, 0x5140);
            kc[4] = __byte_perm(c[0].x, c[1].x, 0x7362);
            kc[8] = __byte_perm(c[0].y, c[1].y, 0x5140);
            kc[12] = __byte_perm(c[0].y, c[1].y, 0x7362);
            // values: word 16 j + 4 (row / 2) + run holds byte j of rows 2 (row / 2), + 1, and both + 8;
            // even rows write bytes 0 .. 3, odd ones bytes 4 .. 7
            const bool odd = r8 & 1;
            const uint32_t send0 = odd ? c[2].x : c[2].y, send1 = odd ? c[3].x : c[3].y;
            const uint32_t got0 = __shfl_xor_sync(0xffffffffu, send0, 4), got1 = __shfl_xor_sync(0xffffffffu, send1, 4);
            const uint32_t e0 = odd ? got0 : c[2].x, e1 = odd ? got1 : c[3].x;  // even row, low and high half
            const uint32_t o0 = odd ? c[2].y : got0, o1 = odd ? c[3].y : got1;
            uint32_t* vc = piece + (G + gr) * 128 + (odd ? 64 : 0) + (r8 >> 1) * 4 + run;
            const uint32_t ea = __byte_perm(e0, e1, 0x5140), eb = __byte_perm(e0, e1, 0x7362);
            const uint32_t oa = __byte_perm(o0, o1, 0x5140), ob = __byte_perm(o0, o1, 0x7362);
            vc[0] = __byte_perm(ea, oa, 0x5410);
            vc[16] = __byte_perm(ea, oa, 0x7632);
            vc[32] = __byte_perm(eb, ob, 0x5410);
            vc[48] = __byte_perm(eb, ob, 0x7632);
        }
        __syncwarp();
        uint4* dst = reinterpret_cast<uint4*>(piece_of(a.c, __shfl_sync(0xffffffffu, win.slot, at), a.head0 + head));
        const uint4* src = reinterpret_cast<const uint4*>(piece);
        for (int i = lane; i < G * kPiece / 16; i += 32) dst[i] = src[i];
    }
    // rows by themselves: their bytes go where they belong
    for (uint32_t left = win.alone; left;) {
        int mine = -1;  // the r8-th row that is left
        uint32_t m = left;
        for (int i = 0; i < 8 && m; ++i, m &= m - 1)
            if (i == r8) mine = __ffs(m) - 1;
        left = m;
        const int slot = __shfl_sync(0xffffffffu, win.slot, mine & 15);
        const int64_t row = mine >= 0 ? i0 + mine : 0;
        uint8_t* piece = piece_of(a.c, mine >= 0 ? slot : 0, a.head0 + head);
        const int r = slot & 15;
        for (int gr = 0; gr < G; ++gr) {
            uint32_t x[2][8];
            load16(x[0], k0 + row * a.k_row + gr * 64, a.aligned);
            load16(x[1], v0 + row * a.v_row + gr * 64, a.aligned);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint2 c;
                const uint32_t sm = quantise<T>(x[i], &c);
                if (mine >= 0) {
                    uint8_t* codes = piece + (i * G + gr) * 512;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        codes[i ? value_byte(r, run * 8 + j) : key_byte(r, run * 8 + j)] =
                            uint8_t((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
                    if (run == 0) *reinterpret_cast<uint32_t*>(piece + G * 1024 + (r * G + gr) * 8 + i * 4) = sm;
                }
            }
        }
    }
}

namespace {

// The lane's 16 values from its eight bytes, scale and minimum, to a row of `T`.
template <int T>
__device__ __forceinline__ void write16(void* base, int64_t at, uint2 code, uint32_t sm) {
    const float s = bf16_lo(sm), m = bf16_hi(sm);
    float x[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t byte = (j < 4 ? code.x : code.y) >> (8 * (j & 3));
        // 2^23 + c as bits, less 2^23
        x[j] = fmaf(s, __uint_as_float((byte & 15u) | 0x4B000000u) - 8388608.f, m);
        x[j + 8] = fmaf(s, __uint_as_float((byte >> 4 & 15u) | 0x4B000000u) - 8388608.f, m);
    }
    if (T == 2) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (T == 0) {
                w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
            } else {
                const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at);
        p[0] = make_uint4(w[0], w[1], w[2], w[3]);
        p[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

}  // namespace

template <int T>
__global__ void __launch_bounds__(32 * kRowsWarps) cache_read_kernel(const CacheRowsArgs a) {
    griddep_wait();
    griddep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = blockIdx.y * kRowsWarps + warp;
    if (head >= a.n_heads) return;
    const int total = a.c.n_pages << a.c.page_shift, G = a.c.groups;
    const int r8 = lane >> 2, run = lane & 3;
    for (int half = 0; half < 2; ++half) {
        const int64_t i = int64_t(blockIdx.x) * 16 + half * 8 + r8;
        if (i >= a.n_tokens) continue;
        const int slot = a.slots[i];
        if (slot >= total && run == 0) atomicOr(a.flags, kFlagBounds);
        const bool live = slot >= 0 && slot < total;
        const int r = slot & 15, hi = r >> 3;
        const uint8_t* piece = piece_of(a.c, live ? slot : 0, a.head0 + head);
        for (int gr = 0; gr < G; ++gr) {
            const int64_t at = (i * a.n_heads + head) * (64 * G) + gr * 64 + run * 16;
            uint2 sm = make_uint2(0u, 0u), kc = make_uint2(0u, 0u), vc = make_uint2(0u, 0u);
            if (live) {
                sm = *reinterpret_cast<const uint2*>(piece + G * 1024 + (r * G + gr) * 8);
                // words that hold the row's bytes beside those of its neighbours
                const uint32_t* kw = reinterpret_cast<const uint32_t*>(piece + gr * 512) + (r & 7) * 16 + run;
                const uint32_t* vw = reinterpret_cast<const uint32_t*>(piece + (G + gr) * 512) + ((r & 7) >> 1) * 4 + run;
                const int ks = hi ? 0x7531 : 0x6420, vs = (r & 1) * 2 + hi;  // byte selectors
                const uint32_t b0 = __byte_perm(kw[0], kw[4], ks), b1 = __byte_perm(kw[8], kw[12], ks);
                kc = make_uint2(b0, b1);
                const int pick = vs | (4 + vs) << 4;
                vc.x = __byte_perm(__byte_perm(vw[0], vw[16], pick), __byte_perm(vw[32], vw[48], pick), 0x5410);
                vc.y = __byte_perm(__byte_perm(vw[64], vw[80], pick), __byte_perm(vw[96], vw[112], pick), 0x5410);
            }
            write16<T>(a.out_k, at, kc, sm.x);
            write16<T>(a.out_v, at, vc, sm.y);
        }
    }
}

cudaError_t launch_cache_append(const CacheRowsArgs& a, cudaStream_t s) {
    if (a.n_tokens <= 0) return cudaSuccess;
    const dim3 grid(unsigned((int64_t(a.n_tokens) + 15) / 16), unsigned((a.n_heads + kRowsWarps - 1) / kRowsWarps));
    auto kernel = a.dtype == 0 ? cache_append_kernel<0> : cache_append_kernel<1>;
    return launch_pdl(kernel, grid, dim3(32 * kRowsWarps), 0, s, a);
}

cudaError_t launch_cache_read(const CacheRowsArgs& a, cudaStream_t s) {
    if (a.n_tokens <= 0) return cudaSuccess;
    const dim3 grid(unsigned((int64_t(a.n_tokens) + 15) / 16), unsigned((a.n_heads + kRowsWarps - 1) / kRowsWarps));
    auto kernel = a.dtype == 0 ? cache_read_kernel<0> : a.dtype == 1 ? cache_read_kernel<1> : cache_read_kernel<2>;
    return launch_pdl(kernel, grid, dim3(32 * kRowsWarps), 0, s, a);
}

}  // namespace clef
