// Kernels of the paged 4-bit memory cache: page accounts, store, read back.  The stored
// form and its byte layout are described in clef_cache.h.
#include "cache.h"
#include "common.cuh"
#include "kernels.h"

namespace clef {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCtas = 8;  // CTAs of a large step's cluster

// Inclusive sums of two numbers over the block's threads (1024), in thread order; `tmp` holds
// 2 x 32 values.
__device__ __forceinline__ int2 block_scan(int x, int y, int (*tmp)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
            x += u;
            y += v;
        }
    }
    __syncthreads();  // tmp may still be read by the previous scan
    if (lane == 31) {
        tmp[0][warp] = x;
        tmp[1][warp] = y;
    }
    __syncthreads();
    int s = tmp[0][lane], t = tmp[1][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o), v = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) {
            s += u;
            t += v;
        }
    }
    const int bx = __shfl_sync(0xffffffffu, s, max(warp - 1, 0)), by = __shfl_sync(0xffffffffu, t, max(warp - 1, 0));
    return warp > 0 ? make_int2(x + bx, y + by) : make_int2(x, y);
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

}  // namespace

// Page accounts: one CTA, or a cluster of them that share out the page moves and the slots
// (each CTA works out what every request gives back, needs and gains by itself, one thread a
// request, in three scans; a search in the sums finds the request of a page or slot).  Three
// phases with the cluster's barrier between them: pages come back, pages are granted, slots
// are written.  Bound by the latency of these dependent steps, not by bytes; each thread has
// four moves under way at a time.
__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const CachePlanArgs a) {
    griddep_wait();
    griddep_launch();
    __shared__ int tmp[2][32];
    __shared__ int s_rel[kPlanThreads], s_more[kPlanThreads], s_have[kPlanThreads], s_old[kPlanThreads];
    __shared__ int s_cu[kPlanThreads + 1];
    __shared__ int s_grant;
    const int t = threadIdx.x;
    const bool alone = gridDim.x == 1;
    const int first = blockIdx.x * kPlanThreads + t, step = gridDim.x * kPlanThreads;
    const int page = 1 << a.page_shift;
    const int64_t cap = int64_t(a.width) << a.page_shift;
    const bool lead = blockIdx.x == 0;  // reports, and writes what there is one of
    auto meet = [&] {
        if (alone)
            __syncthreads();
        else
            cluster_sync();
    };
    int old = 0, want = 0, have = 0, need = 0;
    if (t < a.B) {
        old = a.lengths[t];
        want = a.want[t];
        const bool bad_old = old < 0 || old > cap;
        if (bad_old || want < 0 || want > cap) {
            if (lead) atomicOr(a.flags, kFlagBounds);
            want = old;  // left as it is
        }
        if (!bad_old) {
            have = int((int64_t(old) + page - 1) >> a.page_shift);
            need = int((int64_t(want) + page - 1) >> a.page_shift);
        }
    }
    int count = *a.free_count;
    if (count < 0 || count > a.n_pages) {
        if (lead && t == 0) atomicOr(a.flags, kFlagBounds);
        count = count < 0 ? 0 : a.n_pages;
    }
    if (t == 0) s_grant = 0;
    const int more = max(need - have, 0);
    const int2 ends = block_scan(max(have - need, 0), more, tmp);
    s_rel[t] = ends.x;
    s_more[t] = ends.y;
    s_have[t] = have;
    s_old[t] = old;
    __syncthreads();
    const int n_rel = s_rel[kPlanThreads - 1];
    const int top = min(count + n_rel, a.n_pages);
    const bool fits = more == 0 || ends.y <= top;
    if (fits && more > 0) atomicMax(&s_grant, ends.y);
    s_cu[t + 1] = block_scan(fits ? max(want - old, 0) : 0, 0, tmp).x;
    if (t == 0) s_cu[0] = 0;
    __syncthreads();
    // give back: ascending index i of (request, page) pairs; the stack takes them in descending order
    for (int i0 = first; i0 < n_rel; i0 += 4 * step) {
        int id[4];
        int64_t at[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * step;
            if (i >= n_rel) continue;
            const int b = upper(s_rel, a.B, i);
            at[u] = int64_t(b) * a.width + s_have[b] - (s_rel[b] - i);
            id[u] = a.table[at[u]];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * step, pos = count + n_rel - 1 - i;
            if (i >= n_rel) continue;
            a.table[at[u]] = -1;
            if (pos < a.n_pages)
                a.free_pages[pos] = id[u];
            else
                atomicOr(a.flags, kFlagBounds);  // more pages came back than there are
        }
    }
    meet();  // everyone has read the old lengths and count; the pages that came back are on the stack
    const int grant = s_grant;  // requests fit in order, so the granted pages are the first ones
    for (int i0 = first; i0 < grant; i0 += 4 * step) {
        int id[4];
        int64_t at[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * step;
            if (i >= grant) continue;
            const int b = upper(s_more, a.B, i);
            at[u] = int64_t(b) * a.width + s_have[b] + i - (b > 0 ? s_more[b - 1] : 0);
            id[u] = a.free_pages[top - 1 - i];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * step;
            if (i >= grant) continue;
            a.table[at[u]] = id[u];
            a.free_pages[top - 1 - i] = -1;
        }
    }
    if (lead) {
        if (t < a.B) {
            if (fits)
                a.lengths[t] = want;
            else
                atomicOr(a.flags, kFlagPages);
            a.cu[t] = s_cu[t];
        }
        if (t == 0) {
            a.cu[a.B] = s_cu[a.B];
            *a.free_count = top - grant;
            if (s_cu[a.B] > a.n_slots) atomicOr(a.flags, kFlagBounds);
        }
    }
    meet();  // the tables are as they will be
    // one slot a thread, or four neighbouring ones: one search, and one page number where they
    // share a page
    const int total = s_cu[a.B], per = a.n_slots <= step ? 1 : 4;
    for (int64_t i0 = per * int64_t(first); i0 < a.n_slots; i0 += per * int64_t(step)) {
        int slot[4] = {-1, -1, -1, -1};
        if (i0 < total) {
            int b = min(upper(s_cu + 1, a.B, int(i0)), a.B - 1), at = -1, id = -1;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = int(i0) + u;
                if (u >= per || i >= total || i >= a.n_slots) break;
                while (b < a.B - 1 && i >= s_cu[b + 1]) {
                    ++b;
                    at = -1;
                }
                const int pos = s_old[b] + i - s_cu[b], col = pos >> a.page_shift;
                if (col != at) {
                    at = col;
                    id = pos >= 0 && col < a.width ? a.table[int64_t(b) * a.width + col] : -1;
                    if (id < 0 || id >= a.n_pages) {
                        atomicOr(a.flags, kFlagBounds);
                        id = -1;
                    }
                }
                if (id >= 0) slot[u] = (id << a.page_shift) | (pos & (page - 1));
            }
        }
        if (per == 4 && i0 + 4 <= a.n_slots && (reinterpret_cast<uintptr_t>(a.slots) & 15) == 0) {
            *reinterpret_cast<int4*>(a.slots + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (u < per && i0 + u < a.n_slots) a.slots[i0 + u] = slot[u];
        }
    }
}

cudaError_t launch_cache_plan(const CachePlanArgs& a, cudaStream_t s) {
    // A cluster pays from a few thousand slots on (its barriers take about a microsecond).
    const unsigned ctas = a.n_slots > 4 * kPlanThreads ? kPlanCtas : 1;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return counted(cudaLaunchKernelEx(&cfg, cache_plan_kernel, a));
}

// ------------------------------------------------------------------- rows
//
// Store: a warp takes a window of 16 consecutive rows, one group of 64 values of one head at a
// time.  Four lanes hold a row's group, 16 values each (lane / 4 is the row of eight, lane % 4
// the run of 16 values): a lane owns the eight code bytes of its run, and a row's minimum and
// maximum cost two exchanges.  Where 16 rows fill a whole piece, wherever in the window they
// start, their codes go through shared memory and out as 16 bytes a lane; other rows write the
// bytes that are their own.  Read back: eight rows a warp, words straight from the piece.
//   131072 rows x 16 heads of 64 in bf16: store 136 us (689 MB, 75 % of the measured copy rate;
// 860 instructions a window and head's group, five of them for each quotient, fill 69 % of the
// issue slots), read back 110 us (92 %).

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
    // range / 15 by the same correction; tiny ranges, where the residual would lose bits, are divided
    const float third = range * (1.f / 15.f);
    float width = fmaf(fmaf(-third, 15.f, range), 1.f / 15.f, third);
    if (!(range > 0x1p-90f && range < INFINITY)) width = __fdiv_rn(range, 15.f);
    const uint16_t sb = float_to_bf16(width);
    const float s = bf16_to_float(sb);
    const bool bad = !(s < INFINITY && fabsf(m) < INFINITY);
    const bool flat = bad || s == 0.f;
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: a small number added to it is rounded to an integer
    uint32_t t[16];
    // tiny scales, and ranges that rounding took past 15 s, go the plain way
    if (!flat && (s < 0x1p-90f || range > 15.4f * s)) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            t[i] = uint32_t(fminf(fmaxf(rintf(__fdiv_rn(less<T>(x[i >> 1], i & 1, m), s)), 0.f), 15.f));
    } else {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));  // within an ulp
        if (flat) r = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float a = less<T>(x[i >> 1], i & 1, m);
            if (T == 1) a = fmaxf(a, 0.f);  // m may have been rounded up past an fp16 minimum
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
__global__ void __launch_bounds__(32 * kRowsWarps, 4) cache_append_kernel(const CacheRowsArgs a) {
    griddep_wait();
    griddep_launch();
    __shared__ __align__(16) uint32_t s_codes[kRowsWarps][256];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r8 = lane >> 2, run = lane & 3, G = a.c.groups;
    for (int64_t i0 = int64_t(blockIdx.x) * 16; i0 < a.n_tokens; i0 += int64_t(gridDim.x) * 16) {
        const Window win = window_of(a.slots, i0, a.n_tokens, a.c.n_pages << a.c.page_shift, a.flags);
        // a warp takes one group of 64 values of one head at a time
        for (int part = blockIdx.y * kRowsWarps + warp; part < a.n_heads * G; part += gridDim.y * kRowsWarps) {
            const int head = part >> (G - 1), gr = part & (G - 1);
            const uint16_t* k0 = static_cast<const uint16_t*>(a.k) + head * a.k_head + gr * 64 + run * 16;
            const uint16_t* v0 = static_cast<const uint16_t*>(a.v) + head * a.v_head + gr * 64 + run * 16;

            const uint32_t start = uint32_t(win.runs >> 16) & 0xffffu;
            if (start) {
                // a whole piece (a window holds the start of one at most): codes laid out in shared
                // memory, then 16 bytes a lane
                const int at = __ffs(start) - 1;
                const int64_t row = i0 + at + r8;
                uint32_t x[4][8];  // keys of rows r8 and r8 + 8, values of the same
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    load16(x[half], k0 + (row + 8 * half) * a.k_row, a.aligned);
                    load16(x[2 + half], v0 + (row + 8 * half) * a.v_row, a.aligned);
                }
                uint8_t* piece = piece_of(a.c, __shfl_sync(0xffffffffu, win.slot, at), a.head0 + head);
                uint2 c[4];
                uint32_t sm[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) sm[i] = quantise<T>(x[i], &c[i]);
                if (run == 0) {
                    uint2* scales = reinterpret_cast<uint2*>(piece + G * 1024) + r8 * G + gr;
                    scales[0] = make_uint2(sm[0], sm[2]);
                    scales[8 * G] = make_uint2(sm[1], sm[3]);
                }
                // keys: word 16 g + 4 t + run holds bytes 2 t, 2 t + 1 of rows g and g + 8
                uint32_t* kc = s_codes[warp] + r8 * 16 + run;
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
                uint32_t* vc = s_codes[warp] + 128 + (odd ? 64 : 0) + (r8 >> 1) * 4 + run;
                const uint32_t ea = __byte_perm(e0, e1, 0x5140), eb = __byte_perm(e0, e1, 0x7362);
                const uint32_t oa = __byte_perm(o0, o1, 0x5140), ob = __byte_perm(o0, o1, 0x7362);
                vc[0] = __byte_perm(ea, oa, 0x5410);
                vc[16] = __byte_perm(ea, oa, 0x7632);
                vc[32] = __byte_perm(eb, ob, 0x5410);
                vc[48] = __byte_perm(eb, ob, 0x7632);
                __syncwarp();
                const uint4* src = reinterpret_cast<const uint4*>(s_codes[warp]) + lane;
                reinterpret_cast<uint4*>(piece + gr * 512)[lane] = src[0];
                reinterpret_cast<uint4*>(piece + (G + gr) * 512)[lane] = src[32];
                __syncwarp();  // the codes are out before the next ones
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
                uint32_t x[2][8];
                load16(x[0], k0 + row * a.k_row, a.aligned);
                load16(x[1], v0 + row * a.v_row, a.aligned);
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
}

namespace {

// Two codes as bf16 numbers (bits 0-3 and 16-19 of x): 128 + c, less 128, exact.
__device__ __forceinline__ uint32_t codes2(uint32_t x) {
    const uint32_t w = (x & 0x000F000Fu) | 0x43004300u, off = 0x43004300u;
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&w),
                                     *reinterpret_cast<const __nv_bfloat162*>(&off));
    return *reinterpret_cast<const uint32_t*>(&v);
}
// scale * c + minimum with c and the scale in bf16, in one fp32 rounding.
__device__ __forceinline__ float stands_for(uint32_t c2, int hi, uint16_t scale, float m) {
    const uint16_t c = uint16_t(hi ? c2 >> 16 : c2 & 0xffffu);
    float d;
    asm("fma.rn.f32.bf16 %0, %1, %2, %3;" : "=f"(d) : "h"(c), "h"(scale), "f"(m));
    return d;
}

// The lane's 16 values from its eight bytes, scale and minimum, to row `i` of `T` (i rows from
// base, `live` where there is one).  Lanes 16 apart hold rows four apart: they swap halves, so
// that a store instruction writes whole 32-byte sectors (half a sector at a time costs 1.3
// times the time).  All lanes of the warp come here.
template <int T>
__device__ __forceinline__ void write16(void* base, int64_t at, int64_t row_stride, bool live, bool other_live, uint2 code,
                                        uint32_t sm) {
    const uint16_t s = uint16_t(sm & 0xffffu);
    const float m = bf16_hi(sm);
    float x[16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t w = h ? code.y : code.x;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // bits 4 e of bytes 0 and 2 (e < 2), of bytes 1 and 3 (e >= 2)
            const uint32_t c = codes2(w >> (4 * (e & 1) + 8 * (e >> 1)));
            const int j = 4 * h + (e >> 1) + 8 * (e & 1);
            x[j] = stands_for(c, 0, s, m);
            x[j + 2] = stands_for(c, 1, s, m);
        }
    }
    constexpr int kWords = T == 2 ? 16 : 8;
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (T == 0) {
            w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
        } else if (T == 1) {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            w[2 * i] = __float_as_uint(x[2 * i]);
            w[2 * i + 1] = __float_as_uint(x[2 * i + 1]);
        }
    }
    // 32 bytes at a time: the lower lane writes the first half of its own row and of the upper
    // lane's, the upper lane the second halves
    const bool upper_lane = threadIdx.x & 16;
    uint32_t* p = static_cast<uint32_t*>(base) + at * (T == 2 ? 4 : 2) / 4;
    const int64_t to_other = (upper_lane ? -4 : 4) * row_stride * (T == 2 ? 4 : 2) / 4;
#pragma unroll
    for (int i = 0; i < kWords; i += 8) {
        uint32_t got[4], own[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            got[j] = __shfl_xor_sync(0xffffffffu, upper_lane ? w[i + j] : w[i + 4 + j], 16);
            own[j] = upper_lane ? w[i + 4 + j] : w[i + j];
        }
        uint32_t* q = p + i + (upper_lane ? 4 : 0);
        uint4* first = reinterpret_cast<uint4*>(upper_lane ? q + to_other : q);
        uint4* second = reinterpret_cast<uint4*>(upper_lane ? q : q + to_other);
        // rows of the lower lanes, then rows of the upper ones
        if (upper_lane ? other_live : live)
            *first = upper_lane ? make_uint4(got[0], got[1], got[2], got[3]) : make_uint4(own[0], own[1], own[2], own[3]);
        if (upper_lane ? live : other_live)
            *second = upper_lane ? make_uint4(own[0], own[1], own[2], own[3]) : make_uint4(got[0], got[1], got[2], got[3]);
    }
}

}  // namespace

template <int T>
__global__ void __launch_bounds__(32 * kRowsWarps) cache_read_kernel(const CacheRowsArgs a) {
    griddep_wait();
    griddep_launch();
    // eight rows a warp; the warp beside it takes the next eight, which share its words
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int run = lane & 3, G = a.c.groups;
    const int64_t row_stride = int64_t(a.n_heads) * (64 * G);
    for (int64_t i0 = int64_t(blockIdx.x) * 16; i0 < a.n_tokens; i0 += int64_t(gridDim.x) * 16) {
        const int64_t i = i0 + (warp & 1) * 8 + (lane >> 2);
        const bool there = i < a.n_tokens, other = (lane & 16 ? i - 4 : i + 4) < a.n_tokens;
        const int slot = there ? a.slots[i] : -1, total = a.c.n_pages << a.c.page_shift;
        if (slot >= total && run == 0) atomicOr(a.flags, kFlagBounds);
        const bool live = slot >= 0 && slot < total;
        const int r = slot & 15, hi = r >> 3;
        for (int part = blockIdx.y * (kRowsWarps / 2) + (warp >> 1); part < a.n_heads * G; part += gridDim.y * (kRowsWarps / 2)) {
            const int head = part >> (G - 1), gr = part & (G - 1);
            const uint8_t* piece = piece_of(a.c, live ? slot : 0, a.head0 + head);
            uint2 sm = make_uint2(0u, 0u), kc = make_uint2(0u, 0u), vc = make_uint2(0u, 0u);
            if (live) {
                sm = *reinterpret_cast<const uint2*>(piece + G * 1024 + (r * G + gr) * 8);
                // words that hold the row's bytes beside those of its neighbours
                const uint32_t* kw = reinterpret_cast<const uint32_t*>(piece + gr * 512) + (r & 7) * 16 + run;
                const uint32_t* vw = reinterpret_cast<const uint32_t*>(piece + (G + gr) * 512) + ((r & 7) >> 1) * 4 + run;
                const int ks = hi ? 0x7531 : 0x6420, at = (r & 1) * 2 + hi, vs = at | (4 + at) << 4;  // byte selectors
                kc = make_uint2(__byte_perm(kw[0], kw[4], ks), __byte_perm(kw[8], kw[12], ks));
                vc.x = __byte_perm(__byte_perm(vw[0], vw[16], vs), __byte_perm(vw[32], vw[48], vs), 0x5410);
                vc.y = __byte_perm(__byte_perm(vw[64], vw[80], vs), __byte_perm(vw[96], vw[112], vs), 0x5410);
            }
            const int64_t at = i * row_stride + part * 64 + run * 16;
            write16<T>(a.out_k, at, row_stride, there, other, kc, sm.x);
            write16<T>(a.out_v, at, row_stride, there, other, vc, sm.y);
        }
    }
}

namespace {

// CTAs over the 16-row windows and, where there are few of those, over the heads' groups that
// `per_cta` warps or pairs of warps leave; each CTA walks several windows of a large call.
// (Store and read back of 131072 rows x 16 heads: 265 us with a CTA for each window and eight
// heads, 245 us with 32 CTAs an SM that walk, 270 with 4.)
dim3 rows_grid(const CacheRowsArgs& a, int per_cta) {
    const int64_t windows = (int64_t(a.n_tokens) + 15) / 16, parts = (a.n_heads * a.c.groups + per_cta - 1) / per_cta;
    const int64_t most = int64_t(num_sms()) * 32;
    if (windows * parts <= most) return dim3(unsigned(windows), unsigned(parts));
    return dim3(unsigned(windows < most ? windows : most), 1);
}

}  // namespace

cudaError_t launch_cache_append(const CacheRowsArgs& a, cudaStream_t s) {
    if (a.n_tokens <= 0) return cudaSuccess;
    auto kernel = a.dtype == 0 ? cache_append_kernel<0> : cache_append_kernel<1>;
    return launch_pdl(kernel, rows_grid(a, kRowsWarps), dim3(32 * kRowsWarps), 0, s, a);
}

cudaError_t launch_cache_read(const CacheRowsArgs& a, cudaStream_t s) {
    if (a.n_tokens <= 0) return cudaSuccess;
    auto kernel = a.dtype == 0 ? cache_read_kernel<0> : a.dtype == 1 ? cache_read_kernel<1> : cache_read_kernel<2>;
    return launch_pdl(kernel, rows_grid(a, kRowsWarps / 2), dim3(32 * kRowsWarps), 0, s, a);
}

}  // namespace clef
