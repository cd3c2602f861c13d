// Shared by the two attention kernels of the 4-bit memory cache: the requests of a call, its
// work items, and small matrix helpers.
#pragma once

#include <algorithm>

#include "cache.h"
#include "common.cuh"
#include "kernels.h"
#include "per_device.h"

namespace clef {

namespace {

constexpr int kAttendWarps = 4;  // of a CTA of either attention kernel
constexpr int kAttendThreads = 32 * kAttendWarps;

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same with nothing added.
__device__ __forceinline__ void mma_f16_16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Transpose of an 8 x 8 block of 16-bit values held one row a group of four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Value codes of two tokens (bits 0-3 and 16-19 of x; bits 4-7 and 20-23) less 8, in fp16, exact.
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, float b) {
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&a), __float2half2_rn(b));
    return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ uint32_t centred_low(uint32_t x) { return sub_f16x2((x & 0x000F000Fu) | 0x64006400u, 1032.f); }
__device__ __forceinline__ uint32_t centred_high(uint32_t x) { return sub_f16x2((x & 0x00F000F0u) | 0x54005400u, 72.f); }

// What a packed pair of fp16 numbers leaves of the two that it was rounded from, in fp16.
__device__ __forceinline__ uint32_t rest_f16(uint32_t w, float lo, float hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return pack_f16(lo - f.x, hi - f.y);
}

// 2^e, e clamped to the normal range.
__device__ __forceinline__ float pow2i(int e) {
    return __uint_as_float(uint32_t(min(max(e, -126), 127) + 127) << 23);
}

// A row's softmax weights meet the matrix unit in fp16, multiplied by the size of the token's values
// (its scale, or the power of two below its largest value) and by a power of two `mul` of the row's own.  It
// moves when the row's reference does, to put the largest product of the step in [4, 8), and down when a
// product exceeds kMostWeight.  Between two moves the products only add, so the largest weight
// that a row has used is 4 at least and the floor of fp16's subnormals 2^-27 of it: a row is as exact as the
// tokens that it gives weight to, whatever others, or tokens that it does not see, hold.
constexpr float kMostWeight = 16384.f;

__device__ __forceinline__ int exponent_of(float x) { return int(__float_as_uint(x) >> 23) - 127; }  // of x >= 0

// The softmax weights of a row are multiplied by 2^-mx (mx > 0): frac 2^-k, with frac in [0.7, 1.5).
struct Decay {
    float frac = 1.f, corr = 1.f;  // corr: the whole factor, 0 where it is below 2^-126
    int k = 0;
    __device__ void set(float mx) {
        const float kf = rintf(fminf(mx, 300.f));
        frac = ex2_approx(kf - mx);
        k = int(kf);
        corr = k > 126 ? 0.f : frac * pow2i(-k);
    }
};

// Moves a row's `mul` for products p * size of at most x, and returns the factor of its sums, whose
// largest is `big` (they stay under 2^102, and give way to no smaller products beyond that).  With no product at
// all (values of zero) the power goes as high as the sums let it: the next products may have any size.
__device__ __forceinline__ float move_weights(float& mul, float x, float big, const Decay& d) {
    const int old = exponent_of(mul);
    int to = x > 0.f ? 2 - exponent_of(fminf(x, 0x1.fffffep127f)) : 119;
    if (big > 0.f) to = min(to, old + d.k + 100 - exponent_of(big));
    to = min(max(to, -126), 119);  // (p mul stays finite)
    mul = pow2i(to);
    const int by = to - old - d.k;
    return by < -126 ? 0.f : d.frac * pow2i(by);
}

// The two elements of a 32-bit word as fp32.
__device__ __forceinline__ float2 unpack2(uint32_t w, int dtype) {
    if (dtype == 0) return make_float2(bf16_lo(w), bf16_hi(w));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// What a CTA needs to know of every request, in shared memory: its keys, first query row and
// query rows, the end of its partial rows as a running sum, and the order of the work items:
// the ends of the requests' whole splits, then the requests by the size of their last, shorter
// split, and the ends of those.
struct Requests {
    int *len, *q0, *nq, *parts, *whole, *order, *last;
    static constexpr int kInts = 7;
    __device__ Requests(int* base, int n)
        : len(base), q0(base + n), nq(base + 2 * n), parts(base + 3 * n), whole(base + 4 * n), order(base + 5 * n),
          last(base + 6 * n) {}
};

struct Request {
    int len, q0, nq, chunks;
};

__device__ __forceinline__ Request request_of(const CacheAttendArgs& a, int b, bool report) {
    Request r;
    r.len = a.lengths[b];
    r.q0 = a.cu_q[b];
    int q1 = a.cu_q[b + 1];
    const int cap = int(min(int64_t(a.width) << a.c.page_shift, int64_t(0x7fffffff)));
    const bool bad = r.len < 0 || r.len > cap || r.q0 < 0 || q1 < r.q0 || q1 > a.total_q || q1 - r.q0 > a.max_q;
    if (bad) {
        if (report) atomicOr(a.flags, kFlagBounds);
        r.len = min(max(r.len, 0), cap);
        r.q0 = min(max(r.q0, 0), a.total_q);
        q1 = min(max(q1, r.q0), a.total_q);
    }
    r.nq = min(q1 - r.q0, a.max_q);
    r.chunks = (r.len - 1) / a.chunk + 1;  // 1 for no keys too
    return r;
}

// Requests of up to so many query rows (queries x the query heads that share a key head) are
// the few-rows kernel's, the others the many-rows kernel's: by the request alone, so that a
// row's result does not depend on the batch.  An item of the first holds up to 32 rows at head size
// 64 and 16 at 128, and these are the borders.  128 requests x 1024 keys in the first and the second, bf16:
//   16 heads of 64:   16 rows 73 and 131 us, 24 rows 105 and 152, 32 rows 146 and 154,
//                     33 rows 269 and 177, 64 rows 283 and 204
//   8 heads of 128:   8 rows 44 and 158 us, 16 rows 73 and 162, 64 rows 252 and 202;
//                     17 to 32 rows, in two items, would take 126-131 us in the first (second: 192)
__host__ __device__ constexpr int few_rows(int groups) { return groups == 1 ? 32 : 16; }

// Inclusive sums of two numbers over the CTA's threads.
__device__ __forceinline__ int2 scan_threads(int x, int y) {
    __shared__ int tmp[2][kAttendWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
            x += u;
            y += v;
        }
    }
    __syncthreads();  // tmp may still be read
    if (lane == 31) {
        tmp[0][warp] = x;
        tmp[1][warp] = y;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        x += tmp[0][w];
        y += tmp[1][w];
    }
    return make_int2(x, y);
}

// Work items of one split of a request: its key/value heads times its blocks of query rows.
// Requests of the other kernel have none.
template <int G, bool MANY>
__device__ __forceinline__ int items_of_split(const CacheAttendArgs& a, int nq, int rows_per_item) {
    const int rows = nq * a.share;
    return (rows > few_rows(G)) == MANY ? (rows + rows_per_item - 1) / rows_per_item * a.kv_heads : 0;
}

// Fills the tables and returns the number of items.  The last splits come in order of size, in
// sixteenths of a split and largest first, requests of one size by number: the same in every
// CTA.
template <int G, bool MANY>
__device__ __forceinline__ int scan_requests(const CacheAttendArgs& a, const Requests& s, int rows_per_item) {
    constexpr int kSizes = 17;  // the last one: requests whose splits are all whole, or that have no items
    __shared__ int count[kAttendWarps][kSizes], total[kSizes];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto size_of = [&](const Request& r) {
        const int left = r.len - (r.chunks - 1) * a.chunk;  // keys of the last split
        return left < a.chunk && items_of_split<G, MANY>(a, r.nq, rows_per_item) > 0 ? 15 - left * 16 / a.chunk : kSizes - 1;
    };
    if (a.B <= 32) {  // one warp does it all: a call for few requests should start soon
        if (warp == 0) {
            Request r = {};
            int size = kSizes, parts = 0, whole = 0;
            if (lane < a.B) {
                r = request_of(a, lane, blockIdx.x == 0);
                size = size_of(r);
                s.len[lane] = r.len;
                s.q0[lane] = r.q0;
                s.nq[lane] = r.nq;
                parts = r.chunks > 1 ? r.chunks * r.nq * a.q_heads : 0;
                whole = r.len / a.chunk * items_of_split<G, MANY>(a, r.nq, rows_per_item);
            }
            int at = 0, sorted = 0;
#pragma unroll
            for (int i = 0; i < kSizes; ++i) {
                const uint32_t m = __ballot_sync(0xffffffffu, size == i);
                if (i < size) at += __popc(m);
                if (i == size) at += __popc(m & ((1u << lane) - 1));
                if (i < kSizes - 1) sorted += __popc(m);
            }
            if (lane < a.B) s.order[at] = lane;
            __syncwarp();
            int last = lane < sorted ? items_of_split<G, MANY>(a, s.nq[s.order[lane]], rows_per_item) : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, parts, o), y = __shfl_up_sync(0xffffffffu, whole, o);
                const int z = __shfl_up_sync(0xffffffffu, last, o);
                if (lane >= o) {
                    parts += x;
                    whole += y;
                    last += z;
                }
            }
            if (lane < a.B) {
                s.parts[lane] = parts;
                s.whole[lane] = whole;
                s.last[lane] = last;
            }
        }
        __syncthreads();
        return s.whole[a.B - 1] + s.last[a.B - 1];
    }
    if (threadIdx.x < kSizes) total[threadIdx.x] = 0;
    for (int b0 = 0; b0 < a.B; b0 += kAttendThreads) {
        const int b = b0 + threadIdx.x;
        int size = kSizes - 1;
        if (b < a.B) {
            const Request r = request_of(a, b, blockIdx.x == 0);
            s.len[b] = r.len;
            s.q0[b] = r.q0;
            s.nq[b] = r.nq;
            size = size_of(r);
        }
        for (int i = threadIdx.x; i < kAttendWarps * kSizes; i += kAttendThreads) (&count[0][0])[i] = 0;
        __syncthreads();
        const uint32_t same = __match_any_sync(0xffffffffu, size);
        const int rank = __popc(same & ((1u << lane) - 1));
        if (rank == 0) count[warp][size] = __popc(same);
        __syncthreads();
        if (b < a.B) {
            int before = total[size] + rank;
            for (int w = 0; w < warp; ++w) before += count[w][size];
            s.last[b] = size << 16 | before;  // for now
        }
        __syncthreads();
        if (threadIdx.x < kSizes)
            for (int w = 0; w < kAttendWarps; ++w) total[threadIdx.x] += count[w][threadIdx.x];
        __syncthreads();
    }
    for (int b = threadIdx.x; b < a.B; b += kAttendThreads) {
        const int size = s.last[b] >> 16;
        int at = s.last[b] & 0xffff;
        for (int i = 0; i < size; ++i) at += total[i];
        s.order[at] = b;
    }
    __syncthreads();
    // running sums, a run of neighbouring requests a thread
    const int per = (a.B + kAttendThreads - 1) / kAttendThreads;
    const int b0 = threadIdx.x * per, b1 = min(b0 + per, a.B);
    int sorted = 0;
    for (int i = 0; i < kSizes - 1; ++i) sorted += total[i];
    int parts = 0, whole = 0, last = 0;
    for (int b = b0; b < b1; ++b) {
        const int chunks = (s.len[b] - 1) / a.chunk + 1;
        parts += chunks > 1 ? chunks * s.nq[b] * a.q_heads : 0;
        whole += s.len[b] / a.chunk * items_of_split<G, MANY>(a, s.nq[b], rows_per_item);
        last += b < sorted ? items_of_split<G, MANY>(a, s.nq[s.order[b]], rows_per_item) : 0;
        s.parts[b] = parts;
        s.whole[b] = whole;
        s.last[b] = last;
    }
    const int2 ends = scan_threads(whole, last);
    const int parts_end = scan_threads(parts, 0).x;
    for (int b = b0; b < b1; ++b) {
        s.parts[b] += parts_end - parts;
        s.whole[b] += ends.x - whole;
        s.last[b] += ends.y - last;
    }
    __syncthreads();
    return s.whole[a.B - 1] + s.last[a.B - 1];
}

// The item of a CTA's n-th turn: items, largest first, are dealt out in rows that run forward
// and back, so that the sums of their sizes come out nearly even (a decoding step of 64 requests
// of 156 to 16384 keys, 8 heads of 128: 52 us, and 58 us dealt in the requests' order).
__device__ __forceinline__ int item_of_turn(int n) {
    return n * int(gridDim.x) + ((n & 1) ? int(gridDim.x) - 1 - int(blockIdx.x) : int(blockIdx.x));
}

// A work item: a split of request b's keys, key/value head h, a block of its query rows.
struct Item {
    int b, h, split, row0, rows, t0, t1, ahead, p0;
};

// Number of entries of the non-decreasing `ends` (n of them) that are <= i, at most n - 1.
__device__ __forceinline__ int entry_of(const int* ends, int n, int i) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] <= i)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

template <int ROWS>
__device__ __forceinline__ Item item_of(const CacheAttendArgs& a, const Requests& s, int w) {
    Item k;
    const int n_whole = s.whole[a.B - 1];
    const bool last = w >= n_whole;
    int it = last ? w - n_whole : w;
    const int* ends = last ? s.last : s.whole;
    const int e = entry_of(ends, a.B, it);
    it -= e ? ends[e - 1] : 0;
    k.b = last ? s.order[e] : e;
    const int len = s.len[k.b], nq = s.nq[k.b];
    const int n_rows = nq * a.share;
    const int n_blocks = (n_rows + ROWS - 1) / ROWS;
    const int rest = n_blocks == 1 ? it : it / n_blocks;
    k.row0 = (it - rest * n_blocks) * ROWS;
    const int split = rest / a.kv_heads;
    k.h = rest - split * a.kv_heads;
    k.split = last ? len / a.chunk : split;
    k.rows = min(ROWS, n_rows - k.row0);
    k.t0 = k.split * a.chunk;
    k.t1 = min(k.t0 + a.chunk, len);
    k.ahead = len - nq;  // causal: query i sees keys 0 .. ahead + i
    if (a.causal) k.t1 = min(k.t1, k.ahead + a.by_share(k.row0 + k.rows - 1) + 1);
    k.p0 = k.t0 >> a.c.page_shift;
    return k;
}

// One 4-byte word to shared memory, asynchronously.
__device__ __forceinline__ void cp_async4(void* smem_dst, const void* gsrc) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(smem_dst)), "l"(gsrc) : "memory");
}

// CTAs of `kernel` that the current device holds when requests are few, its shared-memory limit
// (`most` bytes) raised at the device's first call; `state` is the kernel's own.
template <typename Kernel>
cudaError_t resident_ctas(PerDevice<int>& state, Kernel kernel, int most, int usual, int* ctas) {
    int device = 0;
    const cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    return cudaError_t(state.get(device, ctas, [&](int* n) -> int {
        int resident = 0;
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kernel, kAttendThreads, usual);
        *n = std::max(resident, 1) * num_sms();
        return e;
    }));
}

}  // namespace

}  // namespace clef
