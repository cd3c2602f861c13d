// Shared by the two attention kernels of the 4-bit memory cache: the requests of a call, its
// work items, and small matrix helpers.
#pragma once

#include "cache.h"
#include "common.cuh"
#include "kernels.h"

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

// 2^e, e clamped to the normal range.
__device__ __forceinline__ float pow2i(int e) {
    return __uint_as_float(uint32_t(min(max(e, -126), 127) + 127) << 23);
}

// The two elements of a 32-bit word as fp32.
__device__ __forceinline__ float2 unpack2(uint32_t w, int dtype) {
    if (dtype == 0) return make_float2(bf16_lo(w), bf16_hi(w));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// What a CTA needs to know of every request, in shared memory: the ends of its work items and
// of its partial rows as running sums, its keys, its first query row and its query rows.
struct Requests {
    int *items, *parts, *len, *q0, *nq;
    __device__ Requests(int* base, int n) : items(base), parts(base + n), len(base + 2 * n), q0(base + 3 * n), nq(base + 4 * n) {}
};

// r / share for query rows: share_inv = ceil(2^40 / share), exact while r * share < 2^40.
__device__ __forceinline__ int by_share(const CacheAttendArgs& a, int r) {
    return int((uint64_t(uint32_t(r)) * a.share_inv) >> 40);
}

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
    r.chunks = max(1, int((int64_t(r.len) + a.chunk - 1) / a.chunk));
    return r;
}

// Requests of up to so many query rows (queries x the query heads that share a key head) are
// the few-rows kernel's, the others the many-rows kernel's: by the request alone, so that a
// row's result does not depend on the batch.  128 requests x 1024 keys x 16 heads of 64: 24 rows
// take 89 us there and 137 here, 64 rows 219 there and 180 here.
__host__ __device__ constexpr int few_rows(int groups) { return groups == 1 ? 32 : 16; }

// Fills the tables; every thread of the CTA takes a run of neighbouring requests.  Requests of
// the other kernel have no items.
template <int G, bool MANY>
__device__ __forceinline__ void scan_requests(const CacheAttendArgs& a, const Requests& s, int rows_per_item) {
    __shared__ int tmp[2][kAttendWarps];
    const int per = (a.B + kAttendThreads - 1) / kAttendThreads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b0 = threadIdx.x * per, b1 = min(b0 + per, a.B);
    int items = 0, parts = 0;
    for (int b = b0; b < b1; ++b) {
        const Request r = request_of(a, b, blockIdx.x == 0);
        const int rows = r.nq * a.share;
        if ((rows > few_rows(G)) == MANY) items += r.chunks * ((rows + rows_per_item - 1) / rows_per_item) * a.kv_heads;
        parts += r.chunks > 1 ? r.chunks * r.nq * a.q_heads : 0;
        s.items[b] = items;
        s.parts[b] = parts;
        s.len[b] = r.len;
        s.q0[b] = r.q0;
        s.nq[b] = r.nq;
    }
    int ei = items, ep = parts;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int yi = __shfl_up_sync(0xffffffffu, ei, o), yp = __shfl_up_sync(0xffffffffu, ep, o);
        if (lane >= o) {
            ei += yi;
            ep += yp;
        }
    }
    if (lane == 31) {
        tmp[0][warp] = ei;
        tmp[1][warp] = ep;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        ei += tmp[0][w];
        ep += tmp[1][w];
    }
    for (int b = b0; b < b1; ++b) {
        s.items[b] += ei - items;
        s.parts[b] += ep - parts;
    }
    __syncthreads();
}

// A work item: a split of request b's keys, key/value head h, a block of its query rows.
struct Item {
    int b, h, split, row0, rows, t0, t1, ahead, p0;
};

template <int ROWS>
__device__ __forceinline__ Item item_of(const CacheAttendArgs& a, const Requests& s, int w) {
    Item k;
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s.items[mid] <= w)
            lo = mid + 1;
        else
            hi = mid;
    }
    k.b = lo;
    const int it = w - (lo ? s.items[lo - 1] : 0);
    const int len = s.len[lo], nq = s.nq[lo];
    const int n_rows = nq * a.share;
    const int n_blocks = (n_rows + ROWS - 1) / ROWS;
    const int rest = n_blocks == 1 ? it : it / n_blocks;
    k.row0 = (it - rest * n_blocks) * ROWS;
    k.split = rest / a.kv_heads;
    k.h = rest - k.split * a.kv_heads;
    k.rows = min(ROWS, n_rows - k.row0);
    k.t0 = k.split * a.chunk;
    k.t1 = min(k.t0 + a.chunk, len);
    k.ahead = len - nq;  // causal: query i sees keys 0 .. ahead + i
    if (a.causal) k.t1 = min(k.t1, k.ahead + by_share(a, k.row0 + k.rows - 1) + 1);
    k.p0 = k.t0 >> a.c.page_shift;
    return k;
}

// One 4-byte word to shared memory, asynchronously.
__device__ __forceinline__ void cp_async4(void* smem_dst, const void* gsrc) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(smem_dst)), "l"(gsrc) : "memory");
}

}  // namespace

}  // namespace clef
