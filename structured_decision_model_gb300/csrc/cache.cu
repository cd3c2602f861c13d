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

namespace {

// Byte of a token's 32 code bytes (one group) inside the 512 bytes of a 16-token piece.
__device__ __forceinline__ int key_byte(int r, int j) {
    return (r & 7) * 64 + (j & 7) / 2 * 16 + (j >> 3) * 4 + (j & 1) * 2 + (r >> 3);
}
__device__ __forceinline__ int value_byte(int r, int j) {
    return (j & 7) * 64 + (r & 7) / 2 * 16 + (j >> 3) * 4 + (r & 1) * 2 + (r >> 3);
}

template <int T>
__device__ __forceinline__ float to_f32(uint16_t x) {
    if (T == 0) return bf16_to_float(x);
    return __half2float(__ushort_as_half(x));
}

// Eight values of a row as fp32.
template <int T>
__device__ __forceinline__ void load8(float (&x)[8], const uint16_t* p) {
    uint16_t h[8];
    if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[2 * i] = uint16_t(ws[i] & 0xffff);
            h[2 * i + 1] = uint16_t(ws[i] >> 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = __ldg(p + i);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32<T>(h[i]);
}

// Minimum / maximum that keep a NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Quantises the 64 values that 8 neighbouring lanes hold (8 each).  Returns this lane's
// four code bytes: bytes 4 * (lane & 1) .. + 3 of run (lane & 7) / 2; sm gets the group's
// scale and minimum (bf16, low and high half).
__device__ __forceinline__ uint32_t quantise(const float (&x)[8], uint32_t* sm) {
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = min_nan(lo, x[i]);
        hi = max_nan(hi, x[i]);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const float m = bf16_to_float(float_to_bf16(lo));
    const float s = bf16_to_float(float_to_bf16(__fdiv_rn(fmaxf(hi - m, 0.f), 15.f)));
    const bool bad = !(fabsf(s) < INFINITY && fabsf(m) < INFINITY);
    *sm = bad ? 0x7FC07FC0u : uint32_t(float_to_bf16(s)) | uint32_t(float_to_bf16(m)) << 16;
    uint32_t w[2] = {0, 0};  // one code a byte
    if (!bad && s != 0.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float c = fminf(fmaxf(rintf(__fdiv_rn(x[i] - m, s)), 0.f), 15.f);
            w[i >> 2] |= uint32_t(c) << (8 * (i & 3));
        }
    }
    // an even lane holds the low halves of the run's bytes, its odd neighbour the high ones
    const bool odd = threadIdx.x & 1;
    const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 1);
    return odd ? other | w[1] << 4 : w[0] | other << 4;
}

}  // namespace

constexpr int kRowsWarps = 8;

// One warp: 16 consecutive rows of one head.  Eight lanes hold the 64 values of a row's
// group, so a warp load brings four rows of 128 contiguous bytes.
template <int T>
__global__ void __launch_bounds__(32 * kRowsWarps) cache_append_kernel(const CacheRowsArgs a) {
    griddep_wait();
    griddep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = blockIdx.y * kRowsWarps + warp;
    if (head >= a.n_heads) return;
    const int64_t i0 = int64_t(blockIdx.x) * 16;
    const int total = a.c.n_pages << a.c.page_shift;
    for (int k = 0; k < 4; ++k) {
        const int64_t i = i0 + k * 4 + lane / 8;
        int slot = i < a.n_tokens ? a.slots[i] : -1;
        if (slot >= total) {
            if ((lane & 7) == 0) atomicOr(a.flags, kFlagBounds);
            slot = -1;
        }
        const int64_t row = slot >= 0 ? i : 0;
        const int r = slot & 15;
        uint8_t* piece = a.c.data + ((int64_t(slot >> a.c.page_shift) * a.c.heads + a.head0 + head) *
                                         (a.c.page >> 4) + ((slot & (a.c.page - 1)) >> 4)) * (kPiece * a.c.groups);
        for (int g = 0; g < a.c.groups; ++g) {
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const uint16_t* src = static_cast<const uint16_t*>(kv ? a.v : a.k);
                float x[8];
                load8<T>(x, src + row * (kv ? a.v_row : a.k_row) + head * (kv ? a.v_head : a.k_head) + g * 64 +
                                (lane & 7) * 8);
                uint32_t sm;
                const uint32_t bytes = quantise(x, &sm);
                if (slot < 0) continue;
                uint8_t* codes = piece + (kv * a.c.groups + g) * 512;
                const int j0 = (lane & 7) / 2 * 8 + (lane & 1) * 4;
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    codes[kv ? value_byte(r, j0 + b) : key_byte(r, j0 + b)] = uint8_t(bytes >> (8 * b));
                if ((lane & 7) == 0)
                    *reinterpret_cast<uint32_t*>(piece + a.c.groups * 1024 + (r * a.c.groups + g) * 8 + kv * 4) = sm;
            }
        }
    }
}

// One warp: 4 rows at a time of one head; a lane makes 8 values of a row.
template <int T>
__global__ void __launch_bounds__(32 * kRowsWarps) cache_read_kernel(const CacheRowsArgs a) {
    griddep_wait();
    griddep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = blockIdx.y * kRowsWarps + warp;
    if (head >= a.n_heads) return;
    const int total = a.c.n_pages << a.c.page_shift;
    const int run = (lane & 7) / 2, shift = (lane & 1) * 4;
    for (int k = 0; k < 4; ++k) {
        const int64_t i = int64_t(blockIdx.x) * 16 + k * 4 + lane / 8;
        if (i >= a.n_tokens) continue;
        const int slot = a.slots[i];
        if (slot >= total && (lane & 7) == 0) atomicOr(a.flags, kFlagBounds);
        const bool live = slot >= 0 && slot < total;
        const int r = slot & 15;
        const uint8_t* piece = a.c.data + (live ? ((int64_t(slot >> a.c.page_shift) * a.c.heads + a.head0 + head) *
                                                       (a.c.page >> 4) + ((slot & (a.c.page - 1)) >> 4)) *
                                                      (kPiece * a.c.groups) : 0);
        for (int g = 0; g < a.c.groups; ++g) {
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                float x[8] = {};
                if (live) {
                    const uint8_t* codes = piece + (kv * a.c.groups + g) * 512;
                    const uint32_t sm = *reinterpret_cast<const uint32_t*>(piece + a.c.groups * 1024 +
                                                                           (r * a.c.groups + g) * 8 + kv * 4);
#pragma unroll
                    for (int b = 0; b < 8; ++b) {
                        const int c = codes[kv ? value_byte(r, run * 8 + b) : key_byte(r, run * 8 + b)] >> shift & 15;
                        x[b] = fmaf(bf16_lo(sm), float(c), bf16_hi(sm));
                    }
                }
                void* base = kv ? a.out_v : a.out_k;
                const int64_t at = (i * a.n_heads + head) * (64 * a.c.groups) + g * 64 + (lane & 7) * 8;
                if (T == 2) {
                    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
                    p[0] = make_float4(x[0], x[1], x[2], x[3]);
                    p[1] = make_float4(x[4], x[5], x[6], x[7]);
                } else {
                    uint32_t w[4];
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        if (T == 0) {
                            w[b] = pack_bf16(x[2 * b], x[2 * b + 1]);
                        } else {
                            const __half2 h = __floats2half2_rn(x[2 * b], x[2 * b + 1]);
                            w[b] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                    }
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
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
