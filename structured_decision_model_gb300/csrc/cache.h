// Launchers of the 4-bit memory cache's kernels (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace clef {

constexpr int kCacheMaxRequests = 1024;
constexpr int kFlagPages = 1 << 2;  // flags bit beside those of common.cuh: the free pages ran out
constexpr int kPiece = 1152;  // bytes of 16 tokens, 64 values: key codes, value codes, scales and minima

// A cache as the kernels see it.
struct CacheView {
    uint8_t* data;
    int n_pages, page, page_shift;  // tokens a page and its logarithm
    int heads, groups;              // head size / 64
};

struct CachePlanArgs {
    int B, n_pages, page_shift, width, n_slots;
    int32_t* lengths; const int32_t* want; int32_t* table; int32_t* free_pages; int32_t* free_count;
    int32_t* cu; int32_t* slots; int32_t* flags;
};

struct CacheRowsArgs {
    CacheView c;
    int n_tokens, head0, n_heads, dtype;
    bool aligned;                          // rows and heads start on 16 bytes
    const void* k; int64_t k_row, k_head;  // strides in elements
    const void* v; int64_t v_row, v_head;
    void* out_k; void* out_v;              // read back
    const int32_t* slots; int32_t* flags;
};

// Division of query rows by the query heads that share a key head: r / share = r mul >> shift, exact
// for every 0 <= r < 2^31.  With 2^(l - 1) < share <= 2^l, mul = ceil(2^(31 + l) / share) is over by
// less than share / share <= 2^l / share, so r mul / 2^(31 + l) is over by less than 1 / share; mul is
// below 2^32 and the product below 2^63.
struct RowDivider {
    uint32_t mul, shift;
    __host__ __device__ int operator()(int r) const { return int((uint64_t(uint32_t(r)) * mul) >> shift); }
};
inline RowDivider row_divider(int share) {
    uint32_t l = 0;
    while ((int64_t(1) << l) < share) ++l;
    return {uint32_t(((uint64_t(1) << (31 + l)) + share - 1) / share), 31 + l};
}

struct CacheAttendArgs {
    CacheView c;
    int B, total_q, max_q, q_heads, head0, kv_heads, share, dtype, width, causal;
    const void* q; int64_t q_row, q_head;
    const int32_t* cu_q; const int32_t* table; const int32_t* lengths;
    RowDivider by_share;
    float scale_log2;
    void* out; float* lse; int32_t* flags;
    float* part_o; float* part_lse; int32_t* part_off;  // split partials, their row offset per request
    int64_t part_rows;  // partial rows that the workspace holds
    int chunk, max_chunks;  // keys of a split, most splits of a request
};

// Keys of one split of a request's memory.  It goes by the key/value heads of the call alone,
// so that a row's result does not depend on the batch.  Long splits spend less on their ends,
// short ones spread a lone request over the GPU.  With 1024, 2048 and 4096 keys a split, bf16:
//   one token of 64 requests of 156-16384 keys, 8 heads of 128     54, 52 and 49 us
//   one token over 131072 keys, 16 heads of 64                     43, 40 and 38 us
//   64 queries x 8 requests x 16384 keys, 16 heads of 64          205, 193 and 182 us
//   96 queries x 4 requests x 8192 keys, 8 heads of 128, causal   287, 268 and 334 us
// so 2048 from 8 heads on.  One token over 131001 keys x 2 heads takes 16.5, 15.3 and 18.0 us
// with 512, 1024 and 2048: 1024 below 8 heads.
constexpr int kAttendMaxChunk = 2048;
__host__ __device__ inline int attend_chunk(int kv_heads) { return kv_heads >= 8 ? kAttendMaxChunk : 1024; }

cudaError_t launch_cache_plan(const CachePlanArgs& a, cudaStream_t s);
cudaError_t launch_cache_append(const CacheRowsArgs& a, cudaStream_t s);
cudaError_t launch_cache_read(const CacheRowsArgs& a, cudaStream_t s);
cudaError_t launch_cache_attend(const CacheAttendArgs& a, cudaStream_t s);
cudaError_t launch_cache_attend_rows(const CacheAttendArgs& a, cudaStream_t s);  // its requests of many query rows


}  // namespace clef
