// C ABI of the paged 4-bit memory cache: argument checks and launches.
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "../../include/clef_cache.h"
#include "cache.h"
#include "common.cuh"

using namespace clef;

namespace {

constexpr int64_t kInt32 = int64_t(1) << 31;

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

int check_cache(const clef_cache* c, CacheView* v) {
    if (!c) return CLEF_ERR_INVALID_ARGUMENT;
    if (c->head_dim != 64 && c->head_dim != 128) return CLEF_ERR_UNSUPPORTED_CONFIG;
    int shift = 4;
    while (shift < 8 && (1 << shift) != c->page) ++shift;
    if ((1 << shift) != c->page) return CLEF_ERR_UNSUPPORTED_CONFIG;
    if (c->heads < 1 || c->heads > 1024) return CLEF_ERR_UNSUPPORTED_CONFIG;
    if (c->n_pages < 1 || int64_t(c->n_pages) * c->page >= kInt32) return CLEF_ERR_UNSUPPORTED_CONFIG;
    v->data = static_cast<uint8_t*>(c->data);
    v->n_pages = c->n_pages;
    v->page = c->page;
    v->page_shift = shift;
    v->heads = c->heads;
    v->groups = c->head_dim / 64;
    return CLEF_OK;
}

int check_data(const clef_cache* c) {
    return !c->data || misaligned(c->data, 256) ? CLEF_ERR_INVALID_ARGUMENT : CLEF_OK;
}

bool bad_heads(const clef_cache* c, int head0, int n) { return head0 < 0 || n < 1 || n > c->heads || head0 > c->heads - n; }

// The kernels count tokens, table entries and slots in 32 bits, and step past the last one.
constexpr int64_t kMaxLength = kInt32 - 65536;
constexpr int64_t kMaxEntries = kInt32 / 2;

bool bad_table(const clef_cache* c, int B, int stride) {
    return B < 1 || stride < 1 || int64_t(stride) * c->page > kMaxLength || int64_t(B) * stride > kMaxEntries;
}

// Whether two runs of bytes share one.
bool overlap(const void* p, int64_t n, const void* q, int64_t m) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return n > 0 && m > 0 && (a <= b ? b - a < uintptr_t(n) : a - b < uintptr_t(m));
}

struct AttendSpace {
    int64_t rows = 0, lse = 0, off = 0, bytes = 0;  // partial rows; byte offsets; total
    AttendSpace(int64_t B, int64_t total_q, int64_t q_heads, int64_t dim, int64_t max_len) {
        const int64_t chunk = attend_chunk(1);  // the shortest splits of any call
        const int64_t chunks = (max_len + chunk - 1) / chunk;
        if (chunks <= 1 || total_q < 1) return;
        rows = total_q * q_heads * chunks;
        lse = rows * dim * 4;
        off = (lse + rows * 4 + 255) / 256 * 256;
        bytes = off + (B * 4 + 255) / 256 * 256;
    }
};

}  // namespace

#define CKC(x)                                        \
    do {                                              \
        if ((x) != cudaSuccess) return CLEF_ERR_CUDA; \
    } while (0)

extern "C" {

int clef_cache_size(const clef_cache* cache, size_t* bytes) {
    if (!bytes) return CLEF_ERR_INVALID_ARGUMENT;
    CacheView v;
    const int st = check_cache(cache, &v);
    if (st != CLEF_OK) return st;
    *bytes = size_t(v.n_pages) * v.heads * (v.page / 16) * (size_t(kPiece) * v.groups);
    return CLEF_OK;
}

int clef_cache_plan(const clef_cache* cache, int32_t B, int32_t* lengths, const int32_t* want, int32_t* block_table,
                    int32_t table_stride, int32_t* free_pages, int32_t* free_count, int32_t* cu_new, int32_t* slots,
                    int32_t n_slots, int32_t* flags, void* stream) {
    CacheView v;
    const int st = check_cache(cache, &v);
    if (st != CLEF_OK) return st;
    if (!lengths || !want || !block_table || !free_pages || !free_count || !cu_new || !flags || n_slots < 0 ||
        n_slots > kMaxEntries || (n_slots > 0 && !slots) || bad_table(cache, B, table_stride))
        return CLEF_ERR_INVALID_ARGUMENT;
    for (const void* p : {static_cast<const void*>(lengths), static_cast<const void*>(want),
                          static_cast<const void*>(block_table), static_cast<const void*>(free_pages),
                          static_cast<const void*>(free_count), static_cast<const void*>(cu_new),
                          static_cast<const void*>(slots), static_cast<const void*>(flags)})
        if (misaligned(p, 4)) return CLEF_ERR_INVALID_ARGUMENT;
    if (B > CLEF_CACHE_MAX_REQUESTS) return CLEF_ERR_UNSUPPORTED_CONFIG;
    CachePlanArgs a{};
    a.B = B; a.n_pages = v.n_pages; a.page_shift = v.page_shift; a.width = table_stride; a.n_slots = n_slots;
    a.lengths = lengths; a.want = want; a.table = block_table; a.free_pages = free_pages; a.free_count = free_count;
    a.cu = cu_new; a.slots = slots; a.flags = flags;
    CKC(launch_cache_plan(a, static_cast<cudaStream_t>(stream)));
    return CLEF_OK;
}

int clef_cache_append(const clef_cache* cache, int32_t n_tokens, int32_t head0, int32_t n_heads, int32_t dtype,
                      const void* k, int64_t k_row_stride, int64_t k_head_stride, const void* v, int64_t v_row_stride,
                      int64_t v_head_stride, const int32_t* slots, int32_t* flags, void* stream) {
    CacheRowsArgs a{};
    int st = check_cache(cache, &a.c);
    if (st != CLEF_OK) return st;
    if ((st = check_data(cache)) != CLEF_OK) return st;
    if (n_tokens < 0 || bad_heads(cache, head0, n_heads) || (dtype != CLEF_BF16 && dtype != CLEF_FP16) || !flags)
        return CLEF_ERR_INVALID_ARGUMENT;
    if (n_tokens == 0) return CLEF_OK;
    if (!k || !v || !slots || misaligned(k, 2) || misaligned(v, 2) || misaligned(slots, 4) || misaligned(flags, 4) ||
        k_row_stride < 0 || k_head_stride < 0 || v_row_stride < 0 || v_head_stride < 0)
        return CLEF_ERR_INVALID_ARGUMENT;
    a.n_tokens = n_tokens; a.head0 = head0; a.n_heads = n_heads; a.dtype = dtype;
    a.k = k; a.k_row = k_row_stride; a.k_head = k_head_stride;
    a.v = v; a.v_row = v_row_stride; a.v_head = v_head_stride;
    a.aligned = !misaligned(k, 16) && !misaligned(v, 16) &&
                (k_row_stride | k_head_stride | v_row_stride | v_head_stride) % 8 == 0;
    a.slots = slots; a.flags = flags;
    CKC(launch_cache_append(a, static_cast<cudaStream_t>(stream)));
    return CLEF_OK;
}

int clef_cache_read(const clef_cache* cache, int32_t n_tokens, int32_t head0, int32_t n_heads, int32_t dtype,
                    const int32_t* slots, void* k, void* v, int32_t* flags, void* stream) {
    CacheRowsArgs a{};
    int st = check_cache(cache, &a.c);
    if (st != CLEF_OK) return st;
    if ((st = check_data(cache)) != CLEF_OK) return st;
    if (n_tokens < 0 || bad_heads(cache, head0, n_heads) || dtype < CLEF_BF16 || dtype > CLEF_FP32 || !flags)
        return CLEF_ERR_INVALID_ARGUMENT;
    if (n_tokens == 0) return CLEF_OK;
    if (!k || !v || !slots || misaligned(k, 16) || misaligned(v, 16) || misaligned(slots, 4) || misaligned(flags, 4))
        return CLEF_ERR_INVALID_ARGUMENT;
    a.n_tokens = n_tokens; a.head0 = head0; a.n_heads = n_heads; a.dtype = dtype;
    a.out_k = k; a.out_v = v; a.slots = slots; a.flags = flags;
    CKC(launch_cache_read(a, static_cast<cudaStream_t>(stream)));
    return CLEF_OK;
}

int clef_cache_attend_workspace(const clef_cache* cache, int32_t B, int32_t total_q, int32_t q_heads, int32_t max_length,
                                size_t* bytes) {
    if (!bytes) return CLEF_ERR_INVALID_ARGUMENT;
    CacheView v;
    const int st = check_cache(cache, &v);
    if (st != CLEF_OK) return st;
    if (B < 1 || total_q < 0 || q_heads < 1 || max_length < 1 || max_length > kMaxLength) return CLEF_ERR_INVALID_ARGUMENT;
    *bytes = size_t(AttendSpace(B, total_q, q_heads, cache->head_dim, max_length).bytes);
    return CLEF_OK;
}

int clef_cache_attend(const clef_cache* cache, int32_t B, int32_t total_q, int32_t max_q, int32_t q_heads, int32_t head0,
                      int32_t kv_heads, int32_t dtype, const void* q, int64_t q_row_stride, int64_t q_head_stride,
                      const int32_t* cu_q, const int32_t* block_table, int32_t table_stride, const int32_t* lengths,
                      float scale, int32_t causal, void* out, float* lse, int32_t* flags, void* workspace,
                      size_t workspace_bytes, void* stream) {
    CacheAttendArgs a{};
    int st = check_cache(cache, &a.c);
    if (st != CLEF_OK) return st;
    if ((st = check_data(cache)) != CLEF_OK) return st;
    if (bad_heads(cache, head0, kv_heads) || q_heads < 1 || q_heads % kv_heads || (dtype != CLEF_BF16 && dtype != CLEF_FP16) ||
        total_q < 0 || max_q < 0 || max_q > total_q || bad_table(cache, B, table_stride) || !std::isfinite(scale) ||
        (causal != 0 && causal != 1) || !flags)
        return CLEF_ERR_INVALID_ARGUMENT;
    if (B > CLEF_CACHE_MAX_REQUESTS) return CLEF_ERR_UNSUPPORTED_CONFIG;
    if (max_q == 0) return CLEF_OK;
    if (!q || !cu_q || !block_table || !lengths || !out || misaligned(q, 4) || misaligned(out, 4) || q_row_stride < 0 ||
        q_head_stride < 0 || q_row_stride % 2 || q_head_stride % 2 || misaligned(workspace, 256) || misaligned(cu_q, 4) ||
        misaligned(block_table, 4) || misaligned(lengths, 4) || misaligned(lse, 4) || misaligned(flags, 4))
        return CLEF_ERR_INVALID_ARGUMENT;
    const int64_t max_len = int64_t(table_stride) * cache->page;
    const AttendSpace sp(B, total_q, q_heads, cache->head_dim, max_len);
    // items, query rows x heads and partial rows are counted in 32 bits on the GPU, which rounds them up
    // to blocks of rows and looks a grid of items ahead
    a.chunk = attend_chunk(kv_heads);
    const int64_t chunks = (max_len + a.chunk - 1) / a.chunk;
    if (sp.rows >= kInt32 || chunks * (int64_t(max_q) * (q_heads / kv_heads) / 8 + 1) * kv_heads * B > kMaxLength ||
        int64_t(max_q) * q_heads > kMaxLength)
        return CLEF_ERR_UNSUPPORTED_CONFIG;
    if (sp.bytes > 0 && !workspace) return CLEF_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < size_t(sp.bytes)) return CLEF_ERR_WORKSPACE_TOO_SMALL;
    // several CTAs read a row of queries, and at different times
    const int64_t n_rows = int64_t(total_q) * q_heads, out_bytes = 2 * n_rows * cache->head_dim;
    const __int128 q_span = 2 * (__int128(total_q - 1) * q_row_stride + __int128(q_heads - 1) * q_head_stride + cache->head_dim);
    const int64_t q_bytes = int64_t(std::min(q_span, __int128(INT64_MAX)));
    if (overlap(q, q_bytes, out, out_bytes) ||
        (lse && (overlap(lse, 4 * n_rows, q, q_bytes) || overlap(lse, 4 * n_rows, out, out_bytes))))
        return CLEF_ERR_INVALID_ARGUMENT;
    a.B = B; a.total_q = total_q; a.max_q = max_q; a.q_heads = q_heads; a.head0 = head0; a.kv_heads = kv_heads;
    a.share = q_heads / kv_heads; a.by_share = row_divider(a.share);
    a.dtype = dtype; a.width = table_stride; a.causal = causal;
    a.q = q; a.q_row = q_row_stride; a.q_head = q_head_stride;
    a.cu_q = cu_q; a.table = block_table; a.lengths = lengths;
    a.scale_log2 = float(double(scale) * 1.4426950408889634);
    a.out = out; a.lse = lse; a.flags = flags;
    if (sp.bytes > 0) {
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        a.part_o = reinterpret_cast<float*>(ws);
        a.part_lse = reinterpret_cast<float*>(ws + sp.lse);
        a.part_off = reinterpret_cast<int32_t*>(ws + sp.off);
    }
    a.part_rows = sp.rows;
    a.max_chunks = int(chunks);
    CKC(launch_cache_attend(a, static_cast<cudaStream_t>(stream)));
    return CLEF_OK;
}

int clef_cache_status(int32_t* flags, void* stream) {
    if (!flags || misaligned(flags, 4)) return CLEF_ERR_INVALID_ARGUMENT;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int h = 0;
    CKC(cudaMemcpyAsync(&h, flags, 4, cudaMemcpyDeviceToHost, st));
    CKC(cudaStreamSynchronize(st));
    if (h != 0) CKC(cudaMemsetAsync(flags, 0, 4, st));
    if (h & kFlagTimeout) return CLEF_ERR_DEVICE_TIMEOUT;
    if (h & kFlagBounds) return CLEF_ERR_DEVICE_BOUNDS;
    if (h & kFlagPages) return CLEF_ERR_NO_PAGES;
    return CLEF_OK;
}

}  // extern "C"
