// paged_cache.h — parameters and launches of the cache-append and page-table
// kernels (paged_cache.cu, paged_cache_fp8.cu).
#pragma once

#include "internal.h"

namespace gbattn {

struct AppendParams {
    const uint16_t* K;          // [T][Hkv][d], 16-bit elements
    const uint16_t* V;
    uint16_t* k_cache;          // [num_pages][Hkv][page_size][d]
    uint16_t* v_cache;
    const int64_t* slots;       // [T]
    int* dev_status;
    int T, Hkv, d;
    int num_pages, page_size;
    long long token_stride, head_stride;   // of K and V, in elements
    long long cache_page_stride, cache_head_stride, cache_token_stride;
};

struct TableParams {
    const int32_t* cached_lens;   // [B]
    const int32_t* new_lens;      // [B]
    int32_t* page_table;          // [B][max_pages]
    const int32_t* free_pages;    // [free_capacity]
    const int32_t* num_free;      // [1]
    int32_t* cu_seqlens_q;        // [B + 1]
    int32_t* seq_lens;            // [B]
    int64_t* slots;               // [max_tokens]
    int32_t* pages_taken;         // [1]
    int* dev_status;
    int B, max_pages, page_size, max_tokens, free_capacity;
};

// K (0) and V (1) rows into a cache of e4m3 with a scale per page and head.
struct AppendFp8Params {
    const uint16_t* x[2];       // [T][Hkv][d], 16-bit elements
    uint8_t* cache[2];          // [num_pages][Hkv][page_size][d]
    float* scale[2];            // [num_pages][Hkv]
    const int64_t* slots;       // [T]
    int* dev_status;
    int T, Hkv, d;
    int num_pages, page_size;
    int tile_tokens;            // tokens whose runs are one CTA's (set by the launch)
    long long token_stride, head_stride;   // of K and V, in elements
    long long cache_page_stride, cache_head_stride, cache_token_stride;
};

// Requests of one page-table call: two ints each in shared memory.
constexpr int kMaxTableRequests = 16384;

cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t stream);
cudaError_t launch_append_fp8(const AppendFp8Params& p, bool f16, cudaStream_t stream);
cudaError_t launch_page_table(const TableParams& p, cudaStream_t stream);

}  // namespace gbattn
