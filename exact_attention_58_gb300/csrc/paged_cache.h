// paged_cache.h — parameters and launches of the cache-append and page-table
// kernels (paged_cache.cu).
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

// Requests of one page-table call: two ints each in shared memory.
constexpr int kMaxTableRequests = 16384;

cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t stream);
cudaError_t launch_page_table(const TableParams& p, cudaStream_t stream);

}  // namespace gbattn
