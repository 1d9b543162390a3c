// rope.cuh — rotary positions: parameters shared by the C entry points and the
// kernel.
#pragma once

#include "internal.h"

namespace gbattn {

// Rows of d elements with strides in elements.
struct RopeRows {
    const void* src;
    void* dst;
    long long src_batch, src_head, src_token;
    long long dst_batch, dst_head, dst_token;   // of a cache: page, head, row of a page
};

struct RopeParams {
    RopeRows rows[3];          // Q, K and, on the way into a cache, V (which is not rotated)
    const float* inv_freq;     // [rotary_dim / 2]
    const int32_t* positions;  // [N], or one row of them per batch entry; nullptr: 0, 1, ... (or from cu)
    long long position_batch;
    int heads[3];
    int B, N, d, rotary_dim;
    float scaling, sign;       // factor of the rotated part; -1: the inverse rotation
    // into a cache (B = 1, N tokens)
    const int64_t* slots;
    const int32_t* cu;         // request offsets and lengths, where positions is nullptr
    const int32_t* seq_lens;
    int* dev_status;
    int requests, num_pages, page_size;
    // set by the launch
    int tiles, groups, group_rows, chunks, chunk_rows;
};

// Launches (validated arguments only).
cudaError_t launch_rope(const RopeParams& p, attn_dtype dtype, bool interleaved, cudaStream_t stream);
cudaError_t launch_append_rope(const RopeParams& p, attn_dtype dtype, bool interleaved, cudaStream_t stream);

}  // namespace gbattn
