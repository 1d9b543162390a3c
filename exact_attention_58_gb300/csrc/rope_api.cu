// rope_api.cu — C entry points of rotary positions declared in include/gbattn.h:
// argument validation.  Nothing here allocates, frees or synchronises.
#include <cmath>

#include "rope.cuh"

namespace gbattn {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

attn_status from_cuda(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

// A stride in elements of `es` bytes: a multiple of 16 bytes, positive (or, of what
// is only read, zero).  A dimension of one element has no stride.
bool stride_ok(long long stride, long long extent, int es, bool read_only) {
    return extent == 1 || ((stride > 0 || (read_only && stride == 0)) && stride % (16 / es) == 0 &&
                           stride < (1ll << 39));
}

attn_status check_rotation(int d, int rotary_dim, float scaling, attn_dtype dtype, bool f32) {
    if (dtype != ATTN_DTYPE_BF16 && dtype != ATTN_DTYPE_FP16 && !(f32 && dtype == ATTN_DTYPE_FP32))
        return dtype == ATTN_DTYPE_FP32 || dtype == ATTN_DTYPE_FP8_E4M3 ? ATTN_ERR_UNSUPPORTED
                                                                       : ATTN_ERR_INVALID_ARG;
    if (d != 64 && d != 128 && d != 256) return ATTN_ERR_UNSUPPORTED;
    if (rotary_dim < 1 || rotary_dim > d) return ATTN_ERR_INVALID_ARG;
    if (rotary_dim % 16 != 0) return ATTN_ERR_UNSUPPORTED;
    return std::isfinite(scaling) ? ATTN_OK : ATTN_ERR_INVALID_ARG;
}

}  // namespace
}  // namespace gbattn

using namespace gbattn;

extern "C" {

attn_status attn_rope(const void* Q, const void* K, void* Q_out, void* K_out, const float* inv_freq,
                      const int32_t* positions, int B, int H, int H_k, int N, int d, int rotary_dim,
                      attn_dtype dtype, int64_t q_batch_stride, int64_t q_head_stride,
                      int64_t q_token_stride, int64_t k_batch_stride, int64_t k_head_stride,
                      int64_t k_token_stride, int64_t q_out_batch_stride, int64_t q_out_head_stride,
                      int64_t q_out_token_stride, int64_t k_out_batch_stride,
                      int64_t k_out_head_stride, int64_t k_out_token_stride,
                      int64_t position_batch_stride, float scaling, int interleaved, int inverse,
                      void* stream) {
    if (!Q || !Q_out || !inv_freq || B < 1 || H < 1 || H_k < 0 || N < 1) return ATTN_ERR_INVALID_ARG;
    if (H_k > 0 && (!K || !K_out)) return ATTN_ERR_INVALID_ARG;
    const attn_status st = check_rotation(d, rotary_dim, scaling, dtype, true);
    if (st != ATTN_OK) return st;
    if (N > (1 << 30) || (static_cast<long long>(H) + H_k) * B >= (1ll << 31) ||
        (static_cast<long long>(H) + H_k) * B * (N / 8 + 1ll) >= (1ll << 31))
        return ATTN_ERR_UNSUPPORTED;
    if (positions && B > 1 && position_batch_stride != 0 && position_batch_stride < N) return ATTN_ERR_INVALID_ARG;
    RopeParams p{};
    const int es = dtype == ATTN_DTYPE_FP32 ? 4 : 2;
    p.rows[0] = RopeRows{Q, Q_out, q_batch_stride, q_head_stride, q_token_stride,
                         q_out_batch_stride, q_out_head_stride, q_out_token_stride};
    p.rows[1] = RopeRows{K, K_out, k_batch_stride, k_head_stride, k_token_stride,
                         k_out_batch_stride, k_out_head_stride, k_out_token_stride};
    const int heads[2] = {H, H_k};
    for (int i = 0; i < (H_k > 0 ? 2 : 1); ++i) {
        RopeRows& r = p.rows[i];
        if (!stride_ok(r.src_batch, B, es, true) || !stride_ok(r.src_head, heads[i], es, true) ||
            !stride_ok(r.src_token, N, es, true) || !stride_ok(r.dst_batch, B, es, false) ||
            !stride_ok(r.dst_head, heads[i], es, false) || !stride_ok(r.dst_token, N, es, false) ||
            !aligned(r.src, 16) || !aligned(r.dst, 16))
            return ATTN_ERR_MISALIGNED;
    }
    if (!aligned(inv_freq, 4) || !aligned(positions, 4)) return ATTN_ERR_MISALIGNED;
    p.inv_freq = inv_freq;
    p.positions = positions;
    p.position_batch = positions && B > 1 ? position_batch_stride : 0;
    p.heads[0] = H;
    p.heads[1] = H_k;
    p.B = B;
    p.N = N;
    p.d = d;
    p.rotary_dim = rotary_dim;
    p.scaling = scaling;
    p.sign = inverse ? -1.f : 1.f;
    return from_cuda(launch_rope(p, dtype, interleaved != 0, static_cast<cudaStream_t>(stream)));
}

attn_status attn_cache_append_rope(const void* Q, const void* K, const void* V, void* Q_out,
                                   void* k_cache, void* v_cache, const int64_t* slots,
                                   const float* inv_freq, const int32_t* positions,
                                   const int32_t* cu_seqlens_q, const int32_t* seq_lens, int B, int T,
                                   int H, int H_kv, int d, int rotary_dim, attn_dtype dtype,
                                   int64_t q_token_stride, int64_t q_head_stride,
                                   int64_t kv_token_stride, int64_t kv_head_stride,
                                   int64_t q_out_token_stride, int64_t q_out_head_stride,
                                   int num_pages, int page_size, int64_t cache_page_stride,
                                   int64_t cache_head_stride, int64_t cache_token_stride,
                                   float scaling, int interleaved, int* dev_status, void* stream) {
    if (!Q || !K || !V || !Q_out || !k_cache || !v_cache || !slots || !inv_freq) return ATTN_ERR_INVALID_ARG;
    if (T < 1 || H < 1 || H_kv < 1 || num_pages < 1 || page_size < 1) return ATTN_ERR_INVALID_ARG;
    if (!positions && (!cu_seqlens_q || !seq_lens || B < 1)) return ATTN_ERR_INVALID_ARG;
    const attn_status st = check_rotation(d, rotary_dim, scaling, dtype, false);
    if (st != ATTN_OK) return st;
    if (page_size % 8 != 0 || static_cast<long long>(num_pages) * page_size >= (1ll << 31))
        return ATTN_ERR_UNSUPPORTED;
    const long long rows = static_cast<long long>(H) + 2ll * H_kv;
    if (T > (1 << 30) || (!positions && B > (1 << 30)) || rows >= (1ll << 31) || rows * (T / 8 + 1ll) >= (1ll << 31))
        return ATTN_ERR_UNSUPPORTED;
    if (!stride_ok(q_token_stride, T, 2, true) || !stride_ok(q_head_stride, H, 2, true) ||
        !stride_ok(kv_token_stride, T, 2, true) || !stride_ok(kv_head_stride, H_kv, 2, true) ||
        !stride_ok(q_out_token_stride, T, 2, false) || !stride_ok(q_out_head_stride, H, 2, false) ||
        !stride_ok(cache_page_stride, num_pages, 2, false) || !stride_ok(cache_head_stride, H_kv, 2, false) ||
        !stride_ok(cache_token_stride, page_size, 2, false))
        return ATTN_ERR_MISALIGNED;
    if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(Q_out, 16) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(slots, 8) || !aligned(inv_freq, 4) || !aligned(positions, 4) ||
        !aligned(cu_seqlens_q, 4) || !aligned(seq_lens, 4))
        return ATTN_ERR_MISALIGNED;
    RopeParams p{};
    p.rows[0] = RopeRows{Q, Q_out, 0, q_head_stride, q_token_stride, 0, q_out_head_stride, q_out_token_stride};
    p.rows[1] = RopeRows{K, k_cache, 0, kv_head_stride, kv_token_stride,
                         cache_page_stride, cache_head_stride, cache_token_stride};
    p.rows[2] = p.rows[1];
    p.rows[2].src = V;
    p.rows[2].dst = v_cache;
    p.inv_freq = inv_freq;
    p.positions = positions;
    p.heads[0] = H;
    p.heads[1] = p.heads[2] = H_kv;
    p.B = 1;
    p.N = T;
    p.d = d;
    p.rotary_dim = rotary_dim;
    p.scaling = scaling;
    p.sign = 1.f;
    p.slots = slots;
    p.cu = cu_seqlens_q;
    p.seq_lens = seq_lens;
    p.dev_status = dev_status;
    p.requests = B;
    p.num_pages = num_pages;
    p.page_size = page_size;
    return from_cuda(launch_append_rope(p, dtype, interleaved != 0, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
