// rope.cu — rotary positions of queries and keys, alone and on the way into a
// paged cache.
#include "rope.cuh"

#include "ptx.cuh"

namespace gbattn {
namespace {

// A pair (a, b) of a row's first rotary_dim elements at position t becomes
//   s (a cos w - b sin w),  s (b cos w + a sin w),   w = t inv_freq[i],
// with pairs (i, i + rotary_dim / 2), or (2i, 2i + 1) when interleaved; the inverse
// has -w.  The other elements are copied.
//
// Angles.  t inv_freq has up to 55 bits, and only its place within a turn counts,
// which fp32 would lose from t = 1000 on.  So each frequency becomes the fraction
// of a turn per position, 64 bits after the point (a CTA does it once, in fp64:
// off by 2^-53 for frequencies up to 1, by 2^-53 of the frequency above), and t times it
// modulo 2^64 is the angle, whatever t is, in one integer product.  Its upper 32 bits go to sin and cos: the fast ones
// for the 16-bit types (off by 2^-21 there, a rounding to fp16 by 2^-11 and more),
// sincospif for fp32.
//
// Bound by memory: a thread holds the cosines and sines of 16 bytes of pairs
// at one position and runs over rows (batch entries and heads) of it, so that
// they cost little; a row's 32-byte units are consecutive lanes'.  4 x 16 x 4096
// rows of 128, Q and K, bf16: 43.7 us (6.1 TB/s); 8 x 12 x 1024 of 64, half of it turned,
// fp16: 9.5 us; 15900 tokens of 16 + 2 x 4 heads into a cache: 35 us (5.6 TB/s); the
// 64 tokens of a decoding step, 32 + 2 x 8 heads: 3.0 us.
constexpr int kRopeThreads = 256;
constexpr int kBatch = 2;          // rows whose loads are in flight at a time (of 1, 2, 3, 4, 8 the fastest)
constexpr int kMaxPairs = 128;     // d <= 256

enum RopeType { kBf16, kHalf, kFloat };

template <RopeType kType>
constexpr int kVec = kType == kFloat ? 4 : 8;   // elements of 16 bytes

// 16 bytes to floats and back.
template <RopeType kType>
__device__ __forceinline__ void widen(const uint4& v, float (&f)[kVec<kType>]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kType == kFloat) {
            f[i] = __uint_as_float(w[i]);
        } else {
            f[2 * i] = h2lo_to_f32<kType == kHalf>(w[i]);
            f[2 * i + 1] = h2hi_to_f32<kType == kHalf>(w[i]);
        }
    }
}
template <RopeType kType>
__device__ __forceinline__ uint4 narrow(const float (&f)[kVec<kType>]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kType == kFloat) w[i] = __float_as_uint(f[i]);
        else w[i] = pack_h2<kType == kHalf>(f[2 * i], f[2 * i + 1]);   // the one rounding
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <RopeType kType, bool kInterleaved>
__device__ __forceinline__ void rotate(uint4& x, uint4& y, const float (&c)[kVec<kType>],
                                       const float (&s)[kVec<kType>]) {
    constexpr int V = kVec<kType>;
    float a[V], b[V];
    widen<kType>(x, a);
    widen<kType>(y, b);
    if constexpr (kInterleaved) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float p = a[2 * i], q = a[2 * i + 1], u = b[2 * i], v = b[2 * i + 1];
            a[2 * i] = p * c[i] - q * s[i];
            a[2 * i + 1] = q * c[i] + p * s[i];
            b[2 * i] = u * c[V / 2 + i] - v * s[V / 2 + i];
            b[2 * i + 1] = v * c[V / 2 + i] + u * s[V / 2 + i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float p = a[i], q = b[i];
            a[i] = p * c[i] - q * s[i];
            b[i] = q * c[i] + p * s[i];
        }
    }
    x = narrow<kType>(a);
    y = narrow<kType>(b);
}

// Token t's position from the packed offsets: request b's tokens are the last of
// its seq_lens[b] positions.  False for a token behind the last request.
__device__ __forceinline__ bool packed_position(const RopeParams& p, int t, int& pos) {
    int b = t < p.requests && p.cu[t] == t ? t : 0;   // a step of single tokens
    if (!(p.cu[b] <= t && t < p.cu[b + 1])) {
        int lo = 0, n = p.requests;   // first request whose tokens end after t
        while (n > 0) {
            const int half = n >> 1;
            if (p.cu[lo + half + 1] <= t) {
                lo += half + 1;
                n -= half + 1;
            } else {
                n = half;
            }
        }
        if (lo >= p.requests) return false;
        b = lo;
    }
    pos = static_cast<int>(static_cast<unsigned>(p.seq_lens[b]) - static_cast<unsigned>(p.cu[b + 1]) +
                           static_cast<unsigned>(t));
    return true;
}

template <RopeType kType, bool kInterleaved, bool kCache>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
    constexpr int V = kVec<kType>;
    constexpr int ES = 16 / V;
    grid_dep_wait();
    grid_dep_launch_dependents();   // the next kernel sets itself up meanwhile
    __shared__ unsigned long long s_step[kMaxPairs];
    const int half = p.rotary_dim / 2;
    for (int i = threadIdx.x; i < half; i += kRopeThreads) {
        const double turns = static_cast<double>(p.inv_freq[i]) * 0.15915494309189533577;   // 1 / (2 pi)
        s_step[i] = static_cast<unsigned long long>((turns - floor(turns)) * 18446744073709551616.0);
    }
    // this thread's unit of a row: V pairs, or 2 V elements to copy
    const int units = p.d / (2 * V);   // a power of two
    const int u = static_cast<int>(threadIdx.x) & (units - 1);
    const int tile = static_cast<int>(blockIdx.x) % p.tiles, chunk = static_cast<int>(blockIdx.x) / p.tiles;
    const int group = chunk / p.chunks;
    const long long n_wide = static_cast<long long>(tile) * (kRopeThreads / units) + threadIdx.x / units;
    const int n = static_cast<int>(n_wide);
    bool here = n_wide < p.N;
    const int turning = half / V;   // units with pairs
    const bool turns = u < turning;
    int col0, col1;
    if (!turns) {
        col0 = p.rotary_dim + (u - turning) * 2 * V;
        col1 = col0 + V;
    } else if (kInterleaved) {
        col0 = u * 2 * V;
        col1 = col0 + V;
    } else {
        col0 = u * V;
        col1 = col0 + half;
    }
    int pos = n;
    long long page = 0, row = 0;
    bool stored = true;   // K and V have a place
    if (here) {
        if (p.positions != nullptr) pos = p.positions[group * p.position_batch + n];
        else if (kCache) here = packed_position(p, n, pos);
        if (kCache) {
            const long long slot = p.slots[n];
            stored = here && slot >= 0 && slot < static_cast<long long>(p.num_pages) * p.page_size;
            // -1 marks a token without a slot; anything else out of range is an
            // error, as is a slot of a token that has no position
            if (!stored && slot != -1 && p.dev_status != nullptr)
                atomicCAS(p.dev_status, 0, static_cast<int>(ATTN_ERR_INVALID_ARG));
            page = static_cast<unsigned>(slot) / static_cast<unsigned>(p.page_size);
            row = static_cast<unsigned>(slot) - page * static_cast<unsigned>(p.page_size);
        }
    }
    __syncthreads();
    if (!here) return;
    float c[V], s[V];
    if (turns) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const unsigned long long phase =
                static_cast<unsigned long long>(static_cast<long long>(pos)) * s_step[u * V + i];
            const float turn = static_cast<float>(static_cast<int>(phase >> 32)) * 0x1p-32f;   // [-1/2, 1/2]
            if constexpr (kType == kFloat) sincospif(2.f * turn, &s[i], &c[i]);
            else __sincosf(6.2831853071795864769f * turn, &s[i], &c[i]);
            c[i] *= p.scaling;
            s[i] *= p.scaling * p.sign;
        }
    }
    const int per = p.heads[0] + p.heads[1] + p.heads[2];
    const int first = (chunk - group * p.chunks) * p.chunk_rows;
    const int last = min(first + p.chunk_rows, p.group_rows);
    for (int j0 = first; j0 < last; j0 += kBatch) {
        uint4 x[kBatch], y[kBatch];
        char* dst[kBatch];
        bool rot[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            dst[i] = nullptr;
            const int j = j0 + i;
            if (j >= last) continue;
            const int at = group * p.group_rows + j;
            const int b = at / per;
            int h = at - b * per, which = 0;
            if (h >= p.heads[0]) {
                h -= p.heads[0];
                which = 1;
                if (kCache && h >= p.heads[1]) {
                    h -= p.heads[1];
                    which = 2;
                }
            }
            if (kCache && which > 0 && !stored) continue;
            const RopeRows& r = p.rows[which];
            const char* src = static_cast<const char*>(r.src) +
                              (b * r.src_batch + h * r.src_head + n * r.src_token) * ES;
            x[i] = *reinterpret_cast<const uint4*>(src + col0 * ES);
            y[i] = *reinterpret_cast<const uint4*>(src + col1 * ES);
            dst[i] = static_cast<char*>(r.dst) +
                     (kCache && which > 0 ? page * r.dst_batch + h * r.dst_head + row * r.dst_token
                                          : b * r.dst_batch + h * r.dst_head + n * r.dst_token) * ES;
            rot[i] = turns && which < 2;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (dst[i] == nullptr) continue;
            if (rot[i]) rotate<kType, kInterleaved>(x[i], y[i], c, s);
            *reinterpret_cast<uint4*>(dst[i] + col0 * ES) = x[i];
            *reinterpret_cast<uint4*>(dst[i] + col1 * ES) = y[i];
        }
    }
}

template <bool kCache>
cudaError_t launch(RopeParams p, attn_dtype dtype, bool interleaved, cudaStream_t stream) {
    const int vec = dtype == ATTN_DTYPE_FP32 ? 4 : 8;
    const int tokens = kRopeThreads / (p.d / (2 * vec));   // of a CTA
    p.tiles = (p.N - 1) / tokens + 1;
    p.groups = p.position_batch != 0 ? p.B : 1;
    p.group_rows = p.B / p.groups * (p.heads[0] + p.heads[1] + p.heads[2]);
    // Rows of a thread: about four CTAs an SM, else as few sines as that allows (16
    // CTAs an SM, so one row a thread at 8 x 12 x 1024 x 64: 9.5 -> 16.4 us).
    const long long all = static_cast<long long>(p.tiles) * p.groups * p.group_rows;
    const long long want = all / (152 * 4);
    p.chunk_rows = static_cast<int>(want < 1 ? 1 : want > 16 ? 16 : want);
    p.chunks = (p.group_rows - 1) / p.chunk_rows + 1;
    const unsigned grid = static_cast<unsigned>(static_cast<long long>(p.tiles) * p.groups * p.chunks);
    auto go = [&](auto kern) { return launch_overlapped(kern, grid, kRopeThreads, 0, stream, p); };
    switch (dtype) {
        case ATTN_DTYPE_BF16:
            return interleaved ? go(rope_kernel<kBf16, true, kCache>) : go(rope_kernel<kBf16, false, kCache>);
        case ATTN_DTYPE_FP16:
            return interleaved ? go(rope_kernel<kHalf, true, kCache>) : go(rope_kernel<kHalf, false, kCache>);
        case ATTN_DTYPE_FP32:
            if constexpr (!kCache)
                return interleaved ? go(rope_kernel<kFloat, true, false>) : go(rope_kernel<kFloat, false, false>);
            break;
        default: break;
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, attn_dtype dtype, bool interleaved, cudaStream_t stream) {
    return launch<false>(p, dtype, interleaved, stream);
}

cudaError_t launch_append_rope(const RopeParams& p, attn_dtype dtype, bool interleaved, cudaStream_t stream) {
    return launch<true>(p, dtype, interleaved, stream);
}

}  // namespace gbattn
