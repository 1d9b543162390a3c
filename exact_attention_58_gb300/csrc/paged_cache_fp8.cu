// paged_cache_fp8.cu — writing new rows into a paged key/value cache held in
// e4m3, with one scale per page and head.
#include "fp8.cuh"
#include "paged_cache.h"
#include "ptx.cuh"

namespace gbattn {
namespace {

// A block (a page's rows of one head of K or V) stands for e4m3 x 2^e with the
// smallest e for which its largest value fits, so rounding to e4m3's four
// significant bits is the only rounding: the scale, a power of two, adds none.  New rows that
// exceed what the block's scale can hold raise e: the rows that it held are
// rounded again, by a power of two, which loses only what falls below e4m3's normal numbers.
// A row written to a page's row 0 starts the block anew.
//
// A step's new rows of one page are a run of consecutive tokens.  A CTA takes the
// runs that begin in its share of the tokens, for one head of K or V, one after
// the other: its threads look at 128 tokens at once and mark where runs begin; then,
// run by run, it finds the largest value (the rows stay in registers, as far as they
// fit), the scale, and writes: one launch, no word between CTAs, and no atomics.
// Bound by issue for prompts (15900 tokens of 8 heads, d = 128: 19.8 us, 4.9 TB/s); for
// single tokens, where each CTA has one row, by the chain slot -> scale and row ->
// store (64 tokens 4.2 us).  Eight CTAs an SM (64 registers a thread): with 95
// registers and five of them 22.3 and 4.6 us.
constexpr int kThreads = 128;
constexpr int kChunk = 64;  // tokens whose runs are begun at a time: half of what is looked at
constexpr int kKept = 8;    // 16-byte pieces of the run's rows that a thread keeps

template <bool kF16>
__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = h2lo_to_f32<kF16>(w[i]);
        f[2 * i + 1] = h2hi_to_f32<kF16>(w[i]);
    }
}

// The larger of two pairs of 16-bit values, element by element; of a NaN and a number
// the number.
template <bool kF16>
__device__ __forceinline__ uint32_t max_h2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (kF16) asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 16 e4m3 values times `factor`, rounded again.
__device__ __forceinline__ uint4 round_again(const uint4& v, float factor) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = e4m3x2_to_f16x2(w[i] & 0xffffu), hi = e4m3x2_to_f16x2(w[i] >> 16);
        o[i] = pack_e4m3x4(f16lo_to_f32(lo) * factor, f16hi_to_f32(lo) * factor, f16lo_to_f32(hi) * factor,
                           f16hi_to_f32(hi) * factor);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <bool kF16>
__global__ void __launch_bounds__(kThreads, 8) append_fp8_kernel(const __grid_constant__ AppendFp8Params p) {
    grid_dep_wait();
    grid_dep_launch_dependents();   // the next kernel sets itself up meanwhile
    __shared__ int s_slot[kThreads];
    __shared__ uint32_t s_break[kThreads / 32];   // tokens that do not continue a run
    __shared__ uint32_t s_valid[kThreads / 32];
    __shared__ uint32_t s_amax[kThreads / 32];
    __shared__ int s_len;
    const int tid = static_cast<int>(threadIdx.x);
    const int which = static_cast<int>(blockIdx.x & 1);   // K, V
    const int unit = static_cast<int>(blockIdx.x >> 1);
    const int tile = unit / p.Hkv, h = unit - tile * p.Hkv;
    const long long slots_all = static_cast<long long>(p.num_pages) * p.page_size;
    const unsigned size = static_cast<unsigned>(p.page_size);
    const int t_end = static_cast<int>(min(static_cast<long long>(p.T), (tile + 1ll) * p.tile_tokens));
    const int vecs = p.d / 8;                  // 16-byte pieces of a row
    const int c = tid & (vecs - 1), r0 = tid / vecs, rows_at_once = kThreads / vecs;
    const uint16_t* const src_head = (which ? p.x[1] : p.x[0]) + h * p.head_stride + 8 * c;
    for (int base = tile * p.tile_tokens; base < t_end; base += kChunk) {
        const int t = base + tid;
        const long long slot_t = t < p.T ? p.slots[t] : -1;
        const long long before = t > 0 && t < p.T ? p.slots[t - 1] : -1;
        const bool valid = slot_t >= 0 && slot_t < slots_all;
        const unsigned row_t = static_cast<unsigned>(slot_t) % size;
        const bool cut = !valid || t == 0 || row_t == 0 || before != slot_t - 1;
        // A second run of a page, where the last token ahead that has a slot, within row_t
        // tokens, is of the page: left out and reported, or two CTAs would write one block.
        // (Found by the token's own thread here: a check run by run took 64 single tokens from
        // 4.2 to 4.5 us.)
        bool again = false;
        if (valid && cut) {
            long long ahead = before;
            const int most = min(static_cast<int>(row_t), t);
            auto none = [&]() { return static_cast<unsigned long long>(ahead) >= static_cast<unsigned long long>(slots_all); };
            for (int i = 2; none() && i <= most; i += 8) {
                long long more[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) more[k] = i + k <= most ? p.slots[t - i - k] : -1;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (none()) ahead = more[k];
            }
            again = static_cast<unsigned long long>(ahead - (slot_t - row_t)) < size;
        }
        // -1 marks a token without a slot; anything else out of range is an error
        if (((!valid && slot_t != -1) || again) && p.dev_status != nullptr)
            atomicCAS(p.dev_status, 0, static_cast<int>(ATTN_ERR_INVALID_ARG));
        const uint32_t breaks = __ballot_sync(0xffffffffu, cut), valids = __ballot_sync(0xffffffffu, valid && !again);
        __syncthreads();   // the chunk before is done with them
        s_slot[tid] = static_cast<int>(slot_t);
        if ((tid & 31) == 0) {
            s_break[tid >> 5] = breaks;
            s_valid[tid >> 5] = valids;
        }
        __syncthreads();
        // tokens of this chunk that begin a run, and (of all looked at) breaks
        const unsigned long long low = s_break[0] | static_cast<unsigned long long>(s_break[1]) << 32;
        const unsigned long long high = s_break[2] | static_cast<unsigned long long>(s_break[3]) << 32;
        unsigned long long begins = low & (s_valid[0] | static_cast<unsigned long long>(s_valid[1]) << 32);
        const int mine = min(kChunk, t_end - base);
        if (mine < 64) begins &= (1ull << mine) - 1;
        for (; begins != 0; begins &= begins - 1) {
            const int at = __ffsll(static_cast<long long>(begins)) - 1;
            const int first = base + at;
            const unsigned slot = static_cast<unsigned>(s_slot[at]);
            const unsigned page = slot / size;
            const int row0 = static_cast<int>(slot - page * size);
            // ---- the run's length: up to the next break ----
            const unsigned long long rest = at < 63 ? low >> (at + 1) : 0;
            int len = rest != 0 ? __ffsll(static_cast<long long>(rest))
                      : high != 0 ? 64 - at + __ffsll(static_cast<long long>(high)) - 1 : kThreads - at;
            if (rest == 0 && high == 0) {   // it goes on past what was looked at
                const int room = min(static_cast<int>(size) - row0, p.T - first);
                for (bool more = true; more;) {
                    if (tid == 0) s_len = room;
                    __syncthreads();
                    const int i = len + tid;
                    if (i < room && p.slots[first + i] != static_cast<long long>(slot) + i) atomicMin(&s_len, i);
                    __syncthreads();
                    more = s_len == room && len + kThreads < room;
                    len = more ? len + kThreads : s_len;
                    __syncthreads();
                }
            }
            float* const scale = (which ? p.scale[1] : p.scale[0]) + static_cast<size_t>(page) * p.Hkv + h;
            const uint32_t held = row0 > 0 ? __float_as_uint(*scale) : 0u;   // (asked for ahead of the rows)
            // ---- its largest value ----
            const uint16_t* const src = src_head + first * p.token_stride;
            uint4 kept[kKept];
            uint32_t amax = 0;   // two at a time, in the rows' type
            auto grow = [&](const uint4& v) {
                amax = max_h2<kF16>(max_h2<kF16>(max_h2<kF16>(amax, v.x & 0x7fff7fffu), v.y & 0x7fff7fffu),
                                    max_h2<kF16>(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
            };
#pragma unroll
            for (int i = 0; i < kKept; ++i) {
                const int r = r0 + i * rows_at_once;
                kept[i] = make_uint4(0u, 0u, 0u, 0u);
                if (r < len) kept[i] = *reinterpret_cast<const uint4*>(src + r * p.token_stride);
            }
#pragma unroll
            for (int i = 0; i < kKept; ++i) grow(kept[i]);
            for (int r = r0 + kKept * rows_at_once; r < len; r += rows_at_once)
                grow(*reinterpret_cast<const uint4*>(src + r * p.token_stride));
            const uint32_t warp_max = __reduce_max_sync(
                0xffffffffu, __float_as_uint(fmaxf(h2lo_to_f32<kF16>(amax), h2hi_to_f32<kF16>(amax))));
            if ((tid & 31) == 0) s_amax[tid >> 5] = warp_max;
            __syncthreads();
            uint32_t top = 0;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) top = max(top, s_amax[w]);
            // ---- the scale ----
            int e = fit_exponent(top), old = kLeastScale;
            if (row0 > 0) {
                old = scale_exponent(held);
                if (bad_scale(held) && tid == 0 && p.dev_status != nullptr)
                    atomicCAS(p.dev_status, 0, static_cast<int>(ATTN_ERR_INVALID_ARG));
                e = max(e, old);
            }
            // (every thread has read the old one: the barrier above)
            if (tid == 0) *scale = exp2_int(e);
            // ---- rows of the block before ----
            uint8_t* const block = (which ? p.cache[1] : p.cache[0]) + page * p.cache_page_stride + h * p.cache_head_stride;
            if (row0 > 0 && e > old) {
                const float factor = exp2_int(old - e);
                const int per = p.d / 16;
                for (int i = tid; i < row0 * per; i += kThreads) {
                    const int r = i / per;
                    uint4* at = reinterpret_cast<uint4*>(block + r * p.cache_token_stride + 16 * (i - r * per));
                    *at = round_again(*at, factor);
                }
            }
            // ---- the run's ----
            const float inv = exp2_int(-e);
            auto put = [&](const uint4& v, int r) {
                float f[8];
                widen8<kF16>(v, f);
                const uint32_t lo = pack_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
                const uint32_t hi = pack_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
                *reinterpret_cast<uint2*>(block + (row0 + r) * p.cache_token_stride + 8 * c) = make_uint2(lo, hi);
            };
#pragma unroll
            for (int i = 0; i < kKept; ++i)
                if (r0 + i * rows_at_once < len) put(kept[i], r0 + i * rows_at_once);
            for (int r = r0 + kKept * rows_at_once; r < len; r += rows_at_once)
                put(*reinterpret_cast<const uint4*>(src + r * p.token_stride), r);
            __syncthreads();   // the largest values are read
        }
    }
}

}  // namespace

cudaError_t launch_append_fp8(const AppendFp8Params& params, bool f16, cudaStream_t stream) {
    AppendFp8Params p = params;
    // Tokens of a CTA: one for a decoding step's few, up to a page of a prompt's many.
    const long long want = static_cast<long long>(p.T) * p.Hkv * 2 / (152 * 8);
    p.tile_tokens = static_cast<int>(want < 1 ? 1 : want > p.page_size ? p.page_size : want);
    const long long tiles = (p.T - 1ll) / p.tile_tokens + 1;
    const unsigned grid = static_cast<unsigned>(tiles * p.Hkv * 2);
    return f16 ? launch_overlapped(append_fp8_kernel<true>, grid, kThreads, 0, stream, p)
               : launch_overlapped(append_fp8_kernel<false>, grid, kThreads, 0, stream, p);
}

}  // namespace gbattn
