// paged_cache.cu — the paged key/value cache: writing new rows into it, and
// the page table and slot map of one serving step.
#include "paged_cache.h"

#include "ptx.cuh"

namespace gbattn {
namespace {

// ---------------------------------------------------------------------------
// cache append
// ---------------------------------------------------------------------------
// A copy of T x Hkv rows of K and of V into the slots of a cache: no
// arithmetic, 16 bytes a thread and tensor, bound by memory bandwidth (and by
// the launch for the few rows of a decoding step).  A group of d / 8 threads
// copies one (token, head) row of both tensors, so every access is a whole
// row of 128 to 512 contiguous bytes wherever its page lies.  15800 tokens of 8
// heads, d = 128: 20.3 us, 6.4 TB/s read and written; 64 tokens: 1.7 us.
constexpr int kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendParams p) {
    grid_dep_wait();
    grid_dep_launch_dependents();   // the next kernel sets itself up meanwhile
    const unsigned vecs = static_cast<unsigned>(p.d) / 8;   // 16-byte pieces of a row
    const long long i = static_cast<long long>(blockIdx.x) * kAppendThreads + threadIdx.x;
    const long long row = i / vecs;
    const unsigned c = static_cast<unsigned>(i - row * vecs);
    if (row >= static_cast<long long>(p.T) * p.Hkv) return;
    const int t = static_cast<int>(row / p.Hkv);
    const int h = static_cast<int>(row - static_cast<long long>(t) * p.Hkv);
    const long long slot = p.slots[t];
    if (slot < 0 || slot >= static_cast<long long>(p.num_pages) * p.page_size) {
        // -1 marks a token without a slot; anything else out of range is an error
        if (slot != -1 && p.dev_status != nullptr)
            atomicCAS(p.dev_status, 0, static_cast<int>(ATTN_ERR_INVALID_ARG));
        return;
    }
    const unsigned page = static_cast<unsigned>(slot) / static_cast<unsigned>(p.page_size);
    const unsigned r = static_cast<unsigned>(slot) - page * static_cast<unsigned>(p.page_size);
    const long long src = t * p.token_stride + h * p.head_stride + 8 * c;
    const long long dst = page * p.cache_page_stride + h * p.cache_head_stride +
                          r * p.cache_token_stride + 8 * c;
    const uint4 k = *reinterpret_cast<const uint4*>(p.K + src);
    const uint4 v = *reinterpret_cast<const uint4*>(p.V + src);
    *reinterpret_cast<uint4*>(p.k_cache + dst) = k;
    *reinterpret_cast<uint4*>(p.v_cache + dst) = v;
}

// ---------------------------------------------------------------------------
// page table and slot map
// ---------------------------------------------------------------------------
// Two exclusive sums over the requests (new tokens, then pages to take) and
// one lookup per token.  The data is small (8 bytes a request and token), so
// what counts is the chain of steps: every CTA does both sums itself, in
// shared memory, and then places its own tokens, which needs one launch and no
// word from another CTA.  48 requests of one token 3.7 us, 512 requests and 65500
// tokens 4.4 us: a launch, two dependent loads, two sums and a search.
constexpr int kTableThreads = 512;

// Inclusive sum over the block of one value per thread; `total` is the sum of
// all.  warp_sums: kTableThreads / 32 values in shared memory.
__device__ __forceinline__ long long block_scan(long long x, long long* warp_sums, long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kWarps = kTableThreads / 32;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();   // warp_sums of the scan before is read
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const long long s = warp_sums[w];
        if (w < warp) before += s;
        total += s;
    }
    return before + x;
}

__global__ void __launch_bounds__(kTableThreads) page_table_kernel(const TableParams p) {
    grid_dep_wait();
    grid_dep_launch_dependents();   // the next kernel sets itself up meanwhile
    extern __shared__ int table_smem[];
    int* s_cu = table_smem;               // [B + 1] first token of each request
    int* s_take = table_smem + p.B + 1;   // [B] pages taken by the requests before
    __shared__ long long warp_sums[kTableThreads / 32];
    const long long cap = static_cast<long long>(p.max_pages) * p.page_size;
    const bool first_cta = blockIdx.x == 0;
    const int avail = max(0, min(*p.num_free, p.free_capacity));
    bool bad = first_cta && threadIdx.x == 0 && avail != *p.num_free;

    long long tokens = 0, pages = 0;   // sums over the requests of earlier rounds
    for (int b0 = 0; b0 < p.B; b0 += kTableThreads) {
        const int b = b0 + threadIdx.x;
        long long c = 0, n = 0;
        if (b < p.B) {
            const int c_raw = p.cached_lens[b], n_raw = p.new_lens[b];
            c = max(0ll, min(static_cast<long long>(c_raw), cap));
            n = max(0ll, min(static_cast<long long>(n_raw), cap - c));
            bad |= first_cta && (c != c_raw || n != n_raw);
        }
        long long total;
        const long long end = tokens + block_scan(n, warp_sums, total);
        // tokens past the slot map are dropped
        const long long lo = min(end - n, static_cast<long long>(p.max_tokens));
        const long long hi = min(end, static_cast<long long>(p.max_tokens));
        bad |= first_cta && hi != end;
        tokens += total;
        const long long held = (c + p.page_size - 1) / p.page_size;
        const long long need = (c + hi - lo + p.page_size - 1) / p.page_size - held;
        const long long take = pages + block_scan(need, warp_sums, total) - need;
        pages += total;
        if (b < p.B) {
            s_cu[b] = static_cast<int>(lo);
            s_take[b] = static_cast<int>(min(take, 0x7fffffffll));
            if (b == p.B - 1) s_cu[p.B] = static_cast<int>(hi);
            if (first_cta) {
                p.cu_seqlens_q[b] = static_cast<int>(lo);
                if (b == p.B - 1) p.cu_seqlens_q[p.B] = static_cast<int>(hi);
                p.seq_lens[b] = static_cast<int>(c + hi - lo);
            }
        }
    }
    if (first_cta && threadIdx.x == 0) {
        *p.pages_taken = static_cast<int>(min(pages, static_cast<long long>(avail)));
        bad |= pages > avail;
    }
    __syncthreads();

    for (int t = blockIdx.x * kTableThreads + threadIdx.x; t < p.max_tokens;
         t += gridDim.x * kTableThreads) {
        long long slot = -1;
        if (t < s_cu[p.B]) {
            int lo = 0, n = p.B;   // first request whose tokens end after t
            while (n > 0) {
                const int half = n >> 1;
                if (s_cu[lo + half + 1] <= t) {
                    lo += half + 1;
                    n -= half + 1;
                } else {
                    n = half;
                }
            }
            const int c = static_cast<int>(max(0ll, min(static_cast<long long>(p.cached_lens[lo]), cap)));
            const int pos = c + t - s_cu[lo];
            const int col = pos / p.page_size, row = pos - col * p.page_size;
            const int held = (c + p.page_size - 1) / p.page_size;
            int* entry = p.page_table + static_cast<size_t>(lo) * p.max_pages + col;
            int page;
            if (col < held) {
                page = *entry;   // the page that the cached tokens end in
            } else {
                const long long at = static_cast<long long>(avail) - 1 - s_take[lo] - (col - held);
                page = at >= 0 ? p.free_pages[at] : -1;
                if (row == 0) *entry = page;   // each new page's first token enters it
            }
            if (page >= 0) slot = static_cast<long long>(page) * p.page_size + row;
            else bad = true;
        }
        p.slots[t] = slot;
    }
    if (bad && p.dev_status != nullptr)
        atomicCAS(p.dev_status, 0, static_cast<int>(ATTN_ERR_INVALID_ARG));
}

}  // namespace

cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t stream) {
    const long long n = static_cast<long long>(p.T) * p.Hkv * (p.d / 8);
    const long long grid = (n + kAppendThreads - 1) / kAppendThreads;
    return launch_overlapped(cache_append_kernel, static_cast<unsigned>(grid), kAppendThreads, 0,
                             stream, p);
}

cudaError_t launch_page_table(const TableParams& p, cudaStream_t stream) {
    static std::atomic<unsigned long long> smem_ready{0};
    const cudaError_t e = enable_smem_per_device(
        page_table_kernel, static_cast<int>((2 * kMaxTableRequests + 1) * sizeof(int)), smem_ready);
    if (e != cudaSuccess) return e;
    const int grid = (p.max_tokens + kTableThreads - 1) / kTableThreads;
    return launch_overlapped(page_table_kernel, static_cast<unsigned>(grid < 4 * 152 ? grid : 4 * 152),
                             kTableThreads, (2 * static_cast<size_t>(p.B) + 1) * sizeof(int), stream, p);
}

}  // namespace gbattn
