// paged_api.cu — C entry points of the paged key/value cache declared in
// include/gbattn.h: argument validation, tensor maps and the choice of kernel
// and split.  Nothing here allocates, frees or synchronises.
#include <algorithm>
#include <cmath>

#include "paged.cuh"
#include "paged_cache.h"

namespace gbattn {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

attn_status from_cuda(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

// A stride in elements of `es` bytes: positive, a multiple of 16 bytes, and below
// the 2^40 bytes that a tensor map can hold.  A dimension of one element has no
// stride.
bool stride_ok(long long stride, long long extent, int es = 2) {
    return extent == 1 || (stride > 0 && stride % (16 / es) == 0 && stride < (1ll << 40) / es);
}

// Whether [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Shape of the cache (of elements of `es` bytes) and of what is read from or
// written to it (of type dtype).
attn_status check_cache(int Hkv, int d, attn_dtype dtype, int num_pages, int page_size,
                        long long page_stride, long long head_stride, long long token_stride,
                        int es = 2) {
    if (Hkv < 1 || num_pages < 1 || page_size < 1) return ATTN_ERR_INVALID_ARG;
    if (dtype != ATTN_DTYPE_BF16 && dtype != ATTN_DTYPE_FP16)
        return dtype == ATTN_DTYPE_FP32 || dtype == ATTN_DTYPE_FP8_E4M3 ? ATTN_ERR_UNSUPPORTED
                                                                       : ATTN_ERR_INVALID_ARG;
    if (d != 64 && d != 128 && d != 256) return ATTN_ERR_UNSUPPORTED;
    if (page_size % 8 != 0) return ATTN_ERR_UNSUPPORTED;
    if (static_cast<long long>(num_pages) * page_size >= (1ll << 31)) return ATTN_ERR_UNSUPPORTED;
    if (!stride_ok(page_stride, num_pages, es) || !stride_ok(head_stride, Hkv, es) ||
        !stride_ok(token_stride, page_size, es))
        return ATTN_ERR_MISALIGNED;
    return ATTN_OK;
}

// Which kernel runs, and over how many CTAs.
struct Plan {
    bool decode;           // attn_decode_kernel: few query rows per request
    int tile_tokens;       // tokens of a query tile
    int tiles, tile_div, uniform, splits, cluster;
    size_t slots, descs;   // pieces and joined tiles that the workspace holds
    int rows;              // rows of a slot
};

// Clusters of 1 to 8 CTAs of one SM each that a GB300 runs at once (groups of
// SMs are not all of one size).
constexpr int kClusters[9] = {0, kSMs, 76, 46, 36, 28, 23, 15, 15};

// few > 0: requests of up to that many tokens are another launch's.
Plan plan_one(int B, int H, int Hkv, int total_q, int max_q, long long max_keys, int d, int few) {
    Plan t{};
    const int G = H / Hkv;
    const long long blocks = (max_keys + kTileRows - 1) / kTileRows;
    if (static_cast<long long>(max_q) * G <= 64) {
        t.decode = true;
        t.tile_tokens = max_q;
        t.rows = max_q * G <= 16 ? 16 : (max_q * G <= 32 ? 32 : 64);
        const long long all = static_cast<long long>(B) * Hkv;
        // Few short tiles: the largest clusters that run at once.  A cluster
        // takes as long as its own tile, runs of all tiles as long as the mean
        // one; with lengths spread evenly up to what the page table holds that is
        // half the longest, and the second launch and the pieces' way through
        // memory take about 4 blocks more.
        for (int cs = 8; cs >= 1 && t.cluster == 0; cs /= 2)
            if (all <= kClusters[cs] && (cs == 1 || cs / 2 < blocks) &&
                (blocks + cs - 1) / cs <= 4 + blocks * all / (2 * kSMs))
                t.cluster = cs;
        if (t.cluster > 0) {
            t.tiles = static_cast<int>(all) * t.cluster;
            t.splits = 1;
            return t;
        }
        t.tiles = static_cast<int>(std::min(static_cast<long long>(kSMs), blocks * all));
        t.splits = t.tiles > 1 && blocks > 1 ? 2 : 1;   // a tile can be cut
        t.descs = t.tiles;
        t.slots = 2 * t.descs;
        return t;
    }
    const int per_cta = d == 256 ? 1 : 2;
    t.tile_tokens = kTileRows / G;
    const int cta_tokens = t.tile_tokens * per_cta;
    const long long per_request = (max_q + cta_tokens - 1) / cta_tokens;
    t.tile_div = few > 0 ? std::min(few + 1, std::max(1, cta_tokens / 2)) : cta_tokens;
    const long long packed = total_q / t.tile_div + (few > 0 ? 1ll : static_cast<long long>(B));
    const bool uniform = few == 0 && per_request * B <= packed;
    t.tiles = static_cast<int>(std::min(uniform ? per_request * B : packed, 0x7fffffffll));
    t.uniform = uniform ? static_cast<int>(per_request) : 0;
    // With fewer CTAs than SMs the keys of a tile are shared out, as far as
    // all CTAs still run at once: over a cluster, or over more CTAs where that
    // saves more blocks than joining in a second launch costs (4, about 8 us).
    // Where most requests have no tile, as far as one long request's do, and always
    // over a cluster (two CTAs a tile fit, and there are 48 blocks and more): the
    // pieces' place in the workspace is the other launch's.
    static_assert(kClusters[2] >= kSMs / 2, "tiles that could be split fit clusters of two");
    const long long ctas = (few > 0 ? total_q / cta_tokens + 1ll : t.tiles) * Hkv;
    t.splits = static_cast<int>(std::max(1ll, std::min(kSMs / ctas, blocks)));
    int cs = 8;
    while (cs > 1 && (ctas > kClusters[cs] || cs > blocks)) --cs;
    if (t.splits > 1 && cs > 1 &&
        (few > 0 || (blocks + cs - 1) / cs <= (blocks + t.splits - 1) / t.splits + 4)) {
        t.splits = t.cluster = cs;
        t.rows = per_cta * kTileRows;
        return t;
    }
    t.rows = per_cta * kTileRows;
    if (t.splits > 1) {
        t.descs = static_cast<size_t>(ctas);
        t.slots = t.descs * t.splits;
    }
    return t;
}

// The launches of a call.  Where most requests are short beside the longest (a
// step of decoding with a prompt's chunk in it: the mean at most a quarter of the
// longest), requests of up to `few` tokens go to the decode kernel and the others
// to the tile kernel, if the page table holds at least 48 key blocks a request: a
// single token's tile is one CTA's in the tile kernel, however long its context.
// 32/8 heads, d = 128: 15 tokens over up to 30000 keys beside a chunk of 512, 563
// -> 255 us; 63 over up to 8000, 341 -> 303 us; but 63 over up to 2000, 135 -> 144
// us, hence the 48 blocks (the tile kernel's grid has to have room for more tiles
// than there are, and the empty ones cost it up to 25 us).
struct Plans {
    int count, few;
    Plan plan[2];
};

Plans plan_paged(int B, int H, int Hkv, int total_q, int max_q, long long max_keys, int d) {
    Plans t{};
    const int G = H / Hkv;
    const int few = G <= 64 ? std::max(1, 16 / G) : 0;   // at most 16 rows where one token has no more
    // (2^27: tokens of a tile are at most 15.1 times tile_div, and a tile's number
    // times its tokens, of rows behind the last request too, has to fit 32 bits)
    if (max_q * static_cast<long long>(G) > 64 && few >= 1 && max_keys >= 48 * kTileRows && total_q < (1 << 27) &&
        4ll * total_q <= static_cast<long long>(B) * max_q) {
        t.count = 2;
        t.few = few;
        t.plan[0] = plan_one(B, H, Hkv, total_q, max_q, max_keys, d, few);
        t.plan[1] = plan_one(B, H, Hkv, total_q, few, max_keys, d, 0);
    } else {
        t.count = 1;
        t.plan[0] = plan_one(B, H, Hkv, total_q, max_q, max_keys, d, 0);
    }
    return t;
}

// Workspace bytes: at most one of the launches leaves pieces.
size_t plans_bytes(const Plans& t, int d) {
    size_t bytes = 0;
    for (int i = 0; i < t.count; ++i)
        if (t.plan[i].slots > 0)
            bytes = std::max(bytes, pieces_bytes(t.plan[i].slots, t.plan[i].rows, d, t.plan[i].descs));
    return bytes;
}

attn_status check_paged_shape(int B, int H, int Hkv, int total_q, int max_q, int max_pages,
                              int page_size, int d) {
    if (B < 1 || H < 1 || Hkv < 1 || total_q < 1 || max_q < 1 || max_pages < 1 || page_size < 1)
        return ATTN_ERR_INVALID_ARG;
    if (H % Hkv != 0) return ATTN_ERR_INVALID_ARG;
    if (H / Hkv > kTileRows) return ATTN_ERR_UNSUPPORTED;
    if (d != 64 && d != 128 && d != 256) return ATTN_ERR_UNSUPPORTED;
    if (static_cast<long long>(max_pages) * page_size > kMaxPagedKeys) return ATTN_ERR_UNSUPPORTED;
    if (total_q > (1 << 30) || B > (1 << 30)) return ATTN_ERR_UNSUPPORTED;
    // key blocks of all heads of a request, counted in 32 bits on the device
    if ((static_cast<long long>(max_pages) * page_size / kTileRows + 1) * Hkv >= (1ll << 31))
        return ATTN_ERR_UNSUPPORTED;
    const Plans t = plan_paged(B, H, Hkv, total_q, std::min(max_q, total_q),
                               static_cast<long long>(max_pages) * page_size, d);
    // a persistent CTA's next unit, up to two rounds past the last, fits 32 bits
    for (int i = 0; i < t.count; ++i)
        if (static_cast<long long>(t.plan[i].tiles) * Hkv * t.plan[i].splits >= (1ll << 31) - 2 * kSMs)
            return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

// Tensor map over a cache [num_pages][Hkv][page_size][d] with any strides:
// boxes of box_rows tokens and 64 columns (e4m3: 128, or all 64 in 64-byte rows),
// or (fine) of 8 tokens and all of d.
bool make_tmap_cache(CUtensorMap* map, const void* ptr, attn_dtype dtype, int num_pages, int Hkv,
                     int page_size, int d, long long page_stride, long long head_stride,
                     long long token_stride, int box_rows, bool fine) {
    const bool fp8 = dtype == ATTN_DTYPE_FP8_E4M3;
    auto bytes = [&](long long stride, long long extent) {
        return static_cast<cuuint64_t>(extent == 1 ? d : stride) * (fp8 ? 1 : 2);
    };
    const cuuint64_t ts = bytes(token_stride, page_size), hs = bytes(head_stride, Hkv),
                     ps = bytes(page_stride, num_pages);
    const cuuint64_t pages = static_cast<cuuint64_t>(num_pages), heads = static_cast<cuuint64_t>(Hkv),
                     rows = static_cast<cuuint64_t>(page_size);
    if (fine) {
        const cuuint64_t dims[5] = {64, rows, static_cast<cuuint64_t>(d) / 64, heads, pages};
        const cuuint64_t strides[4] = {ts, 128, hs, ps};
        const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(d) / 64, 1, 1};
        return encode_tmap(map, ptr, dtype, 5, dims, strides, box);
    }
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), rows, heads, pages};
    const cuuint64_t strides[3] = {ts, hs, ps};
    const cuuint32_t box[4] = {fp8 && d > 64 ? 128u : 64u, static_cast<cuuint32_t>(box_rows), 1, 1};
    return encode_tmap(map, ptr, dtype, 4, dims, strides, box,
                       fp8 && d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// Tensor map over packed queries [total_q][H][d]: boxes of `tokens` tokens of
// G heads, whose rows land in shared memory as (token, head).
bool make_tmap_queries(CUtensorMap* map, const void* ptr, attn_dtype dtype, int total_q, int H,
                       int d, long long token_stride, long long head_stride, int G, int tokens) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H),
                                static_cast<cuuint64_t>(total_q)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(H == 1 ? d : head_stride) * 2,
                                   static_cast<cuuint64_t>(total_q == 1 ? static_cast<long long>(d) * H
                                                                        : token_stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(tokens)};
    return encode_tmap(map, ptr, dtype, 3, dims, strides, box);
}

// attn_fwd_paged, or (with scales) attn_fwd_paged_fp8.
attn_status fwd_paged(const void* Q, const void* k_cache, const void* v_cache, bool fp8, const float* k_scale,
                      const float* v_scale, void* O, float* LSE, const int32_t* cu_seqlens_q,
                      const int32_t* seq_lens, const int32_t* page_table, int B, int H, int H_kv, int total_q,
                      int max_seqlen_q, int num_pages, int page_size, int max_pages, int d, attn_dtype dtype,
                      long long q_token_stride, long long q_head_stride, long long cache_page_stride,
                      long long cache_head_stride, long long cache_token_stride, float scale, int causal, int window,
                      void* workspace, size_t workspace_bytes, int* dev_status, void* stream) {
    if (!Q || !k_cache || !v_cache || !O || !LSE || !cu_seqlens_q || !seq_lens || !page_table ||
        (fp8 && (!k_scale || !v_scale)))
        return ATTN_ERR_INVALID_ARG;
    attn_status st = check_cache(H_kv, d, dtype, num_pages, page_size, cache_page_stride,
                                 cache_head_stride, cache_token_stride, fp8 ? 1 : 2);
    if (st != ATTN_OK) return st;
    st = check_paged_shape(B, H, H_kv, total_q, max_seqlen_q, max_pages, page_size, d);
    if (st != ATTN_OK) return st;
    if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
    if (!stride_ok(q_token_stride, total_q) || !stride_ok(q_head_stride, H)) return ATTN_ERR_MISALIGNED;
    if (!aligned(Q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(O, 16) ||
        !aligned(LSE, 16) || !aligned(cu_seqlens_q, 4) || !aligned(seq_lens, 4) ||
        !aligned(page_table, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
        return ATTN_ERR_MISALIGNED;
    const int max_q = std::min(max_seqlen_q, total_q);
    const Plans plans = plan_paged(B, H, H_kv, total_q, max_q,
                                   static_cast<long long>(max_pages) * page_size, d);
    const size_t need = plans_bytes(plans, d);
    if (need > 0) {
        if (workspace == nullptr || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return ATTN_ERR_MISALIGNED;
    }
    PagedParams p{};
    p.O = O;
    p.LSE = LSE;
    p.seq_lens = seq_lens;
    p.page_table = page_table;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.dev_status = dev_status;
    p.lq = SeqLayout{cu_seqlens_q, H, max_q, total_q};
    p.B = B;
    p.Hkv = H_kv;
    p.G = H / H_kv;
    p.few = plans.few;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.page_magic = (1ull << 62) / static_cast<unsigned long long>(page_size) + 1;
    p.causal = causal != 0;
    // a window of 2^30 keys is none: no two positions are that far apart
    p.window = window > 0 && window < kMaxPagedKeys ? window : 0;
    p.scale_log2 = scale * 1.4426950408889634f;
    const bool f16 = dtype == ATTN_DTYPE_FP16;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const attn_dtype cache_dtype = fp8 ? ATTN_DTYPE_FP8_E4M3 : dtype;
    CUtensorMap tq[2], tk[2], tv[2];
    PagedParams params[2];
    for (int i = 0; i < plans.count; ++i) {   // all maps before the first launch
        const Plan& t = plans.plan[i];
        if (t.slots > 0) carve_pieces(p, workspace, t.slots, t.rows, t.descs);
        p.box_rows = std::min(kTileRows, page_size & -page_size);
        // More than 16 boxes of 64 columns a tile: 16 of 8 keys and all columns
        // instead (the decode kernel issues K and V from two warps and has the time).
        p.fine = !t.decode && !fp8 && kTileRows / p.box_rows * (d / 64) > 16;
        if (p.fine) p.box_rows = 8;
        if (fp8 && !t.decode) p.box_rows = std::min(64, p.box_rows);   // (half tiles)
        p.tile_tokens = t.tile_tokens;
        p.tiles = t.tiles;
        p.tile_div = t.tile_div;
        p.uniform_tiles = t.uniform;
        p.splits = t.splits;
        p.cluster = t.cluster;
        p.slot_rows = t.rows;
        params[i] = p;
        if (!make_tmap_queries(&tq[i], Q, dtype, total_q, H, d, q_token_stride, q_head_stride, p.G,
                               p.tile_tokens) ||
            !make_tmap_cache(&tk[i], k_cache, cache_dtype, num_pages, H_kv, page_size, d, cache_page_stride,
                             cache_head_stride, cache_token_stride, p.box_rows, p.fine != 0) ||
            !make_tmap_cache(&tv[i], v_cache, cache_dtype, num_pages, H_kv, page_size, d, cache_page_stride,
                             cache_head_stride, cache_token_stride, p.box_rows, p.fine != 0))
            return ATTN_ERR_CUDA;
    }
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < plans.count && e == cudaSuccess; ++i) {
        const Plan& t = plans.plan[i];
        const auto launch = t.decode ? (fp8 ? launch_paged_decode_fp8 : launch_paged_decode)
                                     : (fp8 ? launch_paged_tiles_fp8 : launch_paged_tiles);
        e = launch(tq[i], tk[i], tv[i], params[i], d, f16, s);
        if (e == cudaSuccess && t.splits > 1 && t.cluster == 0) {
            const int rows = t.tile_tokens * p.G * (t.decode ? 1 : t.rows / kTileRows);
            // pieces of a tile in the mean: CTAs by tiles
            const JoinKind kind = !t.decode ? kJoinMany
                                  : static_cast<long long>(B) * H_kv <= 16 ? kJoinFewRows : kJoinFewPieces;
            e = launch_paged_join(params[i], static_cast<int>(t.descs), rows, kind, d, f16, s);
        }
    }
    return from_cuda(e);
}

}  // namespace
}  // namespace gbattn

using namespace gbattn;

extern "C" {

attn_status attn_page_table(const int32_t* cached_lens, const int32_t* new_lens,
                            int32_t* page_table, const int32_t* free_pages,
                            const int32_t* num_free, int32_t* cu_seqlens_q, int32_t* seq_lens,
                            int64_t* slots, int32_t* pages_taken, int B, int max_pages,
                            int page_size, int max_tokens, int free_capacity, int* dev_status,
                            void* stream) {
    if (!cached_lens || !new_lens || !page_table || !free_pages || !num_free || !cu_seqlens_q ||
        !seq_lens || !slots || !pages_taken)
        return ATTN_ERR_INVALID_ARG;
    if (B < 1 || max_pages < 1 || page_size < 1 || max_tokens < 1 || free_capacity < 1)
        return ATTN_ERR_INVALID_ARG;
    if (B > kMaxTableRequests || page_size % 8 != 0 ||
        static_cast<long long>(max_pages) * page_size > kMaxPagedKeys || max_tokens > (1 << 30))
        return ATTN_ERR_UNSUPPORTED;
    if (!aligned(cached_lens, 4) || !aligned(new_lens, 4) || !aligned(page_table, 4) ||
        !aligned(free_pages, 4) || !aligned(num_free, 4) || !aligned(cu_seqlens_q, 4) ||
        !aligned(seq_lens, 4) || !aligned(slots, 8) || !aligned(pages_taken, 4))
        return ATTN_ERR_MISALIGNED;
    // Every CTA reads the inputs while the first ones already write outputs.
    const size_t nb = static_cast<size_t>(B) * 4;
    const struct { const void* ptr; size_t bytes; } ins[] = {
        {cached_lens, nb}, {new_lens, nb}, {free_pages, static_cast<size_t>(free_capacity) * 4},
        {num_free, 4}, {page_table, nb * max_pages}};
    const struct { const void* ptr; size_t bytes; } outs[] = {
        {cu_seqlens_q, nb + 4}, {seq_lens, nb}, {slots, static_cast<size_t>(max_tokens) * 8},
        {pages_taken, 4}};
    for (const auto& o : outs)
        for (const auto& i : ins)
            if (overlap(o.ptr, o.bytes, i.ptr, i.bytes)) return ATTN_ERR_INVALID_ARG;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i].ptr, outs[i].bytes, outs[j].ptr, outs[j].bytes)) return ATTN_ERR_INVALID_ARG;
    for (int i = 0; i < 4; ++i)   // page_table is an output too
        if (overlap(page_table, nb * max_pages, ins[i].ptr, ins[i].bytes)) return ATTN_ERR_INVALID_ARG;
    TableParams p{};
    p.cached_lens = cached_lens;
    p.new_lens = new_lens;
    p.page_table = page_table;
    p.free_pages = free_pages;
    p.num_free = num_free;
    p.cu_seqlens_q = cu_seqlens_q;
    p.seq_lens = seq_lens;
    p.slots = slots;
    p.pages_taken = pages_taken;
    p.dev_status = dev_status;
    p.B = B;
    p.max_pages = max_pages;
    p.page_size = page_size;
    p.max_tokens = max_tokens;
    p.free_capacity = free_capacity;
    return from_cuda(launch_page_table(p, static_cast<cudaStream_t>(stream)));
}

attn_status attn_cache_append(const void* K, const void* V, void* k_cache, void* v_cache,
                              const int64_t* slots, int T, int H_kv, int d, attn_dtype dtype,
                              int64_t token_stride, int64_t head_stride, int num_pages,
                              int page_size, int64_t cache_page_stride, int64_t cache_head_stride,
                              int64_t cache_token_stride, int* dev_status, void* stream) {
    if (!K || !V || !k_cache || !v_cache || !slots || T < 1) return ATTN_ERR_INVALID_ARG;
    const attn_status st = check_cache(H_kv, d, dtype, num_pages, page_size, cache_page_stride,
                                       cache_head_stride, cache_token_stride);
    if (st != ATTN_OK) return st;
    if (static_cast<long long>(T) * H_kv >= (1ll << 31)) return ATTN_ERR_UNSUPPORTED;
    if (!stride_ok(token_stride, T) || !stride_ok(head_stride, H_kv)) return ATTN_ERR_MISALIGNED;
    if (!aligned(K, 16) || !aligned(V, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(slots, 8))
        return ATTN_ERR_MISALIGNED;
    AppendParams p{};
    p.K = static_cast<const uint16_t*>(K);
    p.V = static_cast<const uint16_t*>(V);
    p.k_cache = static_cast<uint16_t*>(k_cache);
    p.v_cache = static_cast<uint16_t*>(v_cache);
    p.slots = slots;
    p.dev_status = dev_status;
    p.T = T;
    p.Hkv = H_kv;
    p.d = d;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.token_stride = token_stride;
    p.head_stride = head_stride;
    p.cache_page_stride = cache_page_stride;
    p.cache_head_stride = cache_head_stride;
    p.cache_token_stride = cache_token_stride;
    return from_cuda(launch_cache_append(p, static_cast<cudaStream_t>(stream)));
}

attn_status attn_cache_append_fp8(const void* K, const void* V, void* k_cache, void* v_cache,
                                  float* k_scale, float* v_scale, const int64_t* slots, int T,
                                  int H_kv, int d, attn_dtype dtype, int64_t token_stride,
                                  int64_t head_stride, int num_pages, int page_size,
                                  int64_t cache_page_stride, int64_t cache_head_stride,
                                  int64_t cache_token_stride, int* dev_status, void* stream) {
    if (!K || !V || !k_cache || !v_cache || !k_scale || !v_scale || !slots || T < 1) return ATTN_ERR_INVALID_ARG;
    const attn_status st = check_cache(H_kv, d, dtype, num_pages, page_size, cache_page_stride,
                                       cache_head_stride, cache_token_stride, 1);
    if (st != ATTN_OK) return st;
    if (static_cast<long long>(T) * H_kv >= (1ll << 30)) return ATTN_ERR_UNSUPPORTED;
    if (!stride_ok(token_stride, T) || !stride_ok(head_stride, H_kv)) return ATTN_ERR_MISALIGNED;
    if (!aligned(K, 16) || !aligned(V, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(slots, 8))
        return ATTN_ERR_MISALIGNED;
    AppendFp8Params p{};
    p.x[0] = static_cast<const uint16_t*>(K);
    p.x[1] = static_cast<const uint16_t*>(V);
    p.cache[0] = static_cast<uint8_t*>(k_cache);
    p.cache[1] = static_cast<uint8_t*>(v_cache);
    p.scale[0] = k_scale;
    p.scale[1] = v_scale;
    p.slots = slots;
    p.dev_status = dev_status;
    p.T = T;
    p.Hkv = H_kv;
    p.d = d;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.token_stride = token_stride;
    p.head_stride = head_stride;
    p.cache_page_stride = cache_page_stride;
    p.cache_head_stride = cache_head_stride;
    p.cache_token_stride = cache_token_stride;
    return from_cuda(launch_append_fp8(p, dtype == ATTN_DTYPE_FP16, static_cast<cudaStream_t>(stream)));
}

size_t attn_fwd_paged_workspace_size(int B, int H, int H_kv, int total_q, int max_seqlen_q,
                                     int max_pages, int page_size, int d) {
    if (check_paged_shape(B, H, H_kv, total_q, max_seqlen_q, max_pages, page_size, d) != ATTN_OK)
        return 0;
    return plans_bytes(plan_paged(B, H, H_kv, total_q, std::min(max_seqlen_q, total_q),
                                  static_cast<long long>(max_pages) * page_size, d),
                       d);
}

attn_status attn_fwd_paged(const void* Q, const void* k_cache, const void* v_cache, void* O,
                           float* LSE, const int32_t* cu_seqlens_q, const int32_t* seq_lens,
                           const int32_t* page_table, int B, int H, int H_kv, int total_q,
                           int max_seqlen_q, int num_pages, int page_size, int max_pages, int d,
                           attn_dtype dtype, int64_t q_token_stride, int64_t q_head_stride,
                           int64_t cache_page_stride, int64_t cache_head_stride,
                           int64_t cache_token_stride, float scale, int causal, int window,
                           void* workspace, size_t workspace_bytes, int* dev_status,
                           void* stream) {
    return fwd_paged(Q, k_cache, v_cache, false, nullptr, nullptr, O, LSE, cu_seqlens_q, seq_lens, page_table, B, H,
                     H_kv, total_q, max_seqlen_q, num_pages, page_size, max_pages, d, dtype, q_token_stride,
                     q_head_stride, cache_page_stride, cache_head_stride, cache_token_stride, scale, causal, window,
                     workspace, workspace_bytes, dev_status, stream);
}

attn_status attn_fwd_paged_fp8(const void* Q, const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale, void* O, float* LSE,
                               const int32_t* cu_seqlens_q, const int32_t* seq_lens,
                               const int32_t* page_table, int B, int H, int H_kv, int total_q,
                               int max_seqlen_q, int num_pages, int page_size, int max_pages,
                               int d, attn_dtype dtype, int64_t q_token_stride,
                               int64_t q_head_stride, int64_t cache_page_stride,
                               int64_t cache_head_stride, int64_t cache_token_stride, float scale,
                               int causal, int window, void* workspace, size_t workspace_bytes,
                               int* dev_status, void* stream) {
    return fwd_paged(Q, k_cache, v_cache, true, k_scale, v_scale, O, LSE, cu_seqlens_q, seq_lens, page_table, B, H,
                     H_kv, total_q, max_seqlen_q, num_pages, page_size, max_pages, d, dtype, q_token_stride,
                     q_head_stride, cache_page_stride, cache_head_stride, cache_token_stride, scale, causal, window,
                     workspace, workspace_bytes, dev_status, stream);
}

}  // extern "C"
