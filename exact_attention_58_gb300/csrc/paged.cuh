// paged.cuh — attention over a paged key/value cache: parameters shared by the
// host and the kernels, the placement of query rows in tiles, and the layout
// of partial results.
#pragma once

#include "internal.h"
#include "seq.cuh"

namespace gbattn {

// SMs of a GB300; what work is split over.
constexpr int kSMs = 152;

// Largest number of key positions a request can have (max_pages * page_size).
// Positions, windows and tile ends then add up well inside 32 bits.
constexpr long long kMaxPagedKeys = 1ll << 30;

// Weights exp2(s - m) are rounded to the storage type for the product with V, m a
// row's reference.  fp16 holds 2^-24 to just under 2^16, so m is put this far below
// the row's maximum: with the 2^8 that a score may exceed a reference by, weights
// reach 2^15, and the smallest that still count go from 2^-25 of the largest to
// 2^-32.  (Without it 131072 keys 17 nats below the largest lost 0.4% of O: zero in
// the product, but not in the sum, which takes weights unrounded.)  The factor
// cancels in O / l; LSE = m + log2 l.  bf16 has the exponents of fp32 and needs none.
template <bool kF16>
constexpr float kWeightShift = kF16 ? 7.f : 0.f;   // log2 units

// A result that several CTAs computed pieces of, each over its own keys: where
// the pieces are and which output rows they make.  Piece 0 is in slot `slot0`,
// piece i >= 1 in slot `slot1 + (i - 1) * step`.  n = 0: nothing to join.
struct PieceDesc {
    int q_start;   // packed row of the request's first token
    int tok0;      // first token of the tile, counted within the request
    int ntok;      // tokens of the tile
    int hk;        // key/value head
    int n;         // pieces
    int slot0, slot1, step;
};

struct PagedParams {
    void* O;                    // [total_q][H][d]
    float* LSE;                 // [H][total_q]
    const int32_t* seq_lens;    // [B] keys of each request, its new tokens included
    const int32_t* page_table;  // [B][max_pages]
    int* dev_status;
    SeqLayout lq;               // packed queries: cu, H, N = max_seqlen_q, total
    int B, Hkv, G;              // G = H / Hkv query heads read one key/value head
    int num_pages, page_size, max_pages;
    unsigned long long page_magic;   // floor(2^62 / page_size) + 1
    int box_rows;               // keys of one TMA box: the power of two dividing page_size, <= 128
    int fine;                   // tile kernel: boxes of 8 keys and all of d (box_rows = 8)
    int few;                    // > 0: requests of up to this many tokens are the decode kernel's, the
                                // others the tile kernel's; 0: all are the launched kernel's
    int tile_tokens;            // tokens of one 128-row query tile (rows are (token, head of the group))
    int causal, window;
    float scale_log2;           // scale * log2(e)
    // pieces: out[slot][row][d], lse2[slot][row] (log2 units), one descriptor per joined tile
    float* part_o;
    float* part_lse;
    PieceDesc* desc;
    int slot_rows;              // rows of a slot
    int tiles;                  // query tiles of the grid (per key/value head)
    int tile_div;               // tokens per tile index (packed_tile_base)
    int uniform_tiles;          // > 0: every request has this many tiles; 0: tiles follow the packed offsets
    int splits;                 // CTAs that share one tile's keys
    int cluster;                // > 0: CTAs of a cluster, which takes one tile and joins its pieces itself
};

// Keys of request b, clamped to what its page-table row can hold.
__device__ __forceinline__ int paged_keys(const PagedParams& p, int b) {
    const long long cap = static_cast<long long>(p.max_pages) * p.page_size;
    const long long raw = p.seq_lens[b];
    return static_cast<int>(raw < 0 ? 0 : (raw > cap ? cap : raw));
}

// Key range [lo, hi) that queries [first, last] of a request with L keys (at
// key positions query + off) attend between them; lo = hi = 0 when none.
__device__ __forceinline__ void key_range(const PagedParams& p, int first, int last, int off, int L,
                                          int& lo, int& hi) {
    lo = 0;
    hi = p.causal ? min(L, last + off + 1) : L;
    if (p.window > 0) {
        lo = max(0, first + off - p.window + 1);
        if (!p.causal) hi = min(hi, max(0, last + off + p.window));
    }
    if (hi <= lo) lo = hi = 0;
}

// Reports (through dev_status) request lengths and offsets that had to be
// clamped.  Called by every thread of one CTA.
__device__ __forceinline__ void paged_report(const PagedParams& p) {
    if (p.dev_status == nullptr) return;
    bool bad = false;
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
        const int s0 = p.lq.cu[b], s1 = p.lq.cu[b + 1], len = p.seq_lens[b];
        bad |= s0 < 0 || s1 < s0 || s1 > p.lq.total || s1 - s0 > p.lq.N || len != paged_keys(p, b);
    }
    if (bad) atomicCAS(p.dev_status, 0, static_cast<int>(ATTN_ERR_INVALID_ARG));
}

// TMA boxes of the 128-key tile that starts at key k0 of a request, one lane
// per box.  Boxes without a key in [klo, khi) are left out: their pages may
// hold anything, and their table entries need not name a page.
struct PageBox {
    bool needed;
    int page;   // coordinates of the box in the cache
    int row;
};

// Reads the box's table entry; page_box_checked() is for when it is used, a
// tile later, so that nothing waits for the load.
__device__ __forceinline__ PageBox page_box(const PagedParams& p, const int32_t* table, int k0,
                                            int klo, int khi, int lane) {
    PageBox x{false, 0, 0};
    const int key = k0 + lane * p.box_rows;
    if (lane * p.box_rows < kTileRows && key < khi && key + p.box_rows > klo) {
        x.needed = true;
        // key / page_size: exact, key * page_size < 2^62
        const int col = static_cast<int>(__umul64hi(static_cast<unsigned long long>(key) << 2, p.page_magic));
        x.row = key - col * p.page_size;
        x.page = table[col];
    }
    return x;
}
__device__ __forceinline__ int page_box_checked(const PagedParams& p, const PageBox& x) {
    if (static_cast<unsigned>(x.page) < static_cast<unsigned>(p.num_pages)) return x.page;
    if (p.dev_status != nullptr) atomicCAS(p.dev_status, 0, static_cast<int>(ATTN_ERR_INVALID_ARG));
    return p.num_pages;   // outside the cache: the load fills zeros
}

// Host side of the partial results: bytes of `slots` slots of `rows` rows and
// `descs` descriptors, and their places in a workspace.
inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline size_t pieces_bytes(size_t slots, int rows, int d, size_t descs) {
    return align_up(descs * sizeof(PieceDesc), 256) + align_up(slots * rows * sizeof(float), 256) +
           slots * rows * static_cast<size_t>(d) * sizeof(float);
}
inline void carve_pieces(PagedParams& p, void* ws, size_t slots, int rows, size_t descs) {
    char* base = static_cast<char*>(ws);
    p.desc = reinterpret_cast<PieceDesc*>(base);
    base += align_up(descs * sizeof(PieceDesc), 256);
    p.part_lse = reinterpret_cast<float*>(base);
    base += align_up(slots * rows * sizeof(float), 256);
    p.part_o = reinterpret_cast<float*>(base);
    p.slot_rows = rows;
}

// Launches (validated arguments only).
cudaError_t launch_paged_tiles(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const PagedParams& p, int d, bool f16, cudaStream_t stream);
cudaError_t launch_paged_tiles_d128(const CUtensorMap& tq, const CUtensorMap& tk,
                                    const CUtensorMap& tv, const PagedParams& p, bool f16,
                                    cudaStream_t stream);
cudaError_t launch_paged_tiles_d256(const CUtensorMap& tq, const CUtensorMap& tk,
                                    const CUtensorMap& tv, const PagedParams& p, bool f16,
                                    cudaStream_t stream);
// Few query rows per request (max_seqlen_q * G <= 64): p.tiles persistent CTAs,
// p.slot_rows = 16, 32 or 64 rows.
cudaError_t launch_paged_decode(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                const PagedParams& p, int d, bool f16, cudaStream_t stream);
cudaError_t launch_paged_decode_d256(const CUtensorMap& tq, const CUtensorMap& tk,
                                     const CUtensorMap& tv, const PagedParams& p, bool f16,
                                     cudaStream_t stream);
// Joins the pieces of p.desc[0, descs), up to `rows` rows each.
enum JoinKind {
    kJoinFewPieces,   // a few pieces a row
    kJoinFewRows,     // few rows in many pieces each
    kJoinMany,        // many rows and pieces
};
cudaError_t launch_paged_join(const PagedParams& p, int descs, int rows, JoinKind kind, int d, bool f16,
                              cudaStream_t stream);

}  // namespace gbattn
