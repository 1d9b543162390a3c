// attn_paged_kernel.cuh — attention of chunks of new tokens over a paged
// key/value cache.
//
// The online-softmax forward of attn_fwd_kernel.cuh with these differences:
//   * Rows of a query tile are (token, head) pairs: the G query heads that
//     read one key/value head share each K/V tile, so a 128-row tile holds
//     floor(128 / G) tokens of G heads and K/V is read once for all of them.
//   * A 128-key tile is gathered page by page: 128 / box_rows TMA boxes of 64
//     head-dim columns, issued by a lane each, at the (page, row) its page-table
//     entry names.  A TMA instruction costs its warp about 65 cycles, so where
//     pages are small and rows long (kFine) a box is 8 keys of all of d: the
//     tile's 8-row groups then lie one after the other, each with its column
//     blocks of 1 KB, instead of column blocks of 16 KB.
//   * A tile's key blocks can be shared by `splits` CTAs.  Each leaves its
//     normalised output and log-sum-exp as a piece, and they are joined:
//     O = sum_i w_i O_i / sum_i w_i with w_i = exp2(lse2_i - max lse2).  Up to
//     eight CTAs are a cluster and join through distributed shared memory; more
//     leave their pieces in the workspace for a second launch.
//
// Keys outside the range that the CTA's queries attend between them may be
// anything (slots past the last token, pages given back): their scores are
// replaced by -inf before use, and their V rows, whose product with P = 0
// would still be NaN for a NaN or infinite V, are zeroed in shared memory.
//
// Two query tiles per CTA share each K/V block (at head dim 256 one tile, whose
// rows have two softmax threads each).
//
// Bound, like attn_fwd_kernel, by the softmax warps' issue and the chain of
// products per key block (about 2 us for 256 rows x 128 keys at d = 128): whole
// prompts of 4 x 16 x 4096, causal, d = 128, 246 us with other inputs from call to
// call (1118 TFLOP/s; 233 to 240 us over and over on the same ones; the dense kernel
// 225 to 233 either way); a chunk of 512 over 16100 keys, 16 heads, 72 us (950
// TFLOP/s, 128 CTAs of 33 blocks on 152 SMs).
//
// kFp8: a cache of e4m3 with a power-of-two scale per page and head.  TMA loads half
// tiles (D = 256: by 128 columns) as they are, and two warps widen them to fp16 in the
// ring that the products read; scales are factors over the largest of the block's pages,
// which is a factor of its scores and an exponent of its weights (attn_decode_kernel.cuh), or,
// where pages are far apart in size (kSpread), taken page by page in the softmax.
// bf16 queries become fp16 times a power of two a row.  The widening warps bound it
// (a block about 2.7 us): registers leave room for no more than three warps an SM
// sub-partition, and a third on the products' own slows those.  A chunk of 512 over
// 16100 keys 98 us (700 TFLOP/s), whole prompts of 4 x 16 x 4096 345 us.
#pragma once

#include "attn_fwd_kernel.cuh"
#include "fp8.cuh"
#include "paged.cuh"

namespace gbattn {
namespace {

// First index of request b's tiles when tiles follow the packed offsets:
// floor(cu[b] / tile_div) + b, which leaves every request room for its ceil(len /
// T) tiles of T = tile_div tokens; or, where requests of up to `few` tokens have
// none, floor(cu[b] / tile_div) with tile_div = min(few + 1, T / 2), which does so
// for the longer ones (floor(n / tile_div) >= ceil(n / T) for all n > few).
__device__ __forceinline__ int packed_tile_base(const PagedParams& p, int b) {
    return min(max(p.lq.cu[b], 0), p.lq.total) / p.tile_div + (p.few > 0 ? 0 : b);
}

// Request and tile of packed tile index x (whole warp): the last request whose
// base is <= x, found with 32 probes at a time.
__device__ __forceinline__ void find_packed_tile(const PagedParams& p, int x, int& b, int& local) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = p.B;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lo + lane * step;
        const bool below = lane * step < n && packed_tile_base(p, at) <= x;
        const unsigned hit = __ballot_sync(0xffffffffu, below);
        const int k = hit == 0 ? 0 : 31 - __clz(hit);
        lo += k * step;
        n = min(step, n - k * step);
    }
    b = lo;
    local = x - packed_tile_base(p, b);
}

// (kFp8) What the producer passes to the warps that widen e4m3, and to the softmax.
struct Widening {
    uint2 factor[2][16];        // [block][8 keys]: scales over the block's largest, K's and V's, as fp16 twice
    float2 block[8];            // largest scale of K times the softmax scale, exponent of V's (or kUneven)
    int16_t exponents[8][16];   // [block][8 keys] (uneven blocks) of the scales: 256 times K's, plus V's
    int plain[2];               // [block] bit 0, 1: all of K's, V's factors are one
};

// (kFp8) Scales of a block's pages are factors over the largest where they are at most
// 2^kSpread apart: exact in fp16, and the weights, taken times the largest scale of V, count
// down to 2^-29 of a row's largest (2^-32 where all scales are one).  A block whose scales
// are further apart is uneven: widened without factors, and the softmax takes the pages' own
// exponents, so that what a row attends comes out as well whatever pages lie beside it.
constexpr int kSpread = 3;
constexpr float kUneven = 1000.f;
__device__ __forceinline__ int exponent_k(int both) { return (both + 128) >> 8; }
__device__ __forceinline__ int exponent_v(int both) { return both - 256 * exponent_k(both); }

// Uneven blocks' part of the softmax, in short loops in functions of their own: unrolled
// beside the ordinary block's code they slowed that, for its registers and the
// instruction buffer (prompts of 4 x 4096 361 -> 399 us without one uneven block).
//
// Scores in tensor memory, a row of 8 x groups keys per lane, become s + ev.
__device__ __noinline__ void uneven_scores(uint32_t t_S, int groups, const volatile int16_t* exponents,
                                           float scale_log2, float turn) {
#pragma unroll 1
    for (int c = 0; c < groups; ++c) {
        const int both = exponents[c];
        const float f = score_factor(exp2_int(exponent_k(both)) * scale_log2 * turn);
        const float ev = static_cast<float>(exponent_v(both));
        uint32_t x[8];
        tmem_ld8(t_S + 8 * c, x);
        tmem_ld_wait();
        reg_fence(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __float_as_uint(fmaf(__uint_as_float(x[i]), f, ev));
        tmem_st8(t_S + 8 * c, x);
    }
    tmem_st_wait();
}

// All of it for a row with one thread, which attends the block's keys [lo, lim): weights to
// t_P, the row's O (o_cols columns) to its new reference.  Returns reference and sum.
__device__ __noinline__ float2 uneven_block(uint32_t t_S, uint32_t t_P, uint32_t t_O, int o_cols,
                                            const volatile int16_t* exponents, float scale_log2, float turn, int lo,
                                            int lim, float m_ref, float l) {
    uneven_scores(t_S, kTileRows / 8, exponents, scale_log2, turn);
    auto kept = [&](int key, uint32_t x) { return key >= lo && key < lim ? __uint_as_float(x) : -INFINITY; };
    float mx = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < kTileRows; c += 8) {
        uint32_t x[8];
        tmem_ld8(t_S + c, x);
        tmem_ld_wait();
        reg_fence(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, kept(c + i, x[i]));
    }
    const float m_new = fmaxf(m_ref, mx - kWeightShift<true>);
    float alpha = 1.f;
    if (m_ref == -INFINITY) {
        m_ref = m_new;   // O and l are still zero
    } else if (m_new > m_ref + kRescaleThreshold) {
        alpha = ex2_approx(m_ref - m_new);
        m_ref = m_new;
    }
    if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
        for (int c = 0; c < o_cols; c += 8) {
            uint32_t o[8];
            tmem_ld8(t_O + c, o);
            tmem_ld_wait();
            reg_fence(o);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st8(t_O + c, o);
        }
    }
    const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
    float sum = 0.f;
#pragma unroll 1
    for (int c = 0; c < kTileRows; c += 16) {   // weights take half the columns, of scores already read
        uint32_t w[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t x[8];
            tmem_ld8(t_S + c + 8 * h, x);
            tmem_ld_wait();
            reg_fence(x);
            float some = 0.f;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const int k = c + 8 * h + i;
                const float x0 = ex2_approx(kept(k, x[i]) + neg_m), x1 = ex2_approx(kept(k + 1, x[i + 1]) + neg_m);
                w[4 * h + i / 2] = pack_f16x2(x0, x1);
                some += x0 + x1;
            }
            sum = fmaf(some, exp2_int(-exponent_v(exponents[c / 8 + h])), sum);
        }
        tmem_st8(t_P + c / 2, w);
    }
    tmem_st_wait();
    return make_float2(m_ref, fmaf(l, alpha, sum));
}

template <int D, bool kF16, int kTiles, bool kFp8>
struct PagedCfg : FwdCfg<D, false, kF16 || kFp8, false, kTiles> {
    using Base = FwdCfg<D, false, kF16 || kFp8, false, kTiles>;
    // Softmax threads of a row, which share its keys.  One query tile alone has
    // nothing to run while its softmax does: two threads a row halve that (8
    // chunks of 33 to 65 tokens, d = 256: 27.4 -> 25.4 us).  Two tiles fill in for
    // one another, and the barrier per block costs more than it gives (4 x 16 x
    // 4096, d = 128: 245 -> 264 us; d = 64 chunks with a window: 46.9 -> 51.3).
    static constexpr int PARTS = kTiles == 1 ? 2 : 1;
    static constexpr int NC = kTileRows / PARTS;      // keys of a thread
    static constexpr int DC = D / PARTS;              // output columns of a thread
    static constexpr int ROW_THREADS = kTileRows * PARTS;
    static constexpr int CONV_WARP = kTiles * ROW_THREADS / 32 + 2;   // (kFp8) two that widen
    static constexpr int THREADS = kTiles * ROW_THREADS + (kFp8 ? 128 : 64);
    static constexpr int PRODUCER_WARP = kTiles * ROW_THREADS / 32;
    static constexpr int MMA_WARP = PRODUCER_WARP + 1;
    static constexpr int ROW_FLOATS = kTiles * ROW_THREADS;   // one per softmax thread
    static constexpr int PART_BYTES = PARTS > 1 ? 3 * ROW_FLOATS * 4 : 0;   // maxima; sums of two units
    // (kFp8) e4m3 as loaded: 64 rows of up to 128 head-dim columns a slot
    static constexpr int RAW_COLS = D < 128 ? D : 128;
    static constexpr int RAW = 64 * RAW_COLS;
    static constexpr int NRAW = D == 64 ? 8 : D == 128 ? 4 : 3;
    static constexpr int UNITS = 2 * D / RAW_COLS;    // slots of a K or V tile
    static constexpr int TURN_BYTES = 2 * 2 * kTileRows;
    static constexpr int SMEM = Base::SMEM + PART_BYTES + (kFp8 ? NRAW * RAW + TURN_BYTES : 0);
};

template <int D, bool kF16, int kTiles, bool kFine, bool kLoop, bool kFp8>
__global__ void __launch_bounds__(PagedCfg<D, kF16, kTiles, kFp8>::THREADS, 1)
    attn_paged_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const PagedParams p) {
    using C = PagedCfg<D, kF16, kTiles, kFp8>;
    constexpr bool kMmaF16 = kF16 || kFp8;   // type of the products' operands
    constexpr bool kTurnQ = kFp8 && !kF16;   // bf16 queries become fp16 times a power of two a row
    grid_dep_wait();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sQ = smem;                                   // C::TILES tiles
    uint8_t* sKV = smem + C::TILES * C::TILE;             // NSLOT tiles
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (C::TILES + C::NSLOT) * C::TILE + (kFp8 ? C::NRAW * C::RAW : 0));
    uint64_t* bar_q = bars;               // [2] one per query tile
    uint64_t* full = bars + 2;
    constexpr int kPairs = C::NSLOT / 2;
    constexpr bool kBlockRelease = kPairs >= 2;   // see attn_fwd_kernel
    uint64_t* empty = full + C::NSLOT;
    uint64_t* bar_s = empty + C::NSLOT;   // [2]
    uint64_t* bar_p = bar_s + 2;          // [2]
    uint64_t* bar_o = bar_p + 2;          // [2]
    uint64_t* bar_fin = bar_o + 2;
    uint64_t* q_free = bar_fin + 1;       // (kLoop) a tile's last S has read the queries
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(q_free + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    uint64_t* q_turned = bars + 32;       // (kFp8) [2] a query tile is fp16
    uint64_t* meta_full = bars + 34;      // [2] a block's factors
    uint64_t* meta_empty = bars + 36;
    uint64_t* raw_full = bars + 38;       // [NRAW]
    uint64_t* raw_empty = bars + 46;
    volatile Widening& wide = *reinterpret_cast<volatile Widening*>(bars + 54);
    static_assert(54 * 8 + sizeof(Widening) <= 1024, "factors fit behind the barriers");
    uint8_t* sRaw = smem + (C::TILES + C::NSLOT) * C::TILE;   // (kFp8: the ring, and the barriers behind it)
    int8_t* s_turn = reinterpret_cast<int8_t*>(bars) + 1024 + C::PART_BYTES;   // [unit & 1][tile][row] exponents
    float* s_max = reinterpret_cast<float*>(bars + 128);   // (PARTS = 2) [tile][part][row]
    float* s_sum = s_max + C::ROW_FLOATS;                  // and [unit & 1][tile][part][row]

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    // ---- which tokens of which request, which key/value head, which keys ----
    const int G = p.G;
    const int TT = p.tile_tokens;
    // Unit x: a tile of a request and a key/value head (kLoop: a CTA takes one unit
    // of every round of as many as there are CTAs, rounds going up and down the CTAs
    // in turn; else one unit to the p.splits CTAs of a group).  The last tiles of a
    // causal request see the most keys: units are in falling order where all
    // requests have as many tiles, so that a CTA's units weigh the same in sum (4
    // x 16 x 4096 queries, d 128: 7 rounds within 2% of the mean; request by request
    // in equal strides the longest CTA had 23% more).
    const int units = p.tiles * p.Hkv;
    const int split = kLoop ? 0 : static_cast<int>(blockIdx.x) % p.splits;
    const int unit = kLoop ? static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x) / p.splits;
    struct TilePlan {
        int b, start, N, L;           // the request: first packed row, queries (0: no such tile), keys
        int tok0, hk;                 // first token of the tile; key/value head
        int jlo0, jhi0, jlo1, jhi1;   // key blocks of the query tiles
        int klo, khi;                 // keys that the tile's queries attend between them
        int pieces;
    };
    auto plan_of = [&](int x) {
        TilePlan t;
        const int order = x / p.Hkv;
        const int tile = p.tiles - 1 - order;
        t.hk = x - order * p.Hkv;
        int local;
        if (p.uniform_tiles > 0) {
            local = tile / p.B;
            t.b = tile - local * p.B;
        } else {
            find_packed_tile(p, tile, t.b, local);
        }
        const SeqSpan sq = seq_span(p.lq, t.b, nullptr, false);
        t.start = sq.start;
        t.N = sq.len;
        t.L = paged_keys(p, t.b);
        t.tok0 = local * C::TILES * TT;
        if (local < 0 || t.tok0 >= t.N || t.N <= p.few) t.N = t.tok0 = 0;
        const int off = t.L - t.N;   // query i stands at key position i + off
        t.jlo0 = t.jhi0 = t.jlo1 = t.jhi1 = t.klo = t.khi = 0;
#pragma unroll
        for (int i = 0; i < C::TILES; ++i) {
            const int first = t.tok0 + i * TT;
            int lo = 0, hi = 0;
            if (first < t.N) key_range(p, first, min(first + TT, t.N) - 1, off, t.L, lo, hi);
            if (hi > lo) {
                t.klo = t.khi > t.klo ? min(t.klo, lo) : lo;
                t.khi = max(t.khi, hi);
            }
            const int bl = lo / kTileRows, bh = (hi + kTileRows - 1) / kTileRows;
            if (i == 0) { t.jlo0 = bl; t.jhi0 = bh; } else { t.jlo1 = bl; t.jhi1 = bh; }
        }
        t.pieces = 1;
        if (!kLoop) {   // this CTA's share of the blocks
            const int all_lo = t.klo / kTileRows, all_hi = (t.khi + kTileRows - 1) / kTileRows;
            const int share = (all_hi - all_lo + p.splits - 1) / p.splits;
            if (share > 0) t.pieces = (all_hi - all_lo + share - 1) / share;
            if (t.pieces > 1) {
                const int s0 = all_lo + split * share, s1 = min(all_hi, s0 + share);
                t.jlo0 = max(t.jlo0, s0); t.jhi0 = min(t.jhi0, s1);
                t.jlo1 = max(t.jlo1, s0); t.jhi1 = min(t.jhi1, s1);
                if (t.jhi0 <= t.jlo0) t.jlo0 = t.jhi0 = 0;
                if (t.jhi1 <= t.jlo1) t.jlo1 = t.jhi1 = 0;
            }
        }
        return t;
    };
    TilePlan pl = plan_of(unit);
    const int pieces = pl.pieces;
    const bool joined = !kLoop && pieces > 1;
    if (!kLoop) {
        const int ntok = pl.N > 0 ? min(C::TILES * TT, pl.N - pl.tok0) : 0;
        if (threadIdx.x == 0 && split == 0 && p.splits > 1 && p.cluster == 0)
            p.desc[unit] = PieceDesc{pl.start, pl.tok0, ntok, pl.hk, joined ? pieces : 0,
                                     unit * p.splits, unit * p.splits + 1, 1};
    }
    if (blockIdx.x == 0) paged_report(p);
    if (!kLoop && pl.N == 0) return;

    // A cluster's pieces, where the K/V ring and the queries were: rows of D
    // floats in 16-byte groups, group c of row r at c ^ r (mod the groups of a
    // row), so that neither the rows' writers (a row per thread) nor the readers (a
    // group per lane) meet in a bank; and the rows' log-sum-exp.
    float* const s_piece = reinterpret_cast<float*>(sKV);
    float* const s_lse = reinterpret_cast<float*>(sQ);
    constexpr int GROUPS = D / 4;
    static_assert(C::TILES * kTileRows * D * 4 <= C::NSLOT * C::TILE, "a piece fits the ring");
    auto piece_group = [&](int row, int c) { return s_piece + row * D + 4 * (c ^ (row & (GROUPS - 1))); };
    // Joins them, a row per warp, rows dealt out over the cluster's warps.
    auto join_cluster = [&]() {
        cluster_sync();
        constexpr int WARPS = C::THREADS / 32;
        const int ntok = min(C::TILES * TT, pl.N - pl.tok0);
        for (int u = split * WARPS + warp; u < ntok * G; u += p.splits * WARPS) {
            const int ut = u / G, g = u - ut * G;
            const int row = ut / TT * kTileRows + (ut % TT) * G + g;
            float w = lane < p.splits ? ld_cluster(&s_lse[row], lane) : -INFINITY;
            float M = w;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            M = __shfl_sync(0xffffffffu, M, 0);
            w = M == -INFINITY ? 0.f : ex2_approx(w - M);
            float sum = w;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            sum = __shfl_sync(0xffffffffu, sum, 0);
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const int head = pl.hk * G + g;
            uint2* dst = reinterpret_cast<uint2*>(
                static_cast<uint16_t*>(p.O) + ((static_cast<size_t>(pl.start) + pl.tok0 + ut) * p.lq.H + head) * D);
            for (int c = lane; c < GROUPS; c += 32) {
                // all pieces' loads before the first is used
                constexpr unsigned LANES = GROUPS < 32 ? (1u << (GROUPS & 31)) - 1u : 0xffffffffu;
                float4 x[8], acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < p.splits) x[i] = ld_cluster4(piece_group(row, c), i);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float wi = __shfl_sync(LANES, w, i);
                    if (i < p.splits && wi != 0.f) {   // else no key, or no piece at all
                        acc.x += wi * x[i].x;
                        acc.y += wi * x[i].y;
                        acc.z += wi * x[i].z;
                        acc.w += wi * x[i].w;
                    }
                }
                dst[c] = make_uint2(pack_h2<kF16>(acc.x * inv, acc.y * inv), pack_h2<kF16>(acc.z * inv, acc.w * inv));
            }
            __syncwarp();
            if (lane == 0)
                p.LSE[static_cast<size_t>(head) * p.lq.total + pl.start + pl.tok0 + ut] =
                    sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
        }
        cluster_sync();   // no CTA leaves while another reads its piece
    };
    if (!kLoop && split >= pieces) {   // no blocks left for this CTA
        if (p.cluster > 0 && joined) {
            for (int r = threadIdx.x; r < C::TILES * kTileRows; r += C::THREADS) s_lse[r] = -INFINITY;
            join_cluster();
        }
        return;
    }

    // blocks the CTA walks for a plan: tile A's window starts no later than tile B's
    auto first_block = [](const TilePlan& t) { return t.jhi0 > t.jlo0 ? t.jlo0 : t.jlo1; };
    auto num_blocks = [&](const TilePlan& t) { return max(0, max(t.jhi0, t.jhi1) - first_block(t)); };
    // the next unit's plan, or false
    int round = 0;
    auto next_unit = [&]() {
        if (!kLoop) return false;
        const int n = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
        ++round;
        const int x = round * n + ((round & 1) ? n - 1 - c : c);
        if (x >= units) return false;   // only in the last round
        pl = plan_of(x);
        return true;
    };

    // ---- set-up ----
    if (threadIdx.x == 0) {
        mbar_init(&bar_q[0], 1);
        mbar_init(&bar_q[1], 1);
        for (int s = 0; s < C::NSLOT; ++s) {
            mbar_init(&full[s], kFp8 ? 64 : 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < C::NRAW && kFp8; ++s) {
            mbar_init(&raw_full[s], 1);
            mbar_init(&raw_empty[s], 64);
        }
        for (int s = 0; s < 2 && kFp8; ++s) {
            mbar_init(&q_turned[s], 64);
            mbar_init(&meta_full[s], 1);
            mbar_init(&meta_empty[s], 64);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bar_s[t], 1);
            mbar_init(&bar_p[t], C::ROW_THREADS);
            mbar_init(&bar_o[t], 1);
        }
        mbar_init(bar_fin, 1);
        mbar_init(q_free, 1);
        *s_abort = 0;
        fence_mbar_init();
    }
    if (warp == C::MMA_WARP) {
        tmem_alloc(s_tmem, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp == C::PRODUCER_WARP) {
        // ================= TMA producer =================
        if (lane == 0) {
            tma_prefetch_desc(&tmQ);
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
        }
        int seq = 0;                        // ring fills (kFp8: blocks) so far
        int raw_fills = 0;
        int tiles = 0, q_n0 = 0, q_n1 = 0;  // units with blocks; loads of each query tile
        bool ok = true;
        do {
            const int jbeg = first_block(pl), nkv = num_blocks(pl);
            if (nkv == 0) continue;
            const int32_t* table = p.page_table + static_cast<size_t>(pl.b) * p.max_pages;
            PageBox box = page_box(p, table, jbeg * kTileRows, pl.klo, pl.khi, lane);
            if (tiles > 0 && !mbar_wait_warp(q_free, (tiles - 1) & 1, s_abort)) {
                ok = false;
                break;
            }
            ++tiles;
            for (int t = 0; t < C::TILES; ++t) {
                const bool used = t ? pl.jhi1 > pl.jlo1 : pl.jhi0 > pl.jlo0;
                if (used && lane == 0) {
                    mbar_arrive_expect_tx(&bar_q[t], static_cast<uint32_t>(TT * G) * C::ROWB);
                    for (int cb = 0; cb < C::NCB; ++cb)
                        tma_load_3d(sQ + t * C::TILE + cb * C::CB_BYTES, &tmQ, &bar_q[t],
                                    cb * C::BOXW, pl.hk * G, pl.start + pl.tok0 + t * TT);
                }
            }
            q_n0 += pl.jhi0 > pl.jlo0;
            q_n1 += pl.jhi1 > pl.jlo1;
            // (kFp8) A block's scales are taken relative to its largest, so that one
            // factor holds for all its scores and one exponent for all its weights, or
            // (uneven) page by page.  They are read a block ahead and passed on before the
            // block's loads, while the ring is still full (behind the first load, prompts of 4 x
            // 4096 took 361 us instead of 351).  The eight blocks' worth of room is more
            // than this warp runs ahead of the softmax (two blocks, and the ring's up to four).
            int page = p.num_pages;
            uint32_t kb = 0, vb = 0;
            auto ask = [&]() {   // the page of this lane's box, and its scales
                page = box.needed ? page_box_checked(p, box) : p.num_pages;
                kb = vb = 127u << 23;
                if (page < p.num_pages) {
                    const size_t at = static_cast<size_t>(page) * p.Hkv + pl.hk;
                    kb = __float_as_uint(p.k_scale[at]);
                    vb = __float_as_uint(p.v_scale[at]);
                }
            };
            if (kFp8) ask();
            for (int j = jbeg; kFp8 && j < jbeg + nkv && ok; ++j, ++seq) {
                const unsigned needed = __ballot_sync(0xffffffffu, box.needed);
                const int row = box.row, mine_at = box.needed ? page : -1;
                if ((bad_scale(kb) || bad_scale(vb)) && p.dev_status != nullptr)
                    atomicCAS(p.dev_status, 0, static_cast<int>(ATTN_ERR_INVALID_ARG));
                const bool there = page < p.num_pages;
                const int ke = there ? scale_exponent(kb) : kLeastScale, ve = there ? scale_exponent(vb) : kLeastScale;
                const int k_top = __reduce_max_sync(0xffffffffu, ke), v_top = __reduce_max_sync(0xffffffffu, ve);
                ok = mbar_wait_warp_soon(&meta_empty[seq & 1], ((seq >> 1) & 1) ^ 1, s_abort);
                if (!ok) break;
                const int plain = (__all_sync(0xffffffffu, !there || ke == k_top) ? 1 : 0) |
                                  (__all_sync(0xffffffffu, !there || ve == v_top) ? 2 : 0);
                const bool uneven = __any_sync(0xffffffffu, there && max(k_top - ke, v_top - ve) > kSpread);
                const float kf = exp2_int(uneven ? 0 : max(ke - k_top, -60)), vf = exp2_int(uneven ? 0 : max(ve - v_top, -60));
                for (int i = 0; i < p.box_rows / 8 && lane < kTileRows / p.box_rows; ++i) {
                    const int at = lane * (p.box_rows / 8) + i;
                    volatile uint2& f = wide.factor[seq & 1][at];
                    f.x = pack_f16x2(kf, kf);
                    f.y = pack_f16x2(vf, vf);
                    wide.exponents[seq & 7][at] = static_cast<int16_t>(256 * ke + ve);
                }
                if (lane == 0) {
                    wide.plain[seq & 1] = uneven ? 3 : plain;
                    wide.block[seq & 7].x = exp2_int(k_top) * p.scale_log2;
                    wide.block[seq & 7].y = uneven ? kUneven : static_cast<float>(v_top);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&meta_full[seq & 1]);
                if (j + 1 < jbeg + nkv) box = page_box(p, table, (j + 1) * kTileRows, pl.klo, pl.khi, lane);
                const int half_boxes = 64 / p.box_rows;
#pragma unroll 1
                for (int u = 0; u < 2 * C::UNITS; ++u) {
                    const int which = u / C::UNITS, part = u % C::UNITS;   // part: 64 rows, then columns
                    const int n = 2 * C::UNITS * seq + u, slot = n % C::NRAW;
                    ok = mbar_wait_warp_soon(&raw_empty[slot], ((n / C::NRAW) & 1) ^ 1, s_abort);
                    if (!ok) break;
                    const unsigned mine = needed >> ((part & 1) * half_boxes) & ((1u << half_boxes) - 1u);
                    ++raw_fills;
                    if (lane == 0)
                        mbar_arrive_expect_tx(&raw_full[slot],
                                              __popc(mine) * static_cast<uint32_t>(p.box_rows) * C::RAW_COLS);
                    __syncwarp();
                    if (mine_at >= 0 && lane / half_boxes == (part & 1))
                        tma_load_4d(sRaw + slot * C::RAW + lane % half_boxes * p.box_rows * C::RAW_COLS, which ? &tmV : &tmK,
                                    &raw_full[slot], (part >> 1) * C::RAW_COLS, row, pl.hk, mine_at);
                    __syncwarp();
                }
                if (ok) ask();   // (behind the last block once too often)
            }
            for (int j = jbeg; !kFp8 && j < jbeg + nkv && ok; ++j) {
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, box.needed)) *
                                       static_cast<uint32_t>(p.box_rows) * C::ROWB;
                // the next tile's table entries arrive while this tile waits
                PageBox next = box;
                if (j + 1 < jbeg + nkv) next = page_box(p, table, (j + 1) * kTileRows, pl.klo, pl.khi, lane);
                for (int which = 0; which < 2; ++which) {
                    const int slot = seq % C::NSLOT;
                    const uint32_t ph = (seq / C::NSLOT) & 1;
                    bool free_ok;
                    if constexpr (kBlockRelease) {
                        const int bi = seq / 2;
                        const int wb = which == 0 ? bi - kPairs : bi - kPairs + 1;
                        free_ok = bi < kPairs || mbar_wait_warp(&empty[wb % kPairs], (wb / kPairs) & 1, s_abort);
                    } else {
                        free_ok = mbar_wait_warp(&empty[slot], ph ^ 1, s_abort);
                    }
                    if (!free_ok) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&full[slot], bytes);
                    __syncwarp();
                    if (kFine && box.needed) {
                        tma_load_5d(sKV + slot * C::TILE + lane * 8 * C::ROWB, which ? &tmV : &tmK, &full[slot], 0,
                                    box.row, 0, pl.hk, page_box_checked(p, box));
                    } else if (box.needed) {
                        const int page = page_box_checked(p, box);
                        uint8_t* dst = sKV + slot * C::TILE + lane * p.box_rows * 128;
                        const CUtensorMap* m = which ? &tmV : &tmK;
                        for (int cb = 0; cb < C::NCB; ++cb)
                            tma_load_4d(dst + cb * C::CB_BYTES, m, &full[slot], cb * C::BOXW, box.row,
                                        pl.hk, page);
                    }
                    __syncwarp();
                    ++seq;
                }
                box = next;
            }
        } while (ok && next_unit());
        // Drain: every load this warp issued has landed before teardown.
        if (lane == 0) {
            volatile int no_abort = 0;
            if (q_n0 > 0) mbar_wait(&bar_q[0], (q_n0 - 1) & 1, &no_abort);
            if (q_n1 > 0) mbar_wait(&bar_q[1], (q_n1 - 1) & 1, &no_abort);
            constexpr int slots = kFp8 ? C::NRAW : C::NSLOT;
            if (kFp8) seq = raw_fills;
            for (int s = 0; s < slots && s < seq; ++s) {
                const int uses = (seq - s + slots - 1) / slots;
                mbar_wait(kFp8 ? &raw_full[s] : &full[s], (uses - 1) & 1, &no_abort);
            }
        }
        __syncwarp();
    } else if (warp == C::MMA_WARP) {
        // ================= MMA issuer =================
        {
            const uint64_t dq0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
            const uint64_t dq1 = sdesc_adv(dq0, C::TILE);
            // K-major K and MN-major V of slot 0: 8-row groups 1 KB apart and column
            // blocks 16 KB, or (kFine) groups a row group's bytes apart, blocks 1 KB
            const uint64_t dk0 = sdesc_sw128(smem_u32(sKV), 16, kFine ? 8 * C::ROWB : 1024);
            const uint64_t dv0 = sdesc_sw128(smem_u32(sKV), kFine ? 1024 : C::CB_BYTES, kFine ? 8 * C::ROWB : 1024);
            auto issue_qk = [&](int t, int slot) {
                const uint32_t d_tmem = tmem + 128u * t;
                const uint64_t ad = t ? dq1 : dq0;
                const uint64_t bd = sdesc_adv(dk0, slot * C::TILE);
                constexpr uint32_t CB = C::CB_BYTES / 16 - 6, CK = kFine ? 1024 / 16 - 6 : CB;
                if constexpr (C::QK_STEPS == 4) {
                    mma4_ss_f16<2, 2, 2, 2, 2, 2>(d_tmem, ad, bd, C::IDESC_QK, 0u);
                } else {
                    mma8_ss_f16<2, 2, 2, CB, 2, 2, 2, 2, 2, 2, CK, 2, 2, 2>(d_tmem, ad, bd, C::IDESC_QK, 0u);
                    if constexpr (C::QK_STEPS == 16)
                        mma8_ss_f16<2, 2, 2, CB, 2, 2, 2, 2, 2, 2, CK, 2, 2, 2>(
                            d_tmem, sdesc_adv(ad, 2 * C::CB_BYTES),
                            sdesc_adv(bd, 2 * (kFine ? 1024 : C::CB_BYTES)), C::IDESC_QK, 1u);
                }
            };
            auto issue_pv = [&](int t, int slot, bool accumulate) {
                mma_run_ts_f16<8, 8, (kFine ? 2 * 8 * C::ROWB : C::KSTEP * 128) / 16>(tmem + C::O_COL + D * t, tmem + 128u * t,
                                                          sdesc_adv(dv0, slot * C::TILE), C::IDESC_PV,
                                                          accumulate ? 1u : 0u);
            };
            bool ok = true;
            uint32_t g = 0;                   // K/V blocks of the units before
            uint32_t q_n0 = 0, q_n1 = 0;      // units in which a query tile had blocks
            uint32_t p_n0 = 0, p_n1 = 0;      // blocks of a query tile in them
            do {
                const int jlo0 = pl.jlo0, jhi0 = pl.jhi0, jlo1 = pl.jlo1, jhi1 = pl.jhi1;
                auto jlo = [&](int t) { return t ? jlo1 : jlo0; };
                auto jhi = [&](int t) { return t ? jhi1 : jhi0; };
                const int jbeg = first_block(pl), nkv = num_blocks(pl);
                if (nkv == 0) continue;
                if (lane == 0) {
                    // parity of P of block j of query tile t: (p_base(t) + j) & 1
                    const uint32_t p_b0 = p_n0 - jlo0, p_b1 = p_n1 - jlo1;
                    auto p_parity = [&](int t, int j) { return ((t ? p_b1 : p_b0) + j) & 1u; };
                    bool q_ready[2] = {false, false};
                    uint32_t seq = 2 * g;
                    int v_slot = 0;
                    uint32_t v_phase = 0;
                    bool v_ready = false;
                    for (int j = jbeg; j < jbeg + nkv && ok; ++j) {
                        const int kslot = seq % C::NSLOT;
                        const uint32_t kph = (seq / C::NSLOT) & 1;
                        ++seq;
                        const int next_v_slot = seq % C::NSLOT;
                        const uint32_t next_v_phase = (seq / C::NSLOT) & 1;
                        ++seq;
                        bool k_ready = false;
                        constexpr bool kEarlyVRelease = C::NSLOT == 2;   // see attn_fwd_kernel
                        int v_last = -1;
                        for (int t = 0; t < C::TILES; ++t)
                            if (kEarlyVRelease && j - 1 >= jlo(t) && j - 1 < jhi(t)) v_last = t;
                        for (int t = 0; t < C::TILES && ok; ++t) {
                            const bool qk = j >= jlo(t) && j < jhi(t);
                            const bool prev = j - 1 >= jlo(t) && j - 1 < jhi(t);
                            const bool last_pv = prev && j == jhi(t);
                            if (prev) {   // O_t += P_t(j-1) V_{j-1}
                                ok = mbar_wait(&bar_p[t], p_parity(t, j - 1), s_abort);
                                if (!ok) break;
                                tc_fence_after();
                                if (!v_ready) {
                                    ok = mbar_wait(&full[v_slot], v_phase, s_abort);
                                    v_ready = true;
                                    if (!ok) break;
                                    tc_fence_after();
                                }
                                issue_pv(t, v_slot, j - 1 > jlo(t));
                                if (last_pv) tc_commit(&bar_o[t]);
                                if (t == v_last) tc_commit(&empty[v_slot]);
                            }
                            if (qk) {     // S_t = Q_t K_j^T
                                if (!q_ready[t]) {
                                    ok = mbar_wait(kTurnQ ? &q_turned[t] : &bar_q[t], (t ? q_n1 : q_n0) & 1, s_abort);
                                    q_ready[t] = true;
                                    if (!ok) break;
                                    tc_fence_after();
                                }
                                if (!k_ready) {
                                    ok = mbar_wait(&full[kslot], kph, s_abort);
                                    k_ready = true;
                                    if (!ok) break;
                                    tc_fence_after();
                                }
                                issue_qk(t, kslot);
                                tc_commit(&bar_s[t]);
                            }
                        }
                        if (!ok) break;
                        if constexpr (kBlockRelease) {
                            tc_commit(&empty[kslot / 2]);   // pair (seq / 2) % kPairs
                        } else {
                            tc_commit(&empty[kslot]);
                            if (j > jbeg && v_last < 0) tc_commit(&empty[v_slot]);
                        }
                        v_slot = next_v_slot;
                        v_phase = next_v_phase;
                        v_ready = false;
                    }
                    if (kLoop && ok) tc_commit(q_free);
                    for (int t = 0; t < C::TILES && ok; ++t) {   // tiles whose last block is the unit's last
                        if (jhi(t) == jlo(t) || jhi(t) != jbeg + nkv) continue;
                        ok = mbar_wait(&bar_p[t], p_parity(t, jhi(t) - 1), s_abort);
                        if (ok && !v_ready) {
                            ok = mbar_wait(&full[v_slot], v_phase, s_abort);
                            v_ready = true;
                        }
                        if (!ok) break;
                        tc_fence_after();
                        issue_pv(t, v_slot, jhi(t) - 1 > jlo(t));
                        tc_commit(&bar_o[t]);
                        if (!kBlockRelease) tc_commit(&empty[v_slot]);   // (one query tile)
                    }
                }
                g += nkv;
                p_n0 += jhi0 - jlo0;
                p_n1 += jhi1 - jlo1;
                q_n0 += jhi0 > jlo0;
                q_n1 += jhi1 > jlo1;
                ok = __shfl_sync(0xffffffffu, ok, 0);
            } while (ok && next_unit());
            // Drain: no MMA of this CTA is in flight at teardown.
            if (lane == 0) {
                tc_commit(bar_fin);
                volatile int no_abort = 0;
                mbar_wait(bar_fin, 0, &no_abort);
            }
        }
        __syncwarp();
    } else if (kFp8 && warp >= C::CONV_WARP) {
        // ================= K and V from e4m3 to fp16, bf16 queries to fp16 =================
        // A thread takes 16 bytes of a row at a time.  Eight consecutive ones take 64
        // head-dim columns of rows r and r ^ 5: their reads lie in opposite halves of
        // the swizzled 128 bytes (at d = 64: in rows of unlike parity), and their two
        // writes each in the even and the odd 16-byte groups: no two meet in a bank.
        const int tid = static_cast<int>(threadIdx.x) - 32 * C::CONV_WARP;
        constexpr int STEP = D == 64 ? 16 : 8;           // rows from one piece of a thread to its next
        const int cq = tid & 3, x = tid >> 3;
        const int cb = D == 64 ? 0 : x & 1, y = D == 64 ? x : x >> 1;
        const int r0 = ((y >> 2) * 8 + (y & 3)) ^ ((tid & 4) ? 5 : 0);
        const uint8_t* const src0 = sRaw + r0 * C::RAW_COLS +
                                    (((4 * cb + cq) ^ (D == 64 ? (r0 >> 1) & 3 : r0 & 7)) << 4);
        uint8_t* const dst0 = sKV + cb * C::CB_BYTES + r0 * 128;
        const int d0 = ((2 * cq) ^ (r0 & 7)) << 4, d1 = ((2 * cq + 1) ^ (r0 & 7)) << 4;
        int raw = 0;                            // raw slots so far
        int fills = 0, blk = 0;                 // ring fills and blocks so far
        int units8 = 0, q_n0 = 0, q_n1 = 0;     // units with blocks; of each query tile
        bool ok = true;
        do {
            const int jbeg = first_block(pl), nkv = num_blocks(pl);
            if (nkv == 0) continue;
            if constexpr (kTurnQ) {
                // A row's largest element goes to [2^14, 2^15): elements down to 2^-28
                // of it keep all bits, smaller ones are off by 2^-39 of it.
                for (int t = 0; t < C::TILES && ok; ++t) {
                    if (!(t ? pl.jhi1 > pl.jlo1 : pl.jhi0 > pl.jlo0)) continue;
                    ok = mbar_wait_warp(&bar_q[t], (t ? q_n1 : q_n0) & 1, s_abort);
                    if (!ok) break;
                    (t ? q_n1 : q_n0) += 1;
#pragma unroll 1
                    for (int r = tid; r < kTileRows; r += 64) {
                        auto piece = [&](int c) {
                            return reinterpret_cast<uint4*>(sQ + t * C::TILE + (c >> 3) * C::CB_BYTES + r * 128 +
                                                            (((c & 7) ^ (r & 7)) << 4));
                        };
                        uint32_t top = 0;   // largest magnitude, as bf16 bits in either half
#pragma unroll 4
                        for (int c = 0; c < D / 8; ++c) {
                            const uint4 v = *piece(c);
                            top = __vmaxu2(__vmaxu2(top, __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu)),
                                           __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
                        }
                        top = max(top & 0xffffu, top >> 16);
                        const int ea = max(static_cast<int>(top >> 7) - 127, -100);
                        const float up = exp2_int(14 - ea);
                        s_turn[((units8 & 1) * 2 + t) * kTileRows + r] = static_cast<int8_t>(ea - 14);
#pragma unroll 4
                        for (int c = 0; c < D / 8; ++c) {
                            uint4* const at = piece(c);
                            const uint4 v = *at;
                            auto turn = [&](uint32_t w) { return pack_f16x2(bf16lo_to_f32(w) * up, bf16hi_to_f32(w) * up); };
                            *at = make_uint4(turn(v.x), turn(v.y), turn(v.z), turn(v.w));
                        }
                    }
                    fence_proxy_async_smem();
                    mbar_arrive_warp(&q_turned[t]);
                }
                if (!ok) break;
            }
            ++units8;
            for (int j = jbeg; j < jbeg + nkv && ok; ++j, ++blk) {
                ok = mbar_wait_warp_soon(&meta_full[blk & 1], (blk >> 1) & 1, s_abort);
                for (int u = 0; u < 2 * C::UNITS && ok; ++u, ++raw) {
                    const int which = u / C::UNITS, part = u % C::UNITS;
                    const int from = raw % C::NRAW;
                    ok = mbar_wait_warp_soon(&raw_full[from], (raw / C::NRAW) & 1, s_abort);
                    if (!ok) break;
                    if (part == 0) {   // the slot is free
                        if constexpr (kBlockRelease) {
                            const int bi = fills / 2;
                            const int wb = which == 0 ? bi - kPairs : bi - kPairs + 1;
                            ok = bi < kPairs || mbar_wait_warp_soon(&empty[wb % kPairs], (wb / kPairs) & 1, s_abort);
                        } else {
                            ok = mbar_wait_warp_soon(&empty[fills % C::NSLOT], ((fills / C::NSLOT) & 1) ^ 1, s_abort);
                        }
                        if (!ok) break;
                    }
                    const int half = (part & 1) * 64;   // first row
                    const int lo = pl.klo - j * kTileRows - half, hi = pl.khi - j * kTileRows - half;
                    const uint8_t* const src = src0 + from * C::RAW;
                    uint8_t* const dst = dst0 + (fills % C::NSLOT) * C::TILE + (part >> 1) * 2 * C::CB_BYTES + half * 128;
                    const uint32_t* const f = const_cast<const uint32_t*>(&wide.factor[blk & 1][(half + r0) / 8].x) + which;
                    constexpr int PIECES = 64 / STEP;   // all asked for before the first is used
                    uint4 v[PIECES];
                    auto put = [&](int i, const uint32_t (&w)[8]) {
                        *reinterpret_cast<uint4*>(dst + STEP * i * 128 + d0) = make_uint4(w[0], w[1], w[2], w[3]);
                        *reinterpret_cast<uint4*>(dst + STEP * i * 128 + d1) = make_uint4(w[4], w[5], w[6], w[7]);
                    };
                    // Most blocks lie within what is attended and have pages of one
                    // scale: less than half the instructions.
                    if (lo <= 0 && hi >= 64 && (wide.plain[blk & 1] >> which & 1)) {
#pragma unroll
                        for (int i = 0; i < PIECES; ++i)
                            v[i] = *reinterpret_cast<const uint4*>(src + STEP * i * C::RAW_COLS);
#pragma unroll
                        for (int i = 0; i < PIECES; ++i) {
                            uint32_t w[8];
                            e4m3x16_to_f16(v[i], w);
                            put(i, w);
                        }
                    } else {
                        uint32_t m[PIECES];
#pragma unroll
                        for (int i = 0; i < PIECES; ++i) {
                            const int r = r0 + STEP * i;
                            v[i] = make_uint4(0u, 0u, 0u, 0u);   // outside what is attended: whatever is there, even NaN
                            if (r >= lo && r < hi) v[i] = *reinterpret_cast<const uint4*>(src + STEP * i * C::RAW_COLS);
                            m[i] = f[STEP / 4 * i];
                        }
#pragma unroll
                        for (int i = 0; i < PIECES; ++i) {
                            uint32_t w[8];
                            e4m3x16_to_f16(v[i], w);
#pragma unroll
                            for (int e = 0; e < 8; ++e) w[e] = mul_f16x2(w[e], m[i]);
                            put(i, w);
                        }
                    }
                    mbar_arrive_warp(&raw_empty[from]);
                    if (part == C::UNITS - 1) {
                        if (which == 1) mbar_arrive_warp(&meta_empty[blk & 1]);
                        fence_proxy_async_smem();
                        mbar_arrive_warp(&full[fills % C::NSLOT]);
                        ++fills;
                    }
                }
            }
        } while (ok && next_unit());
    } else {
        // ================= softmax (one or two threads per row) =================
        const int t = warp / (C::ROW_THREADS / 32);
        const int part = C::PARTS == 1 ? 0 : (warp >> 2) % C::PARTS;   // keys c0 .. c0 + NC, output columns likewise
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const int c0 = part * C::NC;
        const int tl = r / G;                       // token within the query tile
        const int rg = r - tl * G;                  // head within the group
        const int W = p.window;
        const int bar = 1 + t;                      // hardware barrier of the tile's softmax threads
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t t_S = t_lane + 128u * t + c0;
        const uint32_t t_P = t_lane + 128u * t + c0 / 2;
        const uint32_t t_O = t_lane + C::O_COL + D * t + part * C::DC;
        float* const x_mine = s_max + (t * C::PARTS + part) * kTileRows + r;
        float* const x_other = s_max + (t * C::PARTS + (part ^ 1)) * kTileRows + r;
        int g = 0;       // K/V blocks of the units before
        int s_n = 0;     // blocks of this query tile in them
        int o_n = 0;     // of them with blocks of this query tile
        int u_n = 0;     // units before
        int t_n = 0;     // of them with blocks
        bool ok = true;  // of the warp; a tile's warps agree on it at a unit's end
        do {
        const int L = pl.L, klo = pl.klo, khi = pl.khi;
        const int jlo = t ? pl.jlo1 : pl.jlo0, jhi = t ? pl.jhi1 : pl.jhi0;
        const int first_pos = pl.tok0 + t * TT + L - pl.N, last_pos = first_pos + TT - 1;
        const int pos = first_pos + tl;
        const int fill0 = 2 * (g - first_block(pl)) + 1;   // ring fill of V_j: fill0 + 2 j
        const int s_b = s_n - jlo;                         // parity of S_j: (s_b + j) & 1
        float turn = 1.f;                                  // (kFp8) the row's power of two
        float m_ref = -INFINITY;   // reference, log2 units of scaled scores: a maximum less kWeightShift
        float l = 0.f;             // of this thread's keys
        // A failed wait leaves the results unspecified.  Where a tile's warps meet
        // at barriers the warp goes on to the unit's end all the same.
        for (int j = jlo; j < jhi; ++j) {
            const int k0 = j * kTileRows;
            ok = ok && mbar_wait_warp(&bar_s[t], (s_b + j) & 1, s_abort);
            if (C::PARTS == 1 && !ok) break;
            tc_fence_after();
            // Factor of the scores and (kFp8) exponent of V's scale: weights are taken
            // times 2^ev, references are of s + ev, and the sum takes 2^ev off again.
            float sc = p.scale_log2, ev = 0.f;
            if constexpr (kFp8) {
                if (kTurnQ && j == jlo) turn = exp2_int(s_turn[((t_n & 1) * 2 + t) * kTileRows + r]);
                volatile const float2& block = wide.block[(g - first_block(pl) + j) & 7];
                sc = score_factor(block.x * turn);
                ev = block.y;
            }
            // V rows outside [klo, khi) become zero.  Only after S_j: by then
            // every earlier fill of V_j's slot has been waited for, so that
            // the parity below can only mean this one.
            if (!kFp8 && (k0 < klo || k0 + kTileRows > khi)) {
                const int fill = fill0 + 2 * j;
                const int slot = fill % C::NSLOT;
                ok = ok && mbar_wait_warp(&full[slot], (fill / C::NSLOT) & 1, s_abort);
                if (C::PARTS == 1 && !ok) break;
                if (ok && (k0 + r < klo || k0 + r >= khi)) {
                    for (int cb = part; cb < C::NCB; cb += C::PARTS) {
                        const int at = kFine ? (r >> 3) * 8 * C::ROWB + cb * 1024 + (r & 7) * 128
                                              : cb * C::CB_BYTES + r * 128;
                        uint4* row = reinterpret_cast<uint4*>(sKV + slot * C::TILE + at);
#pragma unroll
                        for (int e = 0; e < 8; ++e) row[e] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_proxy_async_smem();
            }
            const bool wmask = W > 0 && (k0 < last_pos - W + 1 ||
                                         (!p.causal && k0 + kTileRows - 1 > first_pos + W - 1));
            const bool tile_mask = k0 + kTileRows > L ||
                                   (p.causal && k0 + kTileRows - 1 > first_pos) || wmask;
            // keys >= lim and < lo of this thread's are masked (only on masked tiles)
            int lim = tile_mask ? (p.causal ? min(L, pos + 1) : L) - k0 - c0 : C::NC;
            int lo = 0;
            if (wmask) {
                lo = pos - W + 1 - k0 - c0;
                if (!p.causal) lim = min(lim, pos + W - k0 - c0);
            }

            bool uneven = false;   // (where a row has one thread, a function does all of such a block)
            if constexpr (kFp8) {
                if (__builtin_expect(ev == kUneven, 0)) {
                    const volatile int16_t* const exponents = &wide.exponents[(g - first_block(pl) + j) & 7][c0 / 8];
                    if constexpr (C::PARTS == 1) {
                        const float2 ml = uneven_block(t_S, t_P, t_O, j > jlo ? D : 0, exponents, p.scale_log2, turn, lo,
                                                       lim, m_ref, l);
                        m_ref = ml.x;
                        l = ml.y;
                        tc_fence_before();
                        mbar_arrive_warp(&bar_p[t]);
                        continue;
                    }
                    uneven_scores(t_S, C::NC / 8, exponents, p.scale_log2, turn);
                    sc = 1.f;
                    ev = 0.f;
                    uneven = true;
                }
            }

            // ---- row max ----
            float mx;
            uint32_t sr[C::NC / 32][32];
            {
#pragma unroll
                for (int c = 0; c < C::NC / 32; ++c) tmem_ld32(t_S + 32 * c, sr[c]);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < C::NC / 32; ++c) reg_fence(sr[c]);
                if (tile_mask) {
#pragma unroll
                    for (int c = 0; c < C::NC; ++c)
                        if (c >= lim || c < lo) sr[c >> 5][c & 31] = __float_as_uint(-INFINITY);
                }
                float mp[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) mp[k] = -INFINITY;
#pragma unroll
                for (int c = 0; c < C::NC; c += 2)
                    mp[(c >> 1) & 7] = max3f(mp[(c >> 1) & 7], __uint_as_float(sr[c >> 5][c & 31]),
                                             __uint_as_float(sr[c >> 5][(c & 31) + 1]));
                mx = max3f(max3f(mp[0], mp[1], mp[2]), max3f(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7]));
            }
            float m_new = fmaxf(m_ref, kFp8 ? fmaf(mx, sc, ev - kWeightShift<kMmaF16>)
                                            : mx * p.scale_log2 - kWeightShift<kMmaF16>);
            float alpha = 1.f;
            bool warp_rescale = false;
            auto adopt = [&]() {
                const bool want = (m_ref != -INFINITY) && (m_new > m_ref + kRescaleThreshold);
                warp_rescale = __any_sync(0xffffffffu, want);
                if (m_ref == -INFINITY) {
                    m_ref = m_new;   // O and l are still zero: adopt without rescaling
                } else if (warp_rescale) {
                    alpha = ex2_approx(m_ref - m_new);
                    m_ref = m_new;
                }
            };
            if constexpr (C::PARTS == 1) {
                adopt();
            } else {
                // The barrier that asks whether any row of the tile needs a new
                // reference (its first keys, or a score 2^8 above the old one)
                // is also what lets P overwrite S: all of it is read.
                tc_fence_before();
                if (named_barrier_or(bar, C::ROW_THREADS, m_new > m_ref + kRescaleThreshold)) {
                    *x_mine = m_new;
                    named_barrier_sync(bar, C::ROW_THREADS);
                    m_new = fmaxf(m_new, *x_other);
                    adopt();
                }
                tc_fence_after();
            }
            const float neg_m = (m_ref == -INFINITY) ? 0.f : -m_ref;

            // ---- P = exp2(s scale log2e - m), rounded to the storage type for
            // the P V product; the row sum adds the unrounded P ----
            const uint64_t sc2 = f2_pack(sc, sc);
            const float nm = kFp8 ? neg_m + ev : neg_m;
            const uint64_t nm2 = f2_pack(nm, nm);
            float take = exp2_int(-static_cast<int>(ev));   // what the weights were taken times, off again
            uint64_t acc2[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) acc2[k] = f2_pack(0.f, 0.f);
#pragma unroll
            for (int c8 = 0; c8 < C::NC / 16; ++c8) {   // 16 keys, 8 packed words
                uint32_t pk[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int c = 16 * c8 + 2 * e;
                    float x0, x1;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[c >> 5][c & 31]),
                                             __uint_as_float(sr[c >> 5][(c & 31) + 1])),
                                     sc2, nm2),
                              x0, x1);
                    x0 = ex2_approx(x0);
                    x1 = ex2_approx(x1);
                    pk[e] = pack_h2<kMmaF16>(x0, x1);
                    if constexpr (kFp8 && C::PARTS > 1) {
                        if ((e & 3) == 0 && uneven)
                            take = exp2_int(-exponent_v(wide.exponents[(g - first_block(pl) + j) & 7][c0 / 8 + 2 * c8 + e / 4]));
                        acc2[e & 3] = f2_fma(f2_pack(x0, x1), f2_pack(take, take), acc2[e & 3]);
                    } else {
                        acc2[e & 3] = f2_add(acc2[e & 3], f2_pack(x0, x1));
                    }
                }
                tmem_st8(t_P + 8 * c8, pk);
            }
            float rowsum;
            {
                float a0, a1, a2, a3;
                f2_unpack(f2_add(acc2[0], acc2[1]), a0, a1);
                f2_unpack(f2_add(acc2[2], acc2[3]), a2, a3);
                rowsum = (a0 + a1) + (a2 + a3);
            }
            if constexpr (kFp8 && C::PARTS == 1) rowsum *= exp2_int(-static_cast<int>(ev));
            l = l * alpha + rowsum;
            if (warp_rescale && j > jlo) {   // O row *= alpha (PV of block j-1 is complete)
#pragma unroll
                for (int c = 0; c < C::DC / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(t_O + 32 * c, o);
                    tmem_ld_wait();
                    reg_fence(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                    tmem_st32(t_O + 32 * c, o);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive_warp(&bar_p[t]);
        }
        // ---- epilogue: O = acc / l and the log-sum-exp, or a piece of them ----
        const bool any = jhi > jlo;
        if (ok && any) {
            ok = mbar_wait_warp(&bar_o[t], o_n & 1, s_abort);
            tc_fence_after();
        }
        if (joined && p.cluster > 0)   // the ring and the queries are free once every product is done
            ok = mbar_wait_warp(bar_fin, 0, s_abort) && ok;
        if constexpr (C::PARTS > 1) {   // the sum over all keys of the row
            float* const sums = s_sum + (u_n & 1) * C::ROW_FLOATS + t * C::ROW_THREADS + r;
            sums[part * kTileRows] = l;
            ok = !named_barrier_or(bar, C::ROW_THREADS, !ok);
            l = sums[0] + sums[kTileRows];
            ++u_n;
        }
        t_n += num_blocks(pl) > 0;
        g += num_blocks(pl);
        s_n += jhi - jlo;
        o_n += any;
        if (ok) {
            const int tok = pl.tok0 + t * TT + tl;
            const bool row_ok = tl < TT && tok < pl.N;
            const int head = pl.hk * G + rg;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const size_t piece_row =
                (static_cast<size_t>(unit) * p.splits + split) * p.slot_rows + t * kTileRows + r;
            const size_t out_row = (static_cast<size_t>(pl.start) + tok) * p.lq.H + head;
            uint32_t o[32];
#pragma unroll
            for (int c = 0; c < C::DC / 32; ++c) {
                __syncwarp();   // rows past the tile's end skip the stores below
                if (any) {
                    tmem_ld32(t_O + 32 * c, o);
                    tmem_ld_wait();
                    reg_fence(o);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                }
                if (joined && p.cluster > 0) {
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        *reinterpret_cast<float4*>(piece_group(t * kTileRows + r, part * (C::DC / 4) + 8 * c + v)) =
                            make_float4(__uint_as_float(o[4 * v]) * inv, __uint_as_float(o[4 * v + 1]) * inv,
                                        __uint_as_float(o[4 * v + 2]) * inv, __uint_as_float(o[4 * v + 3]) * inv);
                } else if (row_ok && joined) {
                    float4* dst = reinterpret_cast<float4*>(p.part_o + piece_row * D + part * C::DC + 32 * c);
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        dst[v] = make_float4(__uint_as_float(o[4 * v]) * inv, __uint_as_float(o[4 * v + 1]) * inv,
                                             __uint_as_float(o[4 * v + 2]) * inv,
                                             __uint_as_float(o[4 * v + 3]) * inv);
                } else if (row_ok) {
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.O) + out_row * D + part * C::DC + 32 * c);
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack_h2<kF16>(__uint_as_float(o[8 * v + 2 * e]) * inv,
                                                 __uint_as_float(o[8 * v + 2 * e + 1]) * inv);
                        dst[v] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            const float lse2 = l == 0.f ? -INFINITY : m_ref + log2f(l);
            if (joined && p.cluster > 0) {
                if (part == 0) s_lse[t * kTileRows + r] = lse2;
            } else if (row_ok && part == 0) {
                if (joined) p.part_lse[piece_row] = lse2;
                else p.LSE[static_cast<size_t>(head) * p.lq.total + pl.start + tok] = lse2 * kLn2;
            }
        }
        // O_t is read: the next unit's first P V, which overwrites it, waits for P of
        // these threads.
        tc_fence_before();
        } while (ok && next_unit());
    }

    if (joined && p.cluster > 0) {
        __syncwarp();
        join_cluster();
    }
    // ---- teardown ----
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == C::MMA_WARP) tmem_dealloc(tmem, C::TMEM_COLS);
    if (threadIdx.x == 0 && *s_abort && p.dev_status != nullptr)
        atomicCAS(p.dev_status, 0, static_cast<int>(ATTN_ERR_DEVICE_TIMEOUT));
}

template <int D, bool kF16, int kTiles, bool kFine, bool kLoop, bool kFp8 = false>
cudaError_t launch_paged_t(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const PagedParams& p, cudaStream_t stream) {
    using C = PagedCfg<D, kF16, kTiles, kFp8>;
    auto kern = attn_paged_kernel<D, kF16, kTiles, kFine, kLoop, kFp8>;
    static std::atomic<unsigned long long> smem_ready{0};
    const cudaError_t e = enable_smem_per_device(kern, C::SMEM, smem_ready);
    if (e != cudaSuccess) return e;
    const unsigned units = static_cast<unsigned>(p.tiles) * static_cast<unsigned>(p.Hkv);
    const unsigned grid = kLoop ? (units < kSMs ? units : kSMs) : units * static_cast<unsigned>(p.splits);
    return launch_overlapped_cluster(kern, grid, C::THREADS, C::SMEM, p.cluster, true, stream, tq, tk, tv, p);
}

// One unit per CTA or group of CTAs, or (p.splits = 1) a persistent CTA per SM.
template <int D, int kTiles, bool kFine>
cudaError_t launch_paged_f(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const PagedParams& p, bool f16, cudaStream_t s) {
    if (p.splits == 1)
        return f16 ? launch_paged_t<D, true, kTiles, kFine, true>(tq, tk, tv, p, s)
                   : launch_paged_t<D, false, kTiles, kFine, true>(tq, tk, tv, p, s);
    return f16 ? launch_paged_t<D, true, kTiles, kFine, false>(tq, tk, tv, p, s)
               : launch_paged_t<D, false, kTiles, kFine, false>(tq, tk, tv, p, s);
}

template <int D, int kTiles>
cudaError_t launch_paged_8(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p,
                           bool f16, cudaStream_t s) {
    if (p.splits == 1)
        return f16 ? launch_paged_t<D, true, kTiles, false, true, true>(tq, tk, tv, p, s)
                   : launch_paged_t<D, false, kTiles, false, true, true>(tq, tk, tv, p, s);
    return f16 ? launch_paged_t<D, true, kTiles, false, false, true>(tq, tk, tv, p, s)
               : launch_paged_t<D, false, kTiles, false, false, true>(tq, tk, tv, p, s);
}

}  // namespace
}  // namespace gbattn
