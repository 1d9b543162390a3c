// attn_decode_kernel.cuh — attention of a few new tokens per request (single
// tokens, drafted tokens) over a paged key/value cache.
//
// With n = tokens x G query rows per request and key/value head, n <= 64, the
// work is to read the cache once: 4 n flops per 16-bit element of K or V are
// far below what the tensor cores do in the time that the element takes to
// arrive.  So everything serves the stream of K and V tiles:
//   * Transposed products.  S^T = K Q^T puts keys on the 128 tensor-memory
//     lanes and the n rows on N = 16, 32 or 64 columns, so a thread handles
//     one key and N exponentials (not one row and 128 of them, of which only
//     n / 128 would count), and O^T = V^T P^T keeps the head dim on the lanes.
//     K and V are the 128-row operands, read from shared memory as they come.
//   * The row maximum runs over lanes.  A row keeps its reference maximum
//     until a score exceeds it by 2^8, which one barrier with a vote finds
//     out; only then are maxima reduced and O rescaled.  Row sums stay in
//     each thread and are reduced once at the end.
//   * One persistent CTA per SM.  The key blocks of all requests and heads, in
//     order, are cut into as many equal runs as there are CTAs: a CTA takes a
//     run, whatever the request lengths are.  Tiles (request, head) cut by a run's
//     end are joined by a second launch (paged_join_kernel), at most two
//     pieces per CTA.
//   * The producer runs ahead over the ends of tiles: a ring of up to 176 KB
//     of K/V tiles is in flight while the other warps finish a tile.
//
// Warps 0-3: softmax, one key per thread.  Warp 4: TMA producer; walks the
// run, tells the others each segment (a tile's part of the run).  Warp 5: MMA.
#pragma once

#include "attn_fwd_kernel.cuh"
#include "paged.cuh"

namespace gbattn {
namespace {

template <int D, int N>
struct DecodeCfg {
    static constexpr int CHUNKS = D == 256 ? 2 : 1;          // ring slots of one tile
    static constexpr int CW = D / CHUNKS;                    // head-dim columns of a slot
    static constexpr int CCB = CW / 64;                      // 128-byte column blocks of a slot
    static constexpr int CB_BYTES = kTileRows * 128;
    static constexpr int SLOT = CCB * CB_BYTES;
    static constexpr int QCB_BYTES = N * 128;                // Q: column blocks of N rows
    static constexpr int Q_BYTES = (D / 64) * QCB_BYTES;
    static constexpr int P_BYTES = kTileRows * 128;          // P^T: 128 keys of up to 64 rows
    static constexpr int MISC = 2048;                        // barriers, segments, row values
    static constexpr int AVAIL = 232448 - 1024 - MISC - 2 * Q_BYTES - 2 * P_BYTES;
    static constexpr int NSLOT = AVAIL / SLOT < 11 ? AVAIL / SLOT : 11;
    static constexpr int SMEM = 2 * Q_BYTES + 2 * P_BYTES + NSLOT * SLOT + MISC + 1024;
    static constexpr int HALVES = D == 256 ? 2 : 1;          // 128-lane halves of O^T
    static constexpr uint32_t O_COL = 2 * N;                 // S^T in [0, 2N), two buffers
    static constexpr uint32_t TMEM_COLS = 4 * N;
    static constexpr int THREADS = 192;
    static_assert(NSLOT >= 4, "K and V of two blocks in flight");
};

// One tile's part of a CTA's run.
struct Segment {
    int q_start, ntok, hk;   // packed row of the request's first token, its tokens, K/V head
    int off, L;              // query i stands at key off + i; keys of the request
    int klo, khi;            // keys that its queries attend between them
    int j0, nblk;            // first key block and number of blocks; nblk = 0: no more segments
    int out;                 // -1: the whole tile, written to O; else the slot of a piece
    int none;                // the queries attend no key
};

// Key blocks of request b per key/value head: at least one if it has queries,
// so that every row is written.
struct Request {
    int start, n, L, klo, khi, j0, units;
};
__device__ __forceinline__ Request request_of(const PagedParams& p, int b) {
    Request r;
    const SeqSpan sq = seq_span(p.lq, b, nullptr, false);
    r.start = sq.start;
    r.n = sq.len;
    r.L = paged_keys(p, b);
    r.klo = r.khi = 0;
    if (r.n > 0) key_range(p, 0, r.n - 1, r.L - r.n, r.L, r.klo, r.khi);
    r.j0 = r.klo / kTileRows;
    r.units = r.n > 0 ? max(1, (r.khi + kTileRows - 1) / kTileRows - r.j0) : 0;
    return r;
}

// Reference maximum of a row that has met no key: finite, so that a masked
// score minus it is still -inf, and below every score.
constexpr float kNoMax = -3.402823466e38f;

// Order-preserving map of floats to integers, for an integer maximum over the
// warp.
__device__ __forceinline__ int float_key(float x) {
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float key_float(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

// Sums of v[0..N) over the warp, scattered: after it, lane x holds in v[0]
// (and v[1] for N = 64) the sum of column `col` (and col + 1).
template <int N>
__device__ __forceinline__ int warp_sum_scatter(float (&v)[N], int lane) {
    int col = 0;
    int width = N;
#pragma unroll
    for (int step = 16; step >= 1; step >>= 1) {
        if (width > 1) {
            width >>= 1;
            const bool up = (lane & step) != 0;
#pragma unroll
            for (int c = 0; c < N / 2; ++c)
                if (c < width) {
                    const float mine = up ? v[c + width] : v[c];
                    const float theirs = up ? v[c] : v[c + width];
                    v[c] = mine + __shfl_xor_sync(0xffffffffu, theirs, step);
                }
            if (up) col += width;
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], step);
        }
    }
    return col;
}

template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t t, uint32_t (&r)[N]) {
    if constexpr (N == 16) {
        tmem_ld16(t, r);
    } else {
#pragma unroll
        for (int c = 0; c < N / 32; ++c) tmem_ld32(t + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&r[32 * c]));
    }
}
template <int N>
__device__ __forceinline__ void tmem_st_cols(uint32_t t, const uint32_t (&r)[N]) {
    if constexpr (N == 16) {
        tmem_st16(t, r);
    } else {
#pragma unroll
        for (int c = 0; c < N / 32; ++c)
            tmem_st32(t + 32 * c, *reinterpret_cast<const uint32_t(*)[32]>(&r[32 * c]));
    }
}

template <int D, bool kF16, int N>
__global__ void __launch_bounds__(DecodeCfg<D, N>::THREADS, 1)
    attn_decode_kernel(const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const PagedParams p) {
    using C = DecodeCfg<D, N>;
    constexpr int kSoftmax = 128;   // threads of warps 0-3
    constexpr uint32_t FMT = fmt16<kF16>();
    constexpr uint32_t IDESC_S = idesc_f32acc(128, N, FMT, false, false);
    constexpr uint32_t IDESC_O = idesc_f32acc(128, N, FMT, true, true);
    grid_dep_wait();
    grid_dep_launch_dependents();   // the join: it waits for this grid itself
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sKV = smem;
    uint8_t* sP = sKV + C::NSLOT * C::SLOT;      // two buffers
    uint8_t* sQ = sP + 2 * C::P_BYTES;           // two buffers
    uint64_t* bars = reinterpret_cast<uint64_t*>(sQ + 2 * C::Q_BYTES);
    uint64_t* q_full = bars;            // [2] a segment and its queries are there
    uint64_t* q_empty = bars + 2;       // [2] every role is done with them
    uint64_t* s_full = bars + 4;        // [2] S^T of a block
    uint64_t* p_full = bars + 6;        // [2] P^T of a block (V's edge cleared)
    uint64_t* pv_done = bars + 8;       // [2] O^T += V^T P^T of a block
    uint64_t* bar_fin = bars + 10;
    uint64_t* full = bars + 11;         // [NSLOT]
    uint64_t* empty = full + 11;        // [NSLOT]
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(empty + 11);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    volatile Segment* s_seg = reinterpret_cast<volatile Segment*>(bars + 36);   // [2]
    float* s_row = reinterpret_cast<float*>(bars + 48);   // [4][N]: maxima, then sums, of each warp
    float* s_m = s_row + 4 * N;       // [N] reference maxima, log2 units
    float* s_fac = s_m + N;           // [N] factors: of a rescale, then 1 / l
    long long* s_scan = reinterpret_cast<long long*>(s_row);                    // set-up only
    static_assert(2 * sizeof(Segment) <= 12 * 8, "segments fit their place");
    static_assert(48 * 8 + 6 * N * 4 <= C::MISC, "row values fit their place");

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int cta = static_cast<int>(blockIdx.x);
    const int ctas = static_cast<int>(gridDim.x);

    // ---- this CTA's run [u0, u1) of the key blocks of all requests and heads ----
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 1 + kSoftmax);
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], kSoftmax);
            mbar_init(&pv_done[s], 1);
        }
        mbar_init(bar_fin, 1);
        for (int s = 0; s < C::NSLOT; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        *s_abort = 0;
        fence_mbar_init();
    }
    if (warp == 5) {
        tmem_alloc(s_tmem, C::TMEM_COLS);
        tmem_relinquish();
    }
    // Block sum (total of x) and exclusive prefix of the calling thread.
    auto block_scan = [&](long long x, long long& total) {
        long long incl = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        __syncthreads();
        if (lane == 31) s_scan[warp] = incl;
        __syncthreads();
        long long before = 0;
        total = 0;
#pragma unroll
        for (int w = 0; w < C::THREADS / 32; ++w) {
            if (w < warp) before += s_scan[w];
            total += s_scan[w];
        }
        return before + incl - x;
    };
    long long all = 0, mine = 0, excl = 0;
    for (int b0 = 0; b0 < p.B; b0 += C::THREADS) {
        const int b = b0 + static_cast<int>(threadIdx.x);
        mine = b < p.B ? static_cast<long long>(request_of(p, b).units) * p.Hkv : 0;
        long long total;
        excl = block_scan(mine, total);
        all += total;
    }
    // No run is empty: the pieces of a tile are in consecutive CTAs.
    const long long parts = min(all, static_cast<long long>(ctas));
    const long long u0 = cta < parts ? all * cta / parts : 0;
    const long long u1 = cta < parts ? all * (cta + 1) / parts : 0;
    // request that holds unit u0, and where it starts
    long long* s_at = s_scan + 8;
    if (p.B <= C::THREADS) {   // one round: the sums of above
        if (excl <= u0 && u0 < excl + mine) {
            s_at[0] = threadIdx.x;
            s_at[1] = excl;
        }
    } else {
        long long done = 0;
        for (int b0 = 0; b0 < p.B && done <= u0; b0 += C::THREADS) {
            const int b = b0 + static_cast<int>(threadIdx.x);
            mine = b < p.B ? static_cast<long long>(request_of(p, b).units) * p.Hkv : 0;
            long long total;
            excl = done + block_scan(mine, total);
            if (excl <= u0 && u0 < excl + mine) {
                s_at[0] = b;
                s_at[1] = excl;
            }
            done += total;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp == 4) {
        // ================= producer =================
        const long long at_b = s_at[0], at_u = s_at[1];
        __syncwarp();
        if (lane == 0) p.desc[cta].n = 0;
        int fills = 0;    // ring slots filled so far
        int seg = 0;
        bool ok = true;
        if (u0 < u1) {
            if (lane == 0) {
                tma_prefetch_desc(&tmQ);
                tma_prefetch_desc(&tmK);
                tma_prefetch_desc(&tmV);
            }
            // lane x holds request win + x
            int win = static_cast<int>(at_b), b = win;
            Request held = win + lane < p.B ? request_of(p, win + lane) : Request{0, 0, 0, 0, 0, 0, 0};
            int in_req = static_cast<int>(u0 - at_u);   // unit within the request: hk * units + block
            long long u = u0;
            while (u < u1 && ok) {
                Request r;
                {
                    const int x = b - win;
                    r.start = __shfl_sync(0xffffffffu, held.start, x);
                    r.n = __shfl_sync(0xffffffffu, held.n, x);
                    r.L = __shfl_sync(0xffffffffu, held.L, x);
                    r.klo = __shfl_sync(0xffffffffu, held.klo, x);
                    r.khi = __shfl_sync(0xffffffffu, held.khi, x);
                    r.j0 = __shfl_sync(0xffffffffu, held.j0, x);
                    r.units = __shfl_sync(0xffffffffu, held.units, x);
                }
                const int hk = in_req / r.units, blk = in_req - hk * r.units;
                const int nblk = static_cast<int>(min(static_cast<long long>(r.units - blk), u1 - u));
                const bool whole = nblk == r.units;
                const bool none = r.khi <= r.klo;
                const int buf = seg & 1;
                ok = seg < 2 || mbar_wait_warp(&q_empty[buf], ((seg >> 1) & 1) ^ 1, s_abort);
                if (!ok) break;
                if (lane == 0) {
                    volatile Segment& s = s_seg[buf];
                    s.q_start = r.start;
                    s.ntok = r.n;
                    s.hk = hk;
                    s.off = r.L - r.n;
                    s.L = r.L;
                    s.klo = r.klo;
                    s.khi = r.khi;
                    s.j0 = r.j0 + blk;
                    s.nblk = nblk;
                    s.out = whole ? -1 : 2 * cta + (blk == 0 ? 1 : 0);
                    s.none = none;
                    if (!whole && blk == 0) {   // this CTA has the tile's first piece
                        const long long end = u + r.units;
                        const long long last = (end * parts + all - 1) / all - 1;   // CTA that ends it
                        p.desc[cta] = PieceDesc{r.start, 0, r.n, hk, static_cast<int>(last) - cta + 1,
                                                2 * cta + 1, 2 * cta + 2, 2};
                    }
                    if (none) {
                        mbar_arrive(&q_full[buf]);
                    } else {
                        mbar_arrive_expect_tx(&q_full[buf],
                                              static_cast<uint32_t>(p.tile_tokens * p.G) * (2 * D));
                        for (int cb = 0; cb < D / 64; ++cb)
                            tma_load_3d(sQ + buf * C::Q_BYTES + cb * C::QCB_BYTES, &tmQ, &q_full[buf],
                                        cb * 64, hk * p.G, r.start);
                    }
                }
                __syncwarp();
                if (!none) {
                    const int32_t* table = p.page_table + static_cast<size_t>(b) * p.max_pages;
                    const int jbeg = r.j0 + blk;
                    PageBox box = page_box(p, table, jbeg * kTileRows, r.klo, r.khi, lane);
                    for (int j = jbeg; j < jbeg + nblk && ok; ++j) {
                        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, box.needed)) *
                                               static_cast<uint32_t>(p.box_rows) * (2 * C::CW);
                        PageBox next = box;
                        if (j + 1 < jbeg + nblk) next = page_box(p, table, (j + 1) * kTileRows, r.klo, r.khi, lane);
                        for (int part = 0; part < 2 * C::CHUNKS; ++part) {   // K, then V
                            const int slot = fills % C::NSLOT;
                            const uint32_t ph = (fills / C::NSLOT) & 1;
                            if (!mbar_wait_warp(&empty[slot], ph ^ 1, s_abort)) {
                                ok = false;
                                break;
                            }
                            if (lane == 0) mbar_arrive_expect_tx(&full[slot], bytes);
                            __syncwarp();
                            if (box.needed) {
                                const CUtensorMap* m = part < C::CHUNKS ? &tmK : &tmV;
                                const int c0 = (part % C::CHUNKS) * C::CW;
                                uint8_t* dst = sKV + slot * C::SLOT + lane * p.box_rows * 128;
                                for (int cb = 0; cb < C::CCB; ++cb)
                                    tma_load_4d(dst + cb * C::CB_BYTES, m, &full[slot], c0 + cb * 64, box.row,
                                                hk, box.page);
                            }
                            __syncwarp();
                            ++fills;
                        }
                        box = next;
                    }
                }
                ++seg;
                u += nblk;
                in_req += nblk;
                if (in_req == r.units * p.Hkv && u < u1) {   // next request with queries
                    in_req = 0;
                    int nb = -1;
                    int from = b + 1;
                    while (nb < 0 && from < p.B) {
                        if (from >= win + 32) {
                            win = from;
                            held = win + lane < p.B ? request_of(p, win + lane) : Request{0, 0, 0, 0, 0, 0, 0};
                        }
                        const unsigned has = __ballot_sync(0xffffffffu, win + lane >= from && held.units > 0);
                        if (has != 0) nb = win + __ffs(has) - 1;
                        else from = win + 32;
                    }
                    if (nb < 0) break;   // cannot happen: the run ends inside the last request
                    b = nb;
                }
            }
        }
        // no more segments
        bool told = false;
        if (ok && (seg < 2 || mbar_wait_warp(&q_empty[seg & 1], ((seg >> 1) & 1) ^ 1, s_abort))) {
            if (lane == 0) {
                s_seg[seg & 1].nblk = 0;
                mbar_arrive(&q_full[seg & 1]);
            }
            told = true;
        }
        // Drain: every load this warp issued has landed before teardown.  Once
        // the others have been told, segment seg - 2 is known to be there (and
        // its barrier has moved on).
        if (lane == 0) {
            volatile int no_abort = 0;
            for (int s = max(0, seg - (told ? 1 : 2)); s < seg; ++s) mbar_wait(&q_full[s & 1], (s >> 1) & 1, &no_abort);
            for (int s = 0; s < C::NSLOT && s < fills; ++s) {
                const int uses = (fills - s + C::NSLOT - 1) / C::NSLOT;
                mbar_wait(&full[s], (uses - 1) & 1, &no_abort);
            }
        }
        __syncwarp();
    } else if (warp == 5) {
        // ================= MMA issuer =================
        if (lane == 0) {
            const uint64_t dk0 = sdesc_sw128(smem_u32(sKV), 16, 1024);
            // V^T: 64 head-dim columns, the next 64 a column block on (for
            // d = 64 the same again: lanes 64-127 of O^T are not used)
            const uint64_t dv0 = sdesc_sw128(smem_u32(sKV), D == 64 ? 0 : C::CB_BYTES, 1024);
            const uint64_t dp0 = sdesc_sw128(smem_u32(sP), 16, 1024);
            const uint64_t dq0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
            constexpr uint32_t CA = C::CB_BYTES / 16 - 6, CQ = C::QCB_BYTES / 16 - 6;
            int blk = 0;               // blocks issued, over all segments
            int fill = 0;              // ring slot of the next K or V chunk
            bool ok = true;
            // the block whose P V is still to come
            bool have = false;
            bool first = false;
            int v_fill = 0;
            auto wait_fill = [&](int f) { return mbar_wait(&full[f % C::NSLOT], (f / C::NSLOT) & 1, s_abort); };
            auto pv = [&]() {   // O^T (+)= V^T P^T of block blk - 1
                const int i = blk - 1;
                if (!mbar_wait(&p_full[i & 1], (i >> 1) & 1, s_abort)) return false;
                tc_fence_after();
                for (int c = 0; c < C::CHUNKS; ++c) {
                    if (!wait_fill(v_fill + c)) return false;
                    tc_fence_after();
                    const int slot = (v_fill + c) % C::NSLOT;
                    mma8_ss_f16<128, 128, 128, 128, 128, 128, 128, 128, 128, 128, 128, 128, 128, 128>(
                        tmem + C::O_COL + c * N, sdesc_adv(dv0, slot * C::SLOT),
                        sdesc_adv(dp0, (i & 1) * C::P_BYTES), IDESC_O, first ? 0u : 1u);
                    tc_commit(&empty[slot]);
                }
                tc_commit(&pv_done[i & 1]);
                have = false;
                return true;
            };
            for (int seg = 0; ok; ++seg) {
                const int buf = seg & 1;
                // let the last block's P V go first if the next segment is not there yet
                if (have && !mbar_test(&q_full[buf], (seg >> 1) & 1)) ok = pv();
                if (!ok || !mbar_wait(&q_full[buf], (seg >> 1) & 1, s_abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int nblk = s_seg[buf].nblk;
                if (nblk == 0) break;
                if (s_seg[buf].none) {
                    mbar_arrive(&q_empty[buf]);
                    continue;
                }
                for (int x = 0; x < nblk && ok; ++x) {
                    // S^T of this block before P V of the one before it, unless K is late
                    if (have && !mbar_test(&full[fill % C::NSLOT], (fill / C::NSLOT) & 1)) ok = pv();
                    for (int c = 0; c < C::CHUNKS && ok; ++c) {
                        ok = wait_fill(fill + c);
                        if (!ok) break;
                        tc_fence_after();
                        const int slot = (fill + c) % C::NSLOT;
                        const uint64_t ad = sdesc_adv(dk0, slot * C::SLOT);
                        const uint64_t bd = sdesc_adv(dq0, buf * C::Q_BYTES + c * C::CCB * C::QCB_BYTES);
                        if constexpr (D == 64)
                            mma4_ss_f16<2, 2, 2, 2, 2, 2>(tmem + (blk & 1) * N, ad, bd, IDESC_S, 0u);
                        else
                            mma8_ss_f16<2, 2, 2, CA, 2, 2, 2, 2, 2, 2, CQ, 2, 2, 2>(
                                tmem + (blk & 1) * N, ad, bd, IDESC_S, c > 0 ? 1u : 0u);
                        tc_commit(&empty[slot]);
                    }
                    if (!ok) break;
                    tc_commit(&s_full[blk & 1]);
                    if (x == nblk - 1) tc_commit(&q_empty[buf]);
                    if (have) ok = pv();
                    if (!ok) break;
                    have = true;
                    first = x == 0;
                    v_fill = fill + C::CHUNKS;
                    fill += 2 * C::CHUNKS;
                    ++blk;
                }
            }
            if (ok && have) ok = pv();
            // Drain: no MMA of this CTA is in flight at teardown.
            tc_commit(bar_fin);
            volatile int no_abort = 0;
            mbar_wait(bar_fin, 0, &no_abort);
        }
        __syncwarp();
    } else {
        // ================= softmax (one thread per key) =================
        const int tid = static_cast<int>(threadIdx.x);
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        const uint32_t t_O = t_lane + C::O_COL;
        const int G = p.G;
        const float sc = p.scale_log2;
        int blk = 0;    // blocks so far, over all segments
        int fill = 0;   // ring slot of the next K chunk
        bool ok = true;
        for (int seg = 0;; ++seg) {
            const int buf = seg & 1;
            // The four warps meet at barriers inside a segment, so all of them
            // take it or none does; a wait that fails inside leaves the results
            // unspecified and ends the walk at the next segment.
            ok = ok && mbar_wait_warp(&q_full[buf], (seg >> 1) & 1, s_abort);
            if (named_barrier_or(1, kSoftmax, !ok)) break;
            Segment s;
            s.nblk = s_seg[buf].nblk;
            if (s.nblk == 0) break;
            s.q_start = s_seg[buf].q_start;
            s.ntok = s_seg[buf].ntok;
            s.hk = s_seg[buf].hk;
            s.off = s_seg[buf].off;
            s.L = s_seg[buf].L;
            s.klo = s_seg[buf].klo;
            s.khi = s_seg[buf].khi;
            s.j0 = s_seg[buf].j0;
            s.out = s_seg[buf].out;
            s.none = s_seg[buf].none;
            mbar_arrive_warp(&q_empty[buf]);
            const int rows = s.ntok * G;
            float l[N];   // this thread's sums
#pragma unroll
            for (int n = 0; n < N; ++n) l[n] = 0.f;
            for (int x = 0; x < (s.none ? 0 : s.nblk); ++x, ++blk, fill += 2 * C::CHUNKS) {
                const int k0 = (s.j0 + x) * kTileRows;
                const int key = k0 + tid;
                ok = ok && mbar_wait_warp(&s_full[blk & 1], (blk >> 1) & 1, s_abort);
                tc_fence_after();
                uint32_t sr[N];
                tmem_ld_cols<N>(t_lane + (blk & 1) * N, sr);
                tmem_ld_wait();
                reg_fence(sr);
                // Blocks where some row does not attend some key: the range's
                // ends, the causal diagonal (queries are the last ntok keys), and
                // a window's start, which moves with the query.
                const bool cut = k0 < s.klo || k0 + kTileRows > s.khi;
                const bool diagonal = p.causal && k0 + kTileRows - 1 > s.off;
                const bool sliding = p.window > 0 &&
                                     (k0 < s.off + s.ntok - p.window ||
                                      (!p.causal && k0 + kTileRows - 1 > s.off + p.window - 1));
                float v[N];
                if (cut || diagonal || sliding) {
                    int pos = s.off, g = 0;   // key position of row n
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        bool ok_n = n < rows && key >= s.klo && key < s.khi;
                        if (p.causal) ok_n = ok_n && key <= pos;
                        if (p.window > 0) ok_n = ok_n && pos - key < p.window && (p.causal || key - pos < p.window);
                        v[n] = ok_n ? __uint_as_float(sr[n]) * sc : -INFINITY;
                        if (++g == G) {
                            g = 0;
                            ++pos;
                        }
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < N; ++n) v[n] = __uint_as_float(sr[n]) * sc;
                }
                bool grows = x == 0;
                if (x > 0) {
#pragma unroll
                    for (int c = 0; c < N / 4; ++c) {
                        const float4 m4 = reinterpret_cast<const float4*>(s_m)[c];
                        const float mm[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            grows |= 4 * c + e < rows && v[4 * c + e] > mm[e] + kRescaleThreshold;
                    }
                }
                if (named_barrier_or(1, kSoftmax, grows)) {
                    // new reference maxima: over the warp's keys, then over the four warps
                    float mine_max = -INFINITY;
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const float wm = key_float(__reduce_max_sync(0xffffffffu, float_key(v[n])));
                        if ((n & 31) == lane) mine_max = wm;
                        if ((n & 31) == 31 || n == N - 1)
                            if (lane < N) s_row[warp * N + (n & ~31) + lane] = mine_max;
                    }
                    named_barrier_sync(1, kSoftmax);
                    if (tid < N) {
                        const float old = x > 0 ? s_m[tid] : kNoMax;
                        const float mt = fmaxf(fmaxf(old, fmaxf(s_row[tid], s_row[N + tid])),
                                               fmaxf(s_row[2 * N + tid], s_row[3 * N + tid]));
                        s_m[tid] = mt;
                        s_fac[tid] = ex2_approx(old - mt);
                    }
                    named_barrier_sync(1, kSoftmax);
                    if (x > 0) {   // sums and O^T columns, once P V of the block before is in
                        ok = ok && mbar_wait_warp(&pv_done[(blk - 1) & 1], ((blk - 1) >> 1) & 1, s_abort);
                        tc_fence_after();
#pragma unroll
                        for (int n = 0; n < N; ++n) l[n] *= s_fac[n];
#pragma unroll
                        for (int h = 0; h < C::HALVES; ++h) {
                            uint32_t o[N];
                            tmem_ld_cols<N>(t_O + h * N, o);
                            tmem_ld_wait();
                            reg_fence(o);
#pragma unroll
                            for (int n = 0; n < N; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * s_fac[n]);
                            tmem_st_cols<N>(t_O + h * N, o);
                        }
                        tmem_st_wait();
                    }
                }
                // P^T: this key's N weights, rounded to the storage type for the
                // product with V; the sum takes them unrounded
                if (blk >= 2) ok = ok && mbar_wait_warp(&pv_done[blk & 1], ((blk >> 1) & 1) ^ 1, s_abort);
                uint8_t* row = sP + (blk & 1) * C::P_BYTES + tid * 128;
#pragma unroll
                for (int c = 0; c < N / 8; ++c) {
                    const float4 ma = reinterpret_cast<const float4*>(s_m)[2 * c];
                    const float4 mb = reinterpret_cast<const float4*>(s_m)[2 * c + 1];
                    const float mm[8] = {ma.x, ma.y, ma.z, ma.w, mb.x, mb.y, mb.z, mb.w};
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int n = 8 * c + 2 * e;
                        const float p0 = ex2_approx(v[n] - mm[2 * e]);
                        const float p1 = ex2_approx(v[n + 1] - mm[2 * e + 1]);
                        l[n] += p0;
                        l[n + 1] += p1;
                        w[e] = pack_h2<kF16>(p0, p1);
                    }
                    *reinterpret_cast<uint4*>(row + ((c ^ (tid & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (cut) {
                    // V rows of keys outside [klo, khi) become zero.  Their slots'
                    // fills before this one must have landed, or the parity would
                    // be theirs: with two slots a tile that takes P V of the block
                    // before.
                    if (C::CHUNKS == 2 && blk > 0)
                        ok = ok && mbar_wait_warp(&pv_done[(blk - 1) & 1], ((blk - 1) >> 1) & 1, s_abort);
                    for (int c = 0; c < C::CHUNKS; ++c) {
                        const int f = fill + C::CHUNKS + c;
                        ok = ok && mbar_wait_warp(&full[f % C::NSLOT], (f / C::NSLOT) & 1, s_abort);
                        if (ok && (key < s.klo || key >= s.khi)) {
                            for (int cb = 0; cb < C::CCB; ++cb) {
                                uint4* vr = reinterpret_cast<uint4*>(sKV + (f % C::NSLOT) * C::SLOT +
                                                                     cb * C::CB_BYTES + tid * 128);
#pragma unroll
                                for (int e = 0; e < 8; ++e) vr[e] = make_uint4(0u, 0u, 0u, 0u);
                            }
                        }
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive_warp(&p_full[blk & 1]);
            }
            // ---- the segment's result: sums over all keys, O = acc / l ----
            if (!s.none) {
                const int last = blk - 1;
                ok = ok && mbar_wait_warp(&pv_done[last & 1], (last >> 1) & 1, s_abort);
                tc_fence_after();
            }
            const int col = warp_sum_scatter<N>(l, lane);
            if (N >= 32 || (lane & 1) == 0) {
                s_row[warp * N + col] = l[0];
                if (N == 64) s_row[warp * N + col + 1] = l[1];
            }
            named_barrier_sync(1, kSoftmax);
            if (tid < N) {
                const float sum = (s_row[tid] + s_row[N + tid]) + (s_row[2 * N + tid] + s_row[3 * N + tid]);
                s_fac[tid] = sum == 0.f ? 0.f : 1.f / sum;
                if (tid < rows) {
                    const float lse2 = sum == 0.f ? -INFINITY : s_m[tid] + log2f(sum);
                    if (s.out >= 0) {
                        p.part_lse[static_cast<size_t>(s.out) * p.slot_rows + tid] = lse2;
                    } else {
                        const int tok = tid / G;
                        p.LSE[static_cast<size_t>(s.hk * G + tid - tok * G) * p.lq.total + s.q_start + tok] =
                            lse2 * kLn2;
                    }
                }
            }
            named_barrier_sync(1, kSoftmax);
#pragma unroll
            for (int h = 0; h < C::HALVES; ++h) {
                uint32_t o[N];
                if (!s.none) {
                    tmem_ld_cols<N>(t_O + h * N, o);
                    tmem_ld_wait();
                    reg_fence(o);
                } else {
#pragma unroll
                    for (int n = 0; n < N; ++n) o[n] = 0u;
                }
                if (D >= 128 || tid < D) {
                    const int dcol = h * 128 + tid;
                    size_t at = s.out >= 0 ? static_cast<size_t>(s.out) * p.slot_rows * D + dcol
                                           : (static_cast<size_t>(s.q_start) * p.lq.H + s.hk * G) * D + dcol;
                    const size_t skip = s.out >= 0 ? 0 : static_cast<size_t>(p.lq.H - G) * D;   // to the next token
                    int g = 0;
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        if (n < rows) {
                            const float x = __uint_as_float(o[n]) * s_fac[n];
                            if (s.out >= 0)
                                p.part_o[at] = x;
                            else
                                static_cast<uint16_t*>(p.O)[at] = static_cast<uint16_t>(pack_h2<kF16>(x, 0.f));
                            at += D;
                            if (++g == G) {
                                g = 0;
                                at += skip;
                            }
                        }
                    }
                }
                __syncwarp();
            }
            // O^T is read: the next segment's first P V, which overwrites it,
            // waits for P^T of these threads.
            tc_fence_before();
        }
    }

    // ---- teardown ----
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) tmem_dealloc(tmem, C::TMEM_COLS);
    if (threadIdx.x == 0 && *s_abort && p.dev_status != nullptr)
        atomicCAS(p.dev_status, 0, static_cast<int>(ATTN_ERR_DEVICE_TIMEOUT));
    if (blockIdx.x == 0) paged_report(p);
}

template <int D, bool kF16, int N>
cudaError_t launch_decode_t(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                            const PagedParams& p, cudaStream_t stream) {
    using C = DecodeCfg<D, N>;
    auto kern = attn_decode_kernel<D, kF16, N>;
    static std::atomic<unsigned long long> smem_ready{0};
    const cudaError_t e = enable_smem_per_device(kern, C::SMEM, smem_ready);
    if (e != cudaSuccess) return e;
    return launch_overlapped(kern, static_cast<unsigned>(p.tiles), C::THREADS, C::SMEM, stream, tq, tk, tv, p);
}

template <int D, bool kF16>
cudaError_t launch_decode_n(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                            const PagedParams& p, cudaStream_t stream) {
    switch (p.slot_rows) {
        case 16: return launch_decode_t<D, kF16, 16>(tq, tk, tv, p, stream);
        case 32: return launch_decode_t<D, kF16, 32>(tq, tk, tv, p, stream);
        case 64: return launch_decode_t<D, kF16, 64>(tq, tk, tv, p, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace gbattn
