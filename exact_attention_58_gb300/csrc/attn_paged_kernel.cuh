// attn_paged_kernel.cuh — attention of chunks of new tokens over a paged
// key/value cache.
//
// The online-softmax forward of attn_fwd_kernel.cuh with three differences:
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
// Two query tiles per CTA share each K/V block (one tile at head dim 256).
#pragma once

#include "attn_fwd_kernel.cuh"
#include "paged.cuh"

namespace gbattn {
namespace {

// First index of request b's tiles when tiles follow the packed offsets:
// floor(cu[b] / T) + b, which leaves every request room for ceil(len / T).
__device__ __forceinline__ int packed_tile_base(const SeqLayout& lq, int b, int tokens) {
    return min(max(lq.cu[b], 0), lq.total) / tokens + b;
}

// Request and tile of packed tile index x (whole warp): the last request whose
// base is <= x, found with 32 probes at a time.
__device__ __forceinline__ void find_packed_tile(const SeqLayout& lq, int B, int tokens, int x,
                                                 int& b, int& local) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = B;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lo + lane * step;
        const bool below = lane * step < n && packed_tile_base(lq, at, tokens) <= x;
        const unsigned hit = __ballot_sync(0xffffffffu, below);
        const int k = hit == 0 ? 0 : 31 - __clz(hit);
        lo += k * step;
        n = min(step, n - k * step);
    }
    b = lo;
    local = x - packed_tile_base(lq, b, tokens);
}

template <int D, bool kF16, int kTiles, bool kFine>
__global__ void __launch_bounds__(FwdCfg<D, false, kF16, false, kTiles>::THREADS, 1)
    attn_paged_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const PagedParams p) {
    using C = FwdCfg<D, false, kF16, false, kTiles>;
    grid_dep_wait();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sQ = smem;                                   // C::TILES tiles
    uint8_t* sKV = smem + C::TILES * C::TILE;             // NSLOT tiles
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (C::TILES + C::NSLOT) * C::TILE);
    uint64_t* bar_q = bars;               // [2] one per query tile
    uint64_t* full = bars + 2;
    constexpr int kPairs = C::NSLOT / 2;
    constexpr bool kBlockRelease = kPairs >= 2;   // see attn_fwd_kernel
    uint64_t* empty = full + C::NSLOT;
    uint64_t* bar_s = empty + C::NSLOT;   // [2]
    uint64_t* bar_p = bar_s + 2;          // [2]
    uint64_t* bar_o = bar_p + 2;          // [2]
    uint64_t* bar_fin = bar_o + 2;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bar_fin + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    // ---- which tokens of which request, which key/value head, which keys ----
    const int G = p.G;
    const int TT = p.tile_tokens;
    const int split = static_cast<int>(blockIdx.x) % p.splits;
    const int hk = static_cast<int>(blockIdx.x) / p.splits % p.Hkv;
    // the last tiles of a causal request see the most keys: they start first
    const int tile = p.tiles - 1 - static_cast<int>(blockIdx.x) / p.splits / p.Hkv;
    int b, local;
    if (p.uniform_tiles > 0) {
        b = tile / p.uniform_tiles;
        local = tile - b * p.uniform_tiles;
    } else {
        find_packed_tile(p.lq, p.B, C::TILES * TT, tile, b, local);
    }
    const SeqSpan sq = seq_span(p.lq, b, nullptr, false);
    const int N = sq.len;
    const int tok0 = local * C::TILES * TT;
    const int L = paged_keys(p, b);
    const int off = L - N;   // query i stands at key position i + off
    const bool live = local >= 0 && tok0 < N;
    const int ntok = live ? min(C::TILES * TT, N - tok0) : 0;
    const int32_t* table = p.page_table + static_cast<size_t>(b) * p.max_pages;

    // Key blocks [jlo(t), jhi(t)) that tile t needs, and the key range
    // [klo, khi) of the whole CTA.
    int jlo0 = 0, jlo1 = 0, jhi0 = 0, jhi1 = 0, klo = 0, khi = 0;
#pragma unroll
    for (int t = 0; t < C::TILES; ++t) {
        const int first = tok0 + t * TT;
        int lo = 0, hi = 0;
        if (live && first < N) key_range(p, first, min(first + TT - 1, N - 1), off, L, lo, hi);
        if (hi > lo) {
            klo = khi > klo ? min(klo, lo) : lo;
            khi = max(khi, hi);
        }
        const int bl = lo / kTileRows, bh = (hi + kTileRows - 1) / kTileRows;
        if (t == 0) { jlo0 = bl; jhi0 = bh; } else { jlo1 = bl; jhi1 = bh; }
    }
    // this CTA's share of the blocks
    const int all_lo = klo / kTileRows, all_hi = (khi + kTileRows - 1) / kTileRows;
    const int share = (all_hi - all_lo + p.splits - 1) / p.splits;
    const int pieces = share > 0 ? (all_hi - all_lo + share - 1) / share : 1;
    if (pieces > 1) {
        const int s0 = all_lo + split * share, s1 = min(all_hi, s0 + share);
        jlo0 = max(jlo0, s0); jhi0 = min(jhi0, s1);
        jlo1 = max(jlo1, s0); jhi1 = min(jhi1, s1);
        if (jhi0 <= jlo0) jlo0 = jhi0 = 0;
        if (jhi1 <= jlo1) jlo1 = jhi1 = 0;
    }
    const bool joined = pieces > 1;
    const int unit = tile * p.Hkv + hk;
    if (threadIdx.x == 0 && split == 0 && p.splits > 1 && p.cluster == 0)
        p.desc[unit] = PieceDesc{sq.start, tok0, ntok, hk, live && joined ? pieces : 0,
                                 unit * p.splits, unit * p.splits + 1, 1};
    if (blockIdx.x == 0) paged_report(p);
    if (!live) return;

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
            const int head = hk * G + g;
            uint2* dst = reinterpret_cast<uint2*>(
                static_cast<uint16_t*>(p.O) + ((static_cast<size_t>(sq.start) + tok0 + ut) * p.lq.H + head) * D);
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
                p.LSE[static_cast<size_t>(head) * p.lq.total + sq.start + tok0 + ut] =
                    sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
        }
        cluster_sync();   // no CTA leaves while another reads its piece
    };
    if (split >= pieces) {   // no blocks left for this CTA
        if (p.cluster > 0 && joined) {
            for (int r = threadIdx.x; r < C::TILES * kTileRows; r += C::THREADS) s_lse[r] = -INFINITY;
            join_cluster();
        }
        return;
    }

    auto jlo = [&](int t) { return t ? jlo1 : jlo0; };
    auto jhi = [&](int t) { return t ? jhi1 : jhi0; };
    auto nkv_t = [&](int t) { return jhi(t) - jlo(t); };
    const int jbeg = (nkv_t(0) > 0) ? jlo0 : jlo1;
    const int jend = max(jhi0, jhi1);
    const int nkv = (nkv_t(0) > 0 || nkv_t(1) > 0) ? jend - jbeg : 0;
    auto edge = [&](int j) { return j * kTileRows < klo || (j + 1) * kTileRows > khi; };

    // ---- set-up ----
    if (threadIdx.x == 0) {
        mbar_init(&bar_q[0], 1);
        mbar_init(&bar_q[1], 1);
        for (int s = 0; s < C::NSLOT; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bar_s[t], 1);
            mbar_init(&bar_p[t], kTileRows);
            mbar_init(&bar_o[t], 1);
        }
        mbar_init(bar_fin, 1);
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
        if (nkv > 0) {
            if (lane == 0) {
                tma_prefetch_desc(&tmQ);
                tma_prefetch_desc(&tmK);
                tma_prefetch_desc(&tmV);
            }
            const int ntiles = (nkv_t(1) > 0) ? 2 : 1;
            if (lane == 0) {
                for (int t = 0; t < ntiles; ++t) {
                    mbar_arrive_expect_tx(&bar_q[t], static_cast<uint32_t>(TT * G) * C::ROWB);
                    for (int cb = 0; cb < C::NCB; ++cb)
                        tma_load_3d(sQ + t * C::TILE + cb * C::CB_BYTES, &tmQ, &bar_q[t],
                                    cb * C::BOXW, hk * G, sq.start + tok0 + t * TT);
                }
            }
            int seq = 0;
            bool ok = true;
            PageBox box = page_box(p, table, jbeg * kTileRows, klo, khi, lane);
            for (int j = jbeg; j < jbeg + nkv && ok; ++j) {
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, box.needed)) *
                                       static_cast<uint32_t>(p.box_rows) * C::ROWB;
                // the next tile's table entries arrive while this tile waits
                PageBox next = box;
                if (j + 1 < jbeg + nkv) next = page_box(p, table, (j + 1) * kTileRows, klo, khi, lane);
                for (int which = 0; which < 2; ++which) {
                    const int slot = seq % C::NSLOT;
                    const uint32_t ph = (seq / C::NSLOT) & 1;
                    bool free_ok;
                    if constexpr (kBlockRelease) {
                        const int bi = j - jbeg;
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
                                    box.row, 0, hk, page_box_checked(p, box));
                    } else if (box.needed) {
                        const int page = page_box_checked(p, box);
                        uint8_t* dst = sKV + slot * C::TILE + lane * p.box_rows * 128;
                        const CUtensorMap* m = which ? &tmV : &tmK;
                        for (int cb = 0; cb < C::NCB; ++cb)
                            tma_load_4d(dst + cb * C::CB_BYTES, m, &full[slot], cb * C::BOXW, box.row,
                                        hk, page);
                    }
                    __syncwarp();
                    ++seq;
                }
                box = next;
            }
            // Drain: every load this warp issued has landed before teardown.
            if (lane == 0) {
                volatile int no_abort = 0;
                for (int t = 0; t < ntiles; ++t) mbar_wait(&bar_q[t], 0, &no_abort);
                for (int s = 0; s < C::NSLOT && s < seq; ++s) {
                    const int uses = (seq - s + C::NSLOT - 1) / C::NSLOT;
                    mbar_wait(&full[s], (uses - 1) & 1, &no_abort);
                }
            }
        }
        __syncwarp();
    } else if (warp == C::MMA_WARP) {
        // ================= MMA issuer =================
        if (lane == 0 && nkv > 0) {
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
            bool q_ready[2] = {false, false};
            int seq = 0;
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
                        ok = mbar_wait(&bar_p[t], (j - 1 - jlo(t)) & 1, s_abort);
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
                            ok = mbar_wait(&bar_q[t], 0, s_abort);
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
                    tc_commit(&empty[(j - jbeg) % kPairs]);
                } else {
                    tc_commit(&empty[kslot]);
                    if (j > jbeg && v_last < 0) tc_commit(&empty[v_slot]);
                }
                v_slot = next_v_slot;
                v_phase = next_v_phase;
                v_ready = false;
            }
            for (int t = 0; t < C::TILES && ok; ++t) {   // tiles whose last block is the CTA's last
                if (nkv_t(t) == 0 || jhi(t) != jbeg + nkv) continue;
                ok = mbar_wait(&bar_p[t], (jhi(t) - 1 - jlo(t)) & 1, s_abort);
                if (ok && !v_ready) {
                    ok = mbar_wait(&full[v_slot], v_phase, s_abort);
                    v_ready = true;
                }
                if (!ok) break;
                tc_fence_after();
                issue_pv(t, v_slot, jhi(t) - 1 > jlo(t));
                tc_commit(&bar_o[t]);
            }
            // Drain: no MMA of this CTA is in flight at teardown.
            tc_commit(bar_fin);
            volatile int no_abort = 0;
            mbar_wait(bar_fin, 0, &no_abort);
        }
        __syncwarp();
    } else {
        // ================= softmax (one thread per row) =================
        const int t = warp >> 2;
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const int tl = r / G;                       // token within the tile
        const int first_tok = tok0 + t * TT;
        const int tok = first_tok + tl;
        const bool row_ok = tl < TT && tok < N;
        const int head = hk * G + (r - tl * G);
        const int pos = tok + off;
        const int first_pos = first_tok + off, last_pos = first_pos + TT - 1;
        const int ntile = nkv_t(t);
        const int W = p.window;
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t t_S = t_lane + 128u * t;
        const uint32_t t_O = t_lane + C::O_COL + D * t;
        float m_ref = -INFINITY;   // reference max, log2 units of scaled scores
        float l = 0.f;
        bool ok = true;
        for (int j = jlo(t); j < jhi(t); ++j) {
            const int k0 = j * kTileRows;
            if (!mbar_wait_warp(&bar_s[t], (j - jlo(t)) & 1, s_abort)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // V rows outside [klo, khi) become zero.  Only after S_j: by then
            // every earlier fill of V_j's slot has been waited for, so that
            // the parity below can only mean this one.
            if (edge(j)) {
                const int vseq = 2 * (j - jbeg) + 1;
                const int slot = vseq % C::NSLOT;
                if (!mbar_wait_warp(&full[slot], (vseq / C::NSLOT) & 1, s_abort)) {
                    ok = false;
                    break;
                }
                if (k0 + r < klo || k0 + r >= khi) {
                    for (int cb = 0; cb < C::NCB; ++cb) {
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
            // columns >= lim and < lo of this row are masked (only on masked tiles)
            int lim = tile_mask ? (p.causal ? min(L, pos + 1) : L) - k0 : kTileRows;
            int lo = 0;
            if (wmask) {
                lo = pos - W + 1 - k0;
                if (!p.causal) lim = min(lim, pos + W - k0);
            }

            // ---- row max ----
            float mx;
            uint32_t sr[4][32];
            {
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(t_S + 32 * c, sr[c]);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 4; ++c) reg_fence(sr[c]);
                if (tile_mask) {
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (c >= lim || c < lo) sr[c >> 5][c & 31] = __float_as_uint(-INFINITY);
                }
                float mp[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) mp[k] = -INFINITY;
#pragma unroll
                for (int c = 0; c < 128; c += 2)
                    mp[(c >> 1) & 7] = max3f(mp[(c >> 1) & 7], __uint_as_float(sr[c >> 5][c & 31]),
                                             __uint_as_float(sr[c >> 5][(c & 31) + 1]));
                mx = max3f(max3f(mp[0], mp[1], mp[2]), max3f(mp[3], mp[4], mp[5]),
                           fmaxf(mp[6], mp[7]));
            }
            const float m_new = fmaxf(m_ref, mx * p.scale_log2);
            const bool want = (m_ref != -INFINITY) && (m_new > m_ref + kRescaleThreshold);
            const bool warp_rescale = __any_sync(0xffffffffu, want);
            float alpha = 1.f;
            if (m_ref == -INFINITY) {
                m_ref = m_new;   // O and l are still zero: adopt without rescaling
            } else if (warp_rescale) {
                alpha = ex2_approx(m_ref - m_new);
                m_ref = m_new;
            }
            const float neg_m = (m_ref == -INFINITY) ? 0.f : -m_ref;

            // ---- P = exp2(s scale log2e - m), rounded to the storage type for
            // the P V product; the row sum adds the unrounded P ----
            const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2);
            const uint64_t nm2 = f2_pack(neg_m, neg_m);
            uint64_t acc2[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) acc2[k] = f2_pack(0.f, 0.f);
#pragma unroll
            for (int c8 = 0; c8 < 8; ++c8) {   // 16 keys, 8 packed words
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
                    pk[e] = pack_h2<kF16>(x0, x1);
                    acc2[e & 3] = f2_add(acc2[e & 3], f2_pack(x0, x1));
                }
                tmem_st8(t_S + 8 * c8, pk);
            }
            float rowsum;
            {
                float a0, a1, a2, a3;
                f2_unpack(f2_add(acc2[0], acc2[1]), a0, a1);
                f2_unpack(f2_add(acc2[2], acc2[3]), a2, a3);
                rowsum = (a0 + a1) + (a2 + a3);
            }
            l = l * alpha + rowsum;
            if (warp_rescale && j > jlo(t)) {   // O row *= alpha (PV of block j-1 is complete)
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
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
        if (ok && ntile > 0) {
            ok = mbar_wait_warp(&bar_o[t], 0, s_abort);
            tc_fence_after();
        }
        if (joined && p.cluster > 0)   // the ring and the queries are free once every product is done
            ok = mbar_wait_warp(bar_fin, 0, s_abort) && ok;
        if (ok) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const size_t piece_row =
                (static_cast<size_t>(unit) * p.splits + split) * p.slot_rows + t * kTileRows + r;
            const size_t out_row = (static_cast<size_t>(sq.start) + tok) * p.lq.H + head;
            uint32_t o[32];
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                __syncwarp();   // rows past the tile's end skip the stores below
                if (ntile > 0) {
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
                        *reinterpret_cast<float4*>(piece_group(t * kTileRows + r, 8 * c + v)) =
                            make_float4(__uint_as_float(o[4 * v]) * inv, __uint_as_float(o[4 * v + 1]) * inv,
                                        __uint_as_float(o[4 * v + 2]) * inv, __uint_as_float(o[4 * v + 3]) * inv);
                } else if (row_ok && joined) {
                    float4* dst = reinterpret_cast<float4*>(p.part_o + piece_row * D + 32 * c);
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        dst[v] = make_float4(__uint_as_float(o[4 * v]) * inv, __uint_as_float(o[4 * v + 1]) * inv,
                                             __uint_as_float(o[4 * v + 2]) * inv,
                                             __uint_as_float(o[4 * v + 3]) * inv);
                } else if (row_ok) {
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.O) + out_row * D + 32 * c);
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
                s_lse[t * kTileRows + r] = lse2;
            } else if (row_ok) {
                if (joined) p.part_lse[piece_row] = lse2;
                else p.LSE[static_cast<size_t>(head) * p.lq.total + sq.start + tok] = lse2 * kLn2;
            }
        }
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

template <int D, bool kF16, int kTiles, bool kFine = false>
cudaError_t launch_paged_t(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const PagedParams& p, cudaStream_t stream) {
    using C = FwdCfg<D, false, kF16, false, kTiles>;
    auto kern = attn_paged_kernel<D, kF16, kTiles, kFine>;
    static std::atomic<unsigned long long> smem_ready{0};
    const cudaError_t e = enable_smem_per_device(kern, C::SMEM, smem_ready);
    if (e != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>(p.tiles) * static_cast<unsigned>(p.Hkv * p.splits);
    return launch_overlapped_cluster(kern, grid, C::THREADS, C::SMEM, p.cluster, stream, tq, tk, tv, p);
}

}  // namespace
}  // namespace gbattn
