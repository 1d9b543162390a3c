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
//   * The row maximum runs over lanes.  A row keeps its reference (its first
//     block's maximum, for fp16 less 7) until a weight exceeds 2^8 (2^15),
//     which one barrier with a vote finds
//     out; only then are maxima reduced and O rescaled.  Row sums stay in
//     each thread and are reduced once at the end.
//   * One persistent CTA per SM.  The key blocks of all requests and heads, in
//     order, are cut into as many equal runs as there are CTAs: a CTA takes a
//     run, whatever the request lengths are.  Tiles (request, head) cut by a run's
//     end are joined by a second launch (paged_join_kernel), at most two
//     pieces per CTA.
//   * Where tiles are few and short, a cluster of up to eight CTAs takes a tile
//     instead and joins its pieces through distributed shared memory: no
//     workspace, no second launch.
//   * The producers run ahead over the ends of tiles: rings of up to 176 KB
//     of K and V tiles are in flight while the other warps finish a tile.
//
// Warps: four (or, with more than 16 rows, eight, which halve the rows) for
// softmax, one key per thread; one that walks the run, tells the others each
// segment (a tile's part of the run) and loads Q and K; one that loads V (a TMA
// instruction costs its warp about 65 cycles, and small pages take many); one
// that issues S^T products and one for P V: an issuing warp stalls on every
// product and commit, and of these two neither waits for the other's operands.
//
// Bound by DRAM in the long run: a 128-key block of K and V (64 KB at d = 128)
// takes an SM 1.41 us, 7.0 TB/s over the GPU, for up to 32 rows (64 rows 1.6 us);
// 48 requests of up to 4200 keys, 32/8 heads, 86 us (514 MB, 5.95 TB/s).  About 10
// us are fixed: launch, the lengths, the first page ids and the first tiles one
// after the other (5 us), the last tile's output, the join (3 us).  One request of
// 997 keys, 12 heads, d = 64, takes 7.8 us (clusters of eight, no join).
//
// kFp8: a cache of e4m3 with a power-of-two scale per page and head.  Products are in
// fp16, which holds every e4m3 exactly, and the scales stay outside of them: K's is
// a factor of the key's scores, V's an exponent that its weights are taken times (so
// that they fall in fp16's range as they count in O), which the sum takes off again.
// bf16 queries become fp16 times a power of two a row.  Eight more warps widen:
// four K, a key per lane, into tensor memory, where the product reads it as its
// first operand; four V into shared memory.  A block then takes an SM 0.89 us at
// d = 128 (5.6 TB/s; 16 bits 1.4) and 0.78 at d = 64, bound by the roles' instructions and
// handovers and by the tensor pipe (small products: 515 and 587 cycles of about
// 1700), and 1.44 at d = 256, by DRAM.  48 requests of up to 4200 keys, 32/8 heads,
// 66 us (258 MB, 3.9 TB/s; 20 of them start, ends of segments and join); 2 of 70001 and
// more, 33 us; 997 keys, 12 heads, d = 64, 8.5 us.
#pragma once

#include "attn_fwd_kernel.cuh"
#include "fp8.cuh"
#include "paged.cuh"

namespace gbattn {
namespace {

// The kernel's waits.  Inlined polling loops are a third of its code.  Over a cache
// of e4m3 four roles' loops run on every SM sub-partition and starve in its
// instruction buffer, so there (kCall) polling is a function of its own (48
// requests of up to 4200 keys 95.6 -> 71.5 us), and a poll may sleep for up to a
// microsecond in hardware instead of taking issue slots (70.3 -> 66.1).
__device__ __forceinline__ bool try_wait_hint(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(1000)
        : "memory");
    return ok != 0;
}
__device__ __noinline__ bool poll_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (__all_sync(0xffffffffu, try_wait_hint(bar, parity))) return true;
    const unsigned long long t0 = globaltimer();
    for (;;) {
        if (__all_sync(0xffffffffu, try_wait_hint(bar, parity))) return true;
        int give_up = (*abort != 0) || (elapsed_ns(t0) > static_cast<long long>(kWaitLimitNs));
        give_up = __shfl_sync(0xffffffffu, give_up, 0);
        if (give_up) {
            *abort = 1;
            return false;
        }
    }
}
__device__ __noinline__ bool poll_one(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (try_wait_hint(bar, parity)) return true;
    const unsigned long long t0 = globaltimer();
    for (;;) {
        if (try_wait_hint(bar, parity)) return true;
        if (*abort) return false;
        if (elapsed_ns(t0) > static_cast<long long>(kWaitLimitNs)) {
            *abort = 1;
            return false;
        }
    }
}
template <bool kCall>
__device__ __forceinline__ bool wait_warp_soon(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if constexpr (!kCall) return mbar_wait_warp_soon(bar, parity, abort);
    else return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || poll_warp(bar, parity, abort);
}
template <bool kCall>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if constexpr (!kCall) return mbar_wait_warp(bar, parity, abort);
    else return poll_warp(bar, parity, abort);
}
template <bool kCall>
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if constexpr (!kCall) return mbar_wait(bar, parity, abort);
    else return poll_one(bar, parity, abort);
}

template <int D, int N, bool kFp8>
struct DecodeCfg {
    static constexpr int CHUNKS = D == 256 ? 2 : 1;          // ring slots of one tile
    static constexpr int CW = D / CHUNKS;                    // head-dim columns of a slot
    static constexpr int CCB = CW / 64;                      // 128-byte column blocks of a 16-bit chunk
    static constexpr int CB_BYTES = kTileRows * 128;
    static constexpr int CHUNK = CCB * CB_BYTES;             // a chunk's bytes in 16 bits
    static constexpr int SLOT = kFp8 ? CHUNK / 2 : CHUNK;    // and as loaded
    static constexpr int QCB_BYTES = N * 128;                // Q: column blocks of N rows
    static constexpr int Q_BYTES = (D / 64) * QCB_BYTES;
    static constexpr int P_BYTES = kTileRows * 128;          // P^T: 128 keys of up to 64 rows
    static constexpr int MISC0 = 2944;                       // barriers, segments, row values
    static constexpr int MISC = MISC0 + (kFp8 ? 3328 : 0);   // barriers, scales
    static constexpr int ROOM = 232448 - MISC - 2 * Q_BYTES - 2 * P_BYTES;
    // (fp8) Chunks of V widened to fp16: three where that leaves five loads, so that
    // the last blocks' are there when their weights are.
    static constexpr int NW = ROOM - 3 * CHUNK >= 5 * SLOT ? 3 : 2;
    static constexpr int WIDE = kFp8 ? NW * CHUNK : 0;
    static constexpr int AVAIL = ROOM - WIDE;
    static constexpr int NSLOT = AVAIL / SLOT < 11 ? AVAIL / SLOT : 11;
    static constexpr int NK = (NSLOT + 1) / 2, NV = NSLOT / 2;   // K and V rings
    static constexpr int SMEM = 2 * Q_BYTES + 2 * P_BYTES + NSLOT * SLOT + WIDE + MISC;
    static constexpr int HALVES = D == 256 ? 2 : 1;          // 128-lane halves of O^T
    static constexpr uint32_t O_COL = 2 * N;                 // S^T in [0, 2N), two buffers
    // Softmax warpgroups: with 32 or 64 rows (fp8: always) two of them share the columns.
    static constexpr int GROUPS = N > 16 || kFp8 ? 2 : 1;
    static constexpr int NC = N / GROUPS;                    // columns of a thread
    static constexpr uint32_t K_COL = O_COL + HALVES * N;    // (fp8) two chunks of K widened to fp16
    static constexpr uint32_t USED_COLS = K_COL + CW;
    static constexpr uint32_t TMEM_COLS = !kFp8 ? 4 * N : USED_COLS <= 128 ? 128 : USED_COLS <= 256 ? 256 : 512;
    static constexpr int K_WARP = 4 * GROUPS, V_WARP = K_WARP + 1, S_WARP = K_WARP + 2, PV_WARP = K_WARP + 3;
    static constexpr int K_CONV = 4 * GROUPS + 4, V_CONV = K_CONV + 4;   // (fp8) four warps each that widen
    static constexpr int THREADS = 32 * (4 * GROUPS + (kFp8 ? 12 : 4));
    static_assert(N * D * 4 <= (kFp8 ? WIDE : NK * SLOT), "a cluster's piece fits the widened V, or the K ring");
    static_assert(kFp8 ? NV >= 1 : NV >= 2 && NV >= CHUNKS, "two slots a ring, and a tile");
    static_assert(USED_COLS <= 512, "tensor memory");
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
    r.n = p.few > 0 && sq.len > p.few ? 0 : sq.len;
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

// Sums of v[0..N) over the warp, N = 8, 16 or 32, scattered: after it, a lane holds
// in v[0] the sum of the column returned (32 / N neighbouring lanes each).
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
    static_assert(N == 8 || N == 16 || N == 32, "columns of a thread");
    if constexpr (N == 8) tmem_ld8(t, r);
    else if constexpr (N == 16) tmem_ld16(t, r);
    else tmem_ld32(t, r);
}

// A CTA's run [u0, u1) of the units of request 0, 1, ... one after the other.
struct Run {
    long long all, parts;   // units in all; CTAs that have some
    long long u0, u1;
    int b;                  // request that holds u0
    long long b_unit;       // its first unit
};

// Cuts all units into equal runs, one per CTA of the grid, as far as they go
// round (no run in between is empty: the pieces of a tile are in consecutive
// CTAs): boundary i is at floor(all i / parts).  Code that runs once costs its
// fetching, and a wide division is long: the ordinary case does without.
__device__ __forceinline__ void cut_run(Run& r) {
    const uint32_t i = blockIdx.x;
    r.parts = min(r.all, static_cast<long long>(gridDim.x));
    if (i >= r.parts) return;
    if (r.all < (1ll << 24)) {   // times gridDim.x < 2^8: in 32 bits
        const uint32_t n = static_cast<uint32_t>(r.parts), all = static_cast<uint32_t>(r.all);
        r.u0 = all * i / n;
        r.u1 = all * (i + 1) / n;
    } else {
        r.u0 = r.all * i / r.parts;
        r.u1 = r.all * (i + 1) / r.parts;
    }
}

// Walks a CTA's run, segment by segment, with the whole warp: body(request
// index, request, head, first block, blocks, first unit) returns false to stop.
// Returns whether the walk came to its end.
template <typename Body>
__device__ __forceinline__ bool walk_run(const PagedParams& p, const Run& run, int lane, Body&& body) {
    if (run.u0 >= run.u1) return true;
    int b = run.b;
    long long u = run.u0;
    const long long end = run.u1;
    // lane x holds request win + x
    auto load = [&](int at) {
        return at + lane < p.B ? request_of(p, at + lane) : Request{0, 0, 0, 0, 0, 0, 0};
    };
    int win = b;
    Request held = load(win);
    int in_req = static_cast<int>(u - run.b_unit);   // unit within the request: head * units + block
    while (u < end) {
        Request r;
        const int x = b - win;
        r.start = __shfl_sync(0xffffffffu, held.start, x);
        r.n = __shfl_sync(0xffffffffu, held.n, x);
        r.L = __shfl_sync(0xffffffffu, held.L, x);
        r.klo = __shfl_sync(0xffffffffu, held.klo, x);
        r.khi = __shfl_sync(0xffffffffu, held.khi, x);
        r.j0 = __shfl_sync(0xffffffffu, held.j0, x);
        r.units = __shfl_sync(0xffffffffu, held.units, x);
        const int hk = in_req / r.units, blk = in_req - hk * r.units;
        const int nblk = static_cast<int>(min(static_cast<long long>(r.units - blk), end - u));
        if (!body(b, r, hk, blk, nblk, u)) return false;
        u += nblk;
        in_req += nblk;
        if (in_req == r.units * p.Hkv && u < end) {   // next request with queries
            in_req = 0;
            for (++b;;) {
                if (b >= win + 32) {
                    win = b;
                    held = load(win);
                }
                const unsigned has = __ballot_sync(0xffffffffu, win + lane >= b && held.units > 0);
                if (has != 0) {
                    b = win + __ffs(has) - 1;
                    break;
                }
                b = win + 32;
                if (b >= p.B) return true;   // lengths changed under the kernel
            }
        }
    }
    return true;
}

template <int D, bool kF16, int N, bool kFp8>
__global__ void __launch_bounds__(DecodeCfg<D, N, kFp8>::THREADS, 1)
    attn_decode_kernel(const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const PagedParams p) {
    using C = DecodeCfg<D, N, kFp8>;
    constexpr int NC = C::NC;
    constexpr int kSoftmax = 128 * C::GROUPS;   // threads of the softmax warps
    constexpr bool kMmaF16 = kF16 || kFp8;      // type of the products' operands
    constexpr bool kTurnQ = kFp8 && !kF16;      // bf16 queries become fp16 times a power of two a row
    constexpr uint32_t FMT = fmt16<kMmaF16>();
    constexpr uint32_t IDESC_S = idesc_f32acc(128, N, FMT, false, false);
    constexpr uint32_t IDESC_O = idesc_f32acc(128, N, FMT, true, true);
    extern __shared__ __align__(1024) uint8_t smem[];
    if ((smem_u32(smem) & 1023u) != 0) {   // the swizzled tiles need 1024-byte alignment
        grid_dep_wait();
        if (threadIdx.x == 0) {
            if (p.cluster == 0) p.desc[blockIdx.x].n = 0;
            if (p.dev_status != nullptr) atomicCAS(p.dev_status, 0, static_cast<int>(ATTN_ERR_CUDA));
        }
        return;
    }
    uint8_t* sK = smem;                          // NK slots
    uint8_t* sV = sK + C::NK * C::SLOT;          // NV slots
    uint8_t* sW = sV + C::NV * C::SLOT;          // (fp8) NW chunks of V in fp16
    uint8_t* sP = sW + C::WIDE;                  // two buffers
    uint8_t* sQ = sP + 2 * C::P_BYTES;           // two buffers
    uint64_t* bars = reinterpret_cast<uint64_t*>(sQ + 2 * C::Q_BYTES);
    uint64_t* q_full = bars;            // [2] a segment and its queries are there
    uint64_t* q_empty = bars + 2;       // [2] both readers are done with them
    uint64_t* s_full = bars + 4;        // [2] S^T of a block
    uint64_t* p_full = bars + 6;        // [2] P^T of a block (V's edge cleared)
    uint64_t* pv_done = bars + 8;       // [2] O^T += V^T P^T of a block
    uint64_t* bar_fin = bars + 10;      // [2] every MMA of an issuing warp
    uint64_t* k_full = bars + 12;       // [NK]
    uint64_t* k_empty = bars + 18;
    uint64_t* v_full = bars + 24;       // [NV]
    uint64_t* v_empty = bars + 30;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 36);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    volatile int* s_kind = reinterpret_cast<volatile int*>(bars + 37);   // [2] of a block's P V
    volatile Segment* s_seg = reinterpret_cast<volatile Segment*>(bars + 38);   // [2]
    float* s_row = reinterpret_cast<float*>(bars + 50);   // [4][N]: maxima, then sums, of each warp
    float* s_negm = s_row + 4 * N;    // [N] minus the reference maxima, log2 units
    float* s_fac = s_negm + N;        // [N] factors: of a rescale, then 1 / l
    int* s_lo = reinterpret_cast<int*>(s_fac + N);         // [N] first key that a row attends,
    uint32_t* s_num = reinterpret_cast<uint32_t*>(s_lo + N);   // [N] and how many from there on
    float* s_lse = reinterpret_cast<float*>(s_num + N);        // [N] of a cluster's piece
    long long* s_scan = reinterpret_cast<long long*>(s_lse + N);   // [22] set-up only
    static_assert(C::NK <= 6 && C::NV <= 6, "ring barriers");
    static_assert(2 * sizeof(Segment) <= 12 * 8, "segments fit their place");
    static_assert(50 * 8 + 9 * N * 4 + 22 * 8 <= C::MISC0, "row values fit their place");
    // (fp8)
    uint64_t* bars8 = bars + C::MISC0 / 8;
    uint64_t* q_turned = bars8;         // [2] the queries are fp16
    uint64_t* kt_full = bars8 + 2;      // [2] a chunk of K in tensor memory
    uint64_t* kt_empty = bars8 + 4;
    uint64_t* vt_full = bars8 + 6;      // [NW] a chunk of V in fp16
    uint64_t* vt_empty = bars8 + 9;
    uint64_t* sc_full = bars8 + 12;     // [16] the scales of a block
    volatile int* s_vrows = reinterpret_cast<volatile int*>(bars8 + 28);   // [NV] rows of a V slot with keys: lo | hi << 8
    float* s_qs = reinterpret_cast<float*>(bars8 + 32);           // [4][64] a segment's rows' powers of two
    volatile float* s_scale = s_qs + 4 * 64;                      // [16 blocks][16 boxes][2] K's factor, V's exponent
    static_assert(32 * 8 + 4 * 64 * 4 + 16 * 16 * 2 * 4 <= C::MISC - C::MISC0 || !kFp8, "scales fit their place");
    constexpr int kFirst = 1, kStop = 2;   // s_kind: O^T starts anew; no more blocks

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int cta = static_cast<int>(blockIdx.x);

    // ---- this CTA's run [u0, u1) of the key blocks of all requests and heads ----
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 1 + kSoftmax + (kFp8 ? 128 : 0));
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], kSoftmax);
            mbar_init(&pv_done[s], 1);
            mbar_init(&bar_fin[s], 1);
        }
        for (int s = 0; s < C::NK; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], kFp8 ? 128 : 1);
        }
        for (int s = 0; s < C::NV; ++s) {
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], kFp8 ? 128 : 1);
        }
        for (int s = 0; s < 2 && kFp8; ++s) {
            mbar_init(&q_turned[s], 128);
            mbar_init(&kt_full[s], 128);
            mbar_init(&kt_empty[s], 1);
        }
        for (int s = 0; s < C::NW && kFp8; ++s) {
            mbar_init(&vt_full[s], 128);
            mbar_init(&vt_empty[s], 1);
        }
        for (int s = 0; s < 16 && kFp8; ++s) mbar_init(&sc_full[s], 1);
        *s_abort = 0;
        fence_mbar_init();
    }
    if (warp == C::S_WARP) {
        tmem_alloc(s_tmem, C::TMEM_COLS);
        tmem_relinquish();
    }
    // Up to here nothing in global memory was touched: the kernel before may
    // still have been running.
    grid_dep_wait();
    grid_dep_launch_dependents();   // the join: it waits for this grid itself
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
    Run run{0, 1, 0, 0, 0, 0};
    // A cluster's producers find their share by themselves, and so do those of up
    // to 32 requests their run, one request per lane (a microsecond less).
    const bool alone = p.cluster > 0 || p.B <= 32;
    if (!alone) {
        long long* s_at = s_scan + 20;   // request that holds unit u0, and where it starts
        long long mine = 0, excl = 0;
        for (int b0 = 0; b0 < p.B; b0 += C::THREADS) {
            const int b = b0 + static_cast<int>(threadIdx.x);
            mine = b < p.B ? static_cast<long long>(request_of(p, b).units) * p.Hkv : 0;
            long long total;
            excl = block_scan(mine, total);
            run.all += total;
        }
        cut_run(run);
        if (p.B <= C::THREADS) {   // one round: the sums of above
            if (excl <= run.u0 && run.u0 < excl + mine) {
                s_at[0] = threadIdx.x;
                s_at[1] = excl;
            }
        } else {
            long long done = 0;
            for (int b0 = 0; b0 < p.B && done <= run.u0; b0 += C::THREADS) {
                const int b = b0 + static_cast<int>(threadIdx.x);
                mine = b < p.B ? static_cast<long long>(request_of(p, b).units) * p.Hkv : 0;
                long long total;
                excl = done + block_scan(mine, total);
                if (excl <= run.u0 && run.u0 < excl + mine) {
                    s_at[0] = b;
                    s_at[1] = excl;
                }
                done += total;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    if (!alone && run.u0 < run.u1) {
        run.b = static_cast<int>(s_scan[20]);
        run.b_unit = s_scan[21];
    }

    // Calls body for every segment of the CTA: those of its run, or its even
    // share of the cluster's tile.
    auto each_segment = [&](auto&& body) {
        if (p.cluster == 0) return walk_run(p, run, lane, body);
        const int rank = cta % p.cluster, tile = cta / p.cluster;
        const int b = tile / p.Hkv;
        const Request r = request_of(p, b);
        const int share = (r.units + p.cluster - 1) / p.cluster;
        const int first = rank * share;
        return first >= r.units || body(b, r, tile - b * p.Hkv, first, min(share, r.units - first), 0ll);
    };

    // One tile's chunk into a ring slot (whole warp).
    auto load_chunk = [&](const CUtensorMap* map, uint8_t* slot, uint64_t* bar, const PageBox& box,
                          uint32_t bytes, int c0, int hk) {
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
        __syncwarp();
        if (box.needed) {
            const int page = page_box_checked(p, box);
            uint8_t* dst = slot + lane * p.box_rows * 128;
#pragma unroll
            for (int cb = 0; cb < C::CCB; ++cb)
                tma_load_4d(dst + cb * C::CB_BYTES, map, bar, c0 + cb * 64, box.row, hk, page);
        }
        __syncwarp();
    };
    // The K (or V) tiles of one segment through their ring.
    auto load_tiles = [&](const CUtensorMap* map, uint8_t* ring, uint64_t* full, uint64_t* empty,
                          int slots, int& fills, PageBox box, int b, const Request& r, int hk, int blk,
                          int nblk) {
        if (r.khi <= r.klo) return true;
        const int32_t* table = p.page_table + static_cast<size_t>(b) * p.max_pages;
        const int jbeg = r.j0 + blk;
        for (int j = jbeg; j < jbeg + nblk; ++j) {
            const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, box.needed)) *
                                   static_cast<uint32_t>(p.box_rows) * (2 * C::CW);
            PageBox next = box;
            if (j + 1 < jbeg + nblk) next = page_box(p, table, (j + 1) * kTileRows, r.klo, r.khi, lane);
            for (int c = 0; c < C::CHUNKS; ++c, ++fills) {
                const int slot = fills % slots;
                if (!wait_warp_soon<kFp8>(&empty[slot], ((fills / slots) & 1) ^ 1, s_abort)) return false;
                load_chunk(map, ring + slot * C::SLOT, &full[slot], box, bytes, c * C::CW, hk);
            }
            box = next;
        }
        return true;
    };
    // The same for 8-bit tiles.  A lane per box finds the pages of 32 boxes, two tiles
    // and more, at a time: what is done for each tile stays short (tiles come
    // twice as fast as of 16 bits, and a warp that runs now and then finds its code
    // gone from the instruction buffer each time).  K's producer (keys) also gets
    // the scales of the boxes' pages, K's with the softmax scale as a factor of
    // the scores, V's as an exponent of the weights; it passes on a tile's behind the
    // next tile's loads.  The 16 tiles' worth of room is more than K runs ahead of
    // the softmax (by the ring, two chunks in tensor memory and two of S^T).
    const int box_log = 31 - __clz(p.box_rows);
    const int per_log = 7 - box_log;   // boxes of a tile
    int scaled = 0;                    // tiles whose scales have been passed on
    auto boxes8 = [&](int b, const Request& r, int j, int jend) {   // of tiles j, j + 1, ...
        PageBox x{false, 0, 0};
        const int key = j * kTileRows + lane * p.box_rows;
        if (key < min(r.khi, jend * kTileRows) && key + p.box_rows > r.klo) {
            x.needed = true;
            const int col = static_cast<int>(__umul64hi(static_cast<unsigned long long>(key) << 2, p.page_magic));
            x.row = key - col * p.page_size;
            x.page = p.page_table[static_cast<size_t>(b) * p.max_pages + col];
        }
        return x;
    };
    auto load_tiles8 = [&](const CUtensorMap* map, uint8_t* ring, uint64_t* full, uint64_t* empty, int slots,
                           int& fills, PageBox next, int b, const Request& r, int hk, int blk, int nblk, bool keys) {
        if (r.khi <= r.klo) return true;
        const int jend = r.j0 + blk + nblk, tiles = 32 >> per_log;
        const int mine = lane >> per_log, box = lane & ((1 << per_log) - 1);
        uint32_t kb = 0, vb = 0;
        auto ask = [&](const PageBox& x) {
            kb = vb = 127u << 23;   // (of a box that is not loaded: any)
            if (keys && x.needed && static_cast<unsigned>(x.page) < static_cast<unsigned>(p.num_pages)) {
                const size_t at = static_cast<size_t>(x.page) * p.Hkv + hk;
                kb = __float_as_uint(p.k_scale[at]);
                vb = __float_as_uint(p.v_scale[at]);
            }
        };
        ask(next);
#pragma unroll 1
        for (int j0 = r.j0 + blk; j0 < jend; j0 += tiles) {
            const PageBox x = next;
            const int page = x.needed ? page_box_checked(p, x) : 0;
            const unsigned needed = __ballot_sync(0xffffffffu, x.needed);
            const float kf = score_factor(exp2_int(scale_exponent(kb)) * p.scale_log2);
            const float ve = static_cast<float>(scale_exponent(vb));
            if ((bad_scale(kb) || bad_scale(vb)) && p.dev_status != nullptr)
                atomicCAS(p.dev_status, 0, static_cast<int>(ATTN_ERR_INVALID_ARG));
            next = boxes8(b, r, j0 + tiles, jend);
            const int n = min(tiles, jend - j0);
            auto pass_on = [&](int t) {
                if (mine == t) {
                    volatile float* at = s_scale + ((scaled & 15) * 16 + box) * 2;
                    at[0] = kf;
                    at[1] = ve;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_full[scaled & 15]);
                ++scaled;
            };
#pragma unroll 1
            for (int t = 0; t < n; ++t) {
                const unsigned mask = (1u << (1 << per_log)) - 1u;   // of a tile's boxes
                const uint32_t bytes = static_cast<uint32_t>(__popc(needed >> (t << per_log) & mask)) << box_log;
#pragma unroll 1
                for (int c = 0; c < C::CHUNKS; ++c, ++fills) {
                    const int slot = fills % slots;
                    if (!wait_warp_soon<kFp8>(&empty[slot], ((fills / slots) & 1) ^ 1, s_abort)) return false;
                    if (lane == 0) {
                        if (!keys) {
                            const int k0 = (j0 + t) * kTileRows;
                            s_vrows[slot] = max(0, r.klo - k0) | min(kTileRows, r.khi - k0) << 8;
                        }
                        mbar_arrive_expect_tx(&full[slot], bytes * C::CW);
                    }
                    __syncwarp();
                    if (mine == t && x.needed)
                        tma_load_4d(ring + slot * C::SLOT + (box << box_log) * C::CW, map, &full[slot], c * C::CW, x.row,
                                    hk, page);
                    __syncwarp();
                }
                if (keys && t > 0) pass_on(t - 1);
            }
            if (keys) pass_on(n - 1);
            ask(next);
        }
        return true;
    };
    // The boxes of a segment's first tile: asked for before anything else.
    auto first_box = [&](int b, const Request& r, int blk, int nblk) {
        if constexpr (kFp8) return boxes8(b, r, r.j0 + blk, r.j0 + blk + nblk);
        else return page_box(p, p.page_table + static_cast<size_t>(b) * p.max_pages, (r.j0 + blk) * kTileRows, r.klo,
                        r.khi, lane);
    };
    // Every load of a ring has landed.
    auto drain = [&](uint64_t* full, int slots, int fills) {
        volatile int no_abort = 0;
        for (int s = 0; s < slots && s < fills; ++s) {
            const int uses = (fills - s + slots - 1) / slots;
            wait_one<kFp8>(&full[s], (uses - 1) & 1, &no_abort);
        }
    };

    if (p.cluster == 0 && alone && (warp == C::K_WARP || warp == C::V_WARP)) {
        const long long mine = lane < p.B ? static_cast<long long>(request_of(p, lane).units) * p.Hkv : 0;
        long long incl = mine;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        run.all = __shfl_sync(0xffffffffu, incl, 31);
        cut_run(run);
        const unsigned past = __ballot_sync(0xffffffffu, incl > run.u0);
        run.b = past != 0 ? __ffs(past) - 1 : 0;
        run.b_unit = __shfl_sync(0xffffffffu, incl - mine, run.b);
    }

    if (warp == C::K_WARP) {
        // ================= producer of segments, Q and K =================
        if (lane == 0) {
            if (p.cluster == 0) p.desc[cta].n = 0;
            tma_prefetch_desc(&tmQ);
            tma_prefetch_desc(&tmK);
        }
        int fills = 0, seg = 0;
        bool ok = each_segment([&](int b, const Request& r, int hk, int blk, int nblk,
                                                            long long u) {
            const int buf = seg & 1;
            const PageBox box = first_box(b, r, blk, nblk);
            if (seg >= 2 && !wait_warp_soon<kFp8>(&q_empty[buf], ((seg >> 1) & 1) ^ 1, s_abort)) return false;
            if (lane == 0) {
                const bool whole = nblk == r.units, none = r.khi <= r.klo;
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
                s.out = whole ? -1 : (p.cluster > 0 ? 0 : 2 * cta + (blk == 0 ? 1 : 0));
                s.none = none;
                if (p.cluster == 0 && !whole && blk == 0) {   // this CTA has the tile's first piece
                    const long long end = u + r.units;
                    // CTA that ends it: the first whose boundary is at or past `end`
                    const long long last = run.all < (1ll << 24)
                                               ? (static_cast<uint32_t>(end) * static_cast<uint32_t>(run.parts) +
                                                  static_cast<uint32_t>(run.all) - 1) /
                                                         static_cast<uint32_t>(run.all) - 1
                                               : (end * run.parts + run.all - 1) / run.all - 1;
                    p.desc[cta] = PieceDesc{r.start, 0, r.n, hk, static_cast<int>(last) - cta + 1,
                                            2 * cta + 1, 2 * cta + 2, 2};
                }
                if (none) {
                    mbar_arrive(&q_full[buf]);
                } else {
                    mbar_arrive_expect_tx(&q_full[buf], static_cast<uint32_t>(p.tile_tokens * p.G) * (2 * D));
                    for (int cb = 0; cb < D / 64; ++cb)
                        tma_load_3d(sQ + buf * C::Q_BYTES + cb * C::QCB_BYTES, &tmQ, &q_full[buf], cb * 64,
                                    hk * p.G, r.start);
                }
            }
            __syncwarp();
            ++seg;
            if constexpr (kFp8)
                return load_tiles8(&tmK, sK, k_full, k_empty, C::NK, fills, box, b, r, hk, blk, nblk, true);
            else
                return load_tiles(&tmK, sK, k_full, k_empty, C::NK, fills, box, b, r, hk, blk, nblk);
        });
        // no more segments
        bool told = false;
        if (ok && (seg < 2 || wait_warp<kFp8>(&q_empty[seg & 1], ((seg >> 1) & 1) ^ 1, s_abort))) {
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
            for (int s = max(0, seg - (told ? 1 : 2)); s < seg; ++s) wait_one<kFp8>(&q_full[s & 1], (s >> 1) & 1, &no_abort);
            drain(k_full, C::NK, fills);
        }
        __syncwarp();
    } else if (warp == C::V_WARP) {
        // ================= producer of V =================
        if (lane == 0) tma_prefetch_desc(&tmV);
        int fills = 0;
        const bool ok = each_segment([&](int b, const Request& r, int hk, int blk, int nblk, long long) {
            if constexpr (kFp8)
                return load_tiles8(&tmV, sV, v_full, v_empty, C::NV, fills, first_box(b, r, blk, nblk), b, r, hk, blk, nblk,
                                   false);
            else
                return load_tiles(&tmV, sV, v_full, v_empty, C::NV, fills, first_box(b, r, blk, nblk), b, r, hk, blk, nblk);
        });
        if (lane == 0) drain(v_full, C::NV, fills);
        __syncwarp();
        if (kFp8 && ok && wait_warp<kFp8>(&v_empty[fills % C::NV], ((fills / C::NV) & 1) ^ 1, s_abort)) {
            if (lane == 0) {   // no more tiles
                s_vrows[fills % C::NV] = -1;
                mbar_arrive(&v_full[fills % C::NV]);
            }
            __syncwarp();
        }
    } else if (warp == C::S_WARP) {
        // ================= S^T = K Q^T =================
        if (lane == 0) {
            const uint64_t dk0 = sdesc_sw128(smem_u32(sK), 16, 1024);
            const uint64_t dq0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
            constexpr uint32_t CA = C::CB_BYTES / 16 - 6, CQ = C::QCB_BYTES / 16 - 6;
            int blk = 0, fill = 0;   // blocks and ring chunks so far, over all segments
            bool ok = true;
            for (int seg = 0; ok; ++seg) {
                const int buf = seg & 1;
                if (!wait_one<kFp8>(kTurnQ ? &q_turned[buf] : &q_full[buf], (seg >> 1) & 1, s_abort)) break;
                tc_fence_after();
                const int nblk = s_seg[buf].nblk;
                if (nblk == 0) break;
                if (s_seg[buf].none) {
                    mbar_arrive(&q_empty[buf]);
                    continue;
                }
                for (int x = 0; x < nblk && ok; ++x, ++blk) {
                    // S^T's buffer is read once P^T of two blocks before is there
                    ok = blk < 2 || wait_one<kFp8>(&p_full[blk & 1], ((blk >> 1) & 1) ^ 1, s_abort);
                    for (int c = 0; c < C::CHUNKS && ok; ++c, ++fill) {
                        if constexpr (kFp8) {
                            ok = wait_one<kFp8>(&kt_full[fill & 1], (fill >> 1) & 1, s_abort);
                            if (!ok) break;
                            tc_fence_after();
                            for (int cb = 0; cb < C::CCB; ++cb)
                                mma_run_ts_f16<4, 8, 2>(
                                    tmem + (blk & 1) * N, tmem + C::K_COL + (fill & 1) * (C::CW / 2) + 32 * cb,
                                    sdesc_adv(dq0, buf * C::Q_BYTES + (c * C::CCB + cb) * C::QCB_BYTES), IDESC_S,
                                    c + cb > 0 ? 1u : 0u);
                            if (c == C::CHUNKS - 1) tc_commit(&s_full[blk & 1]);
                            tc_commit(&kt_empty[fill & 1]);
                            continue;
                        }
                        const int slot = fill % C::NK;
                        ok = wait_one<kFp8>(&k_full[slot], (fill / C::NK) & 1, s_abort);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t ad = sdesc_adv(dk0, slot * C::SLOT);
                        const uint64_t bd = sdesc_adv(dq0, buf * C::Q_BYTES + c * C::CCB * C::QCB_BYTES);
                        if constexpr (D == 64)
                            mma4_ss_f16<2, 2, 2, 2, 2, 2>(tmem + (blk & 1) * N, ad, bd, IDESC_S, 0u);
                        else
                            mma8_ss_f16<2, 2, 2, CA, 2, 2, 2, 2, 2, 2, CQ, 2, 2, 2>(
                                tmem + (blk & 1) * N, ad, bd, IDESC_S, c > 0 ? 1u : 0u);
                        if (c == C::CHUNKS - 1) tc_commit(&s_full[blk & 1]);
                        tc_commit(&k_empty[slot]);
                    }
                    if (ok && x == nblk - 1) tc_commit(&q_empty[buf]);
                }
            }
            // Drain: no MMA of this warp is in flight at teardown.
            tc_commit(&bar_fin[0]);
            volatile int no_abort = 0;
            wait_one<kFp8>(&bar_fin[0], 0, &no_abort);
        }
        __syncwarp();
    } else if (warp == C::PV_WARP) {
        // ================= O^T (+)= V^T P^T =================
        if (lane == 0) {
            // V^T: 64 head-dim columns, the next 64 a column block on (for
            // d = 64 the same again: lanes 64-127 of O^T are not used)
            const uint64_t dv0 = sdesc_sw128(smem_u32(kFp8 ? sW : sV), D == 64 ? 0 : C::CB_BYTES, 1024);
            constexpr int NVS = kFp8 ? C::NW : C::NV;
            uint64_t* const full = kFp8 ? vt_full : v_full;
            uint64_t* const empty = kFp8 ? vt_empty : v_empty;
            const uint64_t dp0 = sdesc_sw128(smem_u32(sP), 16, 1024);
            int fill = 0;
            bool ok = true;
            for (int blk = 0; ok; ++blk) {
                if (!wait_one<kFp8>(&p_full[blk & 1], (blk >> 1) & 1, s_abort)) break;
                tc_fence_after();
                const int kind = s_kind[blk & 1];
                if (kind == kStop) break;
                for (int c = 0; c < C::CHUNKS; ++c, ++fill) {
                    const int slot = fill % NVS;
                    ok = wait_one<kFp8>(&full[slot], (fill / NVS) & 1, s_abort);
                    if (!ok) break;
                    tc_fence_after();
                    mma8_ss_f16<128, 128, 128, 128, 128, 128, 128, 128, 128, 128, 128, 128, 128, 128>(
                        tmem + C::O_COL + c * N, sdesc_adv(dv0, slot * C::CHUNK),
                        sdesc_adv(dp0, (blk & 1) * C::P_BYTES), IDESC_O, kind == kFirst ? 0u : 1u);
                    if (c == C::CHUNKS - 1) tc_commit(&pv_done[blk & 1]);
                    tc_commit(&empty[slot]);
                }
            }
            // Drain: no MMA of this warp is in flight at teardown.
            tc_commit(&bar_fin[1]);
            volatile int no_abort = 0;
            wait_one<kFp8>(&bar_fin[1], 0, &no_abort);
        }
        __syncwarp();
    } else if (kFp8 && warp >= C::V_CONV) {
        // ================= V from e4m3 to fp16 =================
        // A thread takes 16 bytes of a row at a time.  Eight consecutive ones take 64
        // head-dim columns of rows r and r ^ 5: their reads lie in opposite
        // halves of the swizzled 128 bytes (at d = 64: in rows of unlike parity), and
        // their two writes each in the even and the odd 16-byte groups: no two meet in a bank.
        const int tid = static_cast<int>(threadIdx.x) - 32 * C::V_CONV;
        const int cq = tid & 3, x = tid >> 3;
        const int cb = C::CCB == 2 ? x & 1 : 0, y = C::CCB == 2 ? x >> 1 : x;
        constexpr int STEP = 2048 / C::CW;   // rows from one piece of a thread to its next
        const int r0 = ((y >> 2) * 8 + (y & 3)) ^ ((tid & 4) ? 5 : 0);
        const int sw = C::CW == 128 ? r0 & 7 : (r0 >> 1) & 3;   // (the same in all its rows)
        const uint8_t* const src0 = sV + r0 * C::CW + (((4 * cb + cq) ^ sw) << 4);
        uint8_t* const dst0 = sW + cb * C::CB_BYTES + r0 * 128;
        const int d0 = ((2 * cq) ^ (r0 & 7)) << 4, d1 = ((2 * cq + 1) ^ (r0 & 7)) << 4;
        for (int fill = 0;; ++fill) {
            const int slot = fill % C::NV;
            if (!wait_warp_soon<kFp8>(&v_full[slot], (fill / C::NV) & 1, s_abort)) break;
            const int rows = s_vrows[slot];
            if (rows < 0) break;
            const int lo = rows & 255, hi = rows >> 8;
            const int to = fill % C::NW;
            if (!wait_warp_soon<kFp8>(&vt_empty[to], ((fill / C::NW) & 1) ^ 1, s_abort)) break;
            const uint8_t* const src = src0 + slot * C::SLOT;
            uint8_t* const dst = dst0 + to * C::CHUNK;
            // (a short loop: the four roles' loops on an SM sub-partition share its
            // instruction buffer, and unrolled ones starved one another, 118 -> 96 us
            // for 48 requests of up to 4200 keys)
#pragma unroll 4
            for (int it = 0; it < kTileRows / STEP; ++it) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);   // outside what is attended: whatever is there, even NaN
                if (static_cast<unsigned>(r0 + it * STEP - lo) < static_cast<unsigned>(hi - lo))
                    v = *reinterpret_cast<const uint4*>(src + it * STEP * C::CW);
                uint32_t w[8];
                e4m3x16_to_f16(v, w);
                *reinterpret_cast<uint4*>(dst + it * STEP * 128 + d0) = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4*>(dst + it * STEP * 128 + d1) = make_uint4(w[4], w[5], w[6], w[7]);
            }
            mbar_arrive_warp(&v_empty[slot]);
            fence_proxy_async_smem();
            mbar_arrive_warp(&vt_full[to]);
        }
    } else if (kFp8 && warp >= C::K_CONV) {
        // ================= K from e4m3 to fp16, bf16 queries to fp16 =================
        const int tid = static_cast<int>(threadIdx.x) - 32 * C::K_CONV;
        const uint32_t t_K = tmem + C::K_COL + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        int fill = 0;
        bool ok = true;
        for (int seg = 0; ok; ++seg) {
            const int buf = seg & 1;
            if (!wait_warp_soon<kFp8>(&q_full[buf], (seg >> 1) & 1, s_abort)) break;
            const int nblk = s_seg[buf].nblk;
            const bool none = s_seg[buf].none != 0;
            if constexpr (kTurnQ) {
                // A row's largest element goes to [2^14, 2^15): elements down to 2^-28 of
                // it keep all bits, smaller ones are off by 2^-39 of it.
                if (nblk > 0 && !none) {
                    constexpr int TPR = 128 / N, PIECES = D / 8 / TPR;   // threads and 16-byte pieces of a row
                    const int n = tid / TPR;
                    auto piece = [&](int i) {
                        const int c = tid % TPR + i * TPR;
                        return reinterpret_cast<uint4*>(sQ + buf * C::Q_BYTES + (c >> 3) * C::QCB_BYTES + n * 128 +
                                                        (((c & 7) ^ (n & 7)) << 4));
                    };
                    uint32_t top = 0;   // largest magnitude, as bf16 bits in either half
#pragma unroll 4
                    for (int i = 0; i < PIECES; ++i) {
                        const uint4 v = *piece(i);
                        top = __vmaxu2(__vmaxu2(top, __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu)),
                                       __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
                    }
                    top = max(top & 0xffffu, top >> 16);
#pragma unroll
                    for (int o = 1; o < TPR; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    const int ea = max(static_cast<int>(top >> 7) - 127, -100);
                    const float up = exp2_int(14 - ea);
                    // (four of them: the softmax, which has let go of the queries' buffer by
                    // then, reads them while this warp may be two segments ahead)
                    if (tid % TPR == 0) s_qs[(seg & 3) * 64 + n] = exp2_int(ea - 14);
#pragma unroll 4
                    for (int i = 0; i < PIECES; ++i) {
                        uint4* const at = piece(i);
                        const uint4 v = *at;
                        auto turn = [&](uint32_t w) {
                            return pack_f16x2(bf16lo_to_f32(w) * up, bf16hi_to_f32(w) * up);
                        };
                        *at = make_uint4(turn(v.x), turn(v.y), turn(v.z), turn(v.w));
                    }
                    fence_proxy_async_smem();
                }
                mbar_arrive_warp(&q_turned[buf]);
            }
            mbar_arrive_warp(&q_empty[buf]);
            if (nblk == 0) break;
            for (int x = 0; x < (none ? 0 : nblk * C::CHUNKS) && ok; ++x, ++fill) {
                const int slot = fill % C::NK;
                ok = wait_warp_soon<kFp8>(&k_full[slot], (fill / C::NK) & 1, s_abort);
                if (ok && fill >= 2) ok = wait_warp_soon<kFp8>(&kt_empty[fill & 1], ((fill >> 1) & 1) ^ 1, s_abort);
                if (!ok) break;
                tc_fence_after();
                // a key per lane: 64 head-dim elements at a time
#pragma unroll 1
                for (int cb = 0; cb < C::CCB; ++cb) {
                    uint32_t w[32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c = 4 * cb + i;
                        const uint4 v = *reinterpret_cast<const uint4*>(
                            sK + slot * C::SLOT + tid * C::CW +
                            ((c ^ (C::CW == 128 ? tid & 7 : (tid >> 1) & 3)) << 4));
                        uint32_t h[8];
                        e4m3x16_to_f16(v, h);
#pragma unroll
                        for (int e = 0; e < 8; ++e) w[8 * i + e] = h[e];
                    }
                    tmem_st32(t_K + (fill & 1) * (C::CW / 2) + 32 * cb, w);
                }
                mbar_arrive_warp(&k_empty[slot]);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive_warp(&kt_full[fill & 1]);
            }
        }
    } else {
        // ================= softmax (one thread per key and group of columns) =================
        // The groups share nothing but the barriers: rows are columns here.
        const int tid = static_cast<int>(threadIdx.x) & 127;
        const int quarter = warp & 3;
        const int group = C::GROUPS == 1 ? 0 : warp >> 2;
        const int c0 = group * NC;      // first row of this group
        const int bar = 1 + group;      // the group's hardware barrier
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t t_S = t_lane + c0;
        const uint32_t t_O = t_lane + C::O_COL + c0;
        float* const g_row = s_row + c0;     // [4][N]
        float* const g_negm = s_negm + c0;   // [NC], as the rest
        float* const g_fac = s_fac + c0;
        int* const g_lo = s_lo + c0;
        uint32_t* const g_num = s_num + c0;
        constexpr int W = NC < 16 ? NC : 16;   // columns of O^T at a time
        const int G = p.G;
        const float sc = p.scale_log2;
        const uint64_t sc2 = f2_pack(sc, sc);
        // Pieces go to the workspace, or, in a cluster, to shared memory where
        // the K ring (fp8: widened V) was (this CTA's only segment is over by then).
        float* const piece_o = p.cluster > 0 ? reinterpret_cast<float*>(kFp8 ? sW : sK) : p.part_o;
        float* const piece_lse = p.cluster > 0 ? s_lse : p.part_lse;
        const int piece_rows = p.cluster > 0 ? N : p.slot_rows;
        int blk0 = 0;   // blocks of the segments before
        bool ok = true;
        for (int seg = 0;; ++seg) {
            const int buf = seg & 1;
            // A group's warps meet at barriers inside a segment, so all of them
            // take it or none does; a wait that fails inside leaves the results
            // unspecified and ends the walk at the next segment.
            ok = ok && wait_warp<kFp8>(&q_full[buf], (seg >> 1) & 1, s_abort);
            if (named_barrier_or(bar, 128, !ok)) break;
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
            const int rows = min(NC, s.ntok * G - c0);   // of this group; may be none
            if (tid < NC) {   // what row c0 + tid attends: a run of keys
                const int pos = s.off + (c0 + tid) / G;
                int lo = s.klo, hi = s.khi;
                if (p.causal) hi = min(hi, pos + 1);
                if (p.window > 0) {
                    lo = max(lo, pos - p.window + 1);
                    if (!p.causal) hi = min(hi, pos + p.window);
                }
                g_lo[tid] = lo;
                g_num[tid] = static_cast<uint32_t>(max(0, hi - lo));
            }
            // Blocks where some row does not attend some key: the range's ends, the
            // causal diagonal (queries are the last ntok keys), and a window's
            // start, which moves with the query.  The others begin at keys [clear_lo, clear_hi].
            int clear_lo = s.klo, clear_hi = s.khi - kTileRows;
            if (p.causal) clear_hi = min(clear_hi, s.off - kTileRows + 1);
            if (p.window > 0) {
                clear_lo = max(clear_lo, s.off + s.ntok - p.window);
                if (!p.causal) clear_hi = min(clear_hi, s.off + p.window - kTileRows);
            }
            named_barrier_sync(bar, 128);
            // With eight rows a thread, what a block needs of them stays in registers.
            constexpr bool kKeep = NC == 8;
            uint64_t kept_nm[NC / 2], kept_qs[NC / 2];
            uint64_t l[NC / 2];   // this thread's sums, two rows each
#pragma unroll
            for (int n = 0; n < NC / 2; ++n) l[n] = f2_pack(0.f, 0.f);
            const int nblk = s.none ? 0 : s.nblk;
            for (int x = 0; x < nblk; ++x) {
                const int blk = blk0 + x;
                const int k0 = (s.j0 + x) * kTileRows;
                const int key = k0 + tid;
                // (fp8) The factor of this key's scores and the exponent ev of its V's scale
                float key_f = 1.f, key_ev = 0.f;
                if constexpr (kFp8) {
                    ok = ok && wait_warp_soon<kFp8>(&sc_full[blk & 15], (blk >> 4) & 1, s_abort);
                    const float2 both = const_cast<const float2*>(reinterpret_cast<volatile float2*>(s_scale))[
                        (blk & 15) * 16 + (tid >> box_log)];
                    key_f = both.x;
                    key_ev = both.y;
                }
                ok = ok && wait_warp_soon<kFp8>(&s_full[blk & 1], (blk >> 1) & 1, s_abort);
                tc_fence_after();
                uint32_t sr[NC];
                tmem_ld_cols<NC>(t_S + (blk & 1) * N, sr);
                tmem_ld_wait();
                reg_fence(sr);
                if (k0 < clear_lo || k0 > clear_hi) {
#pragma unroll
                    for (int n = 0; n < NC; ++n)
                        if (static_cast<uint32_t>(key - g_lo[n]) >= g_num[n]) sr[n] = __float_as_uint(-INFINITY);
                }
                // (fp8) Scores become exponents s scale log2e + ev in place: weights are
                // taken times 2^ev, references are of s + ev, and the sum takes 2^ev off again.
                uint64_t off2 = 0;
                if constexpr (kFp8) {
                    const float off = exp2_int(-static_cast<int>(key_ev));
                    const uint64_t f2 = f2_pack(key_f, key_f), ev2 = f2_pack(key_ev, key_ev);
                    off2 = f2_pack(off, off);
                    const uint64_t* const qs = reinterpret_cast<const uint64_t*>(s_qs + (seg & 3) * 64 + c0);
#pragma unroll
                    for (int n = 0; n < NC; n += 2) {
                        uint64_t v = f2_pack(__uint_as_float(sr[n]), __uint_as_float(sr[n + 1]));
                        if (kTurnQ && kKeep && x == 0) kept_qs[n / 2] = qs[n / 2];
                        v = kTurnQ ? f2_fma(f2_mul(v, f2), kKeep ? kept_qs[n / 2] : qs[n / 2], ev2) : f2_fma(v, f2, ev2);
                        float lo, hi;
                        f2_unpack(v, lo, hi);
                        sr[n] = __float_as_uint(lo);
                        sr[n + 1] = __float_as_uint(hi);
                    }
                }
                // Exponents s scale log2e - m, two rows at a time.  Rows past the
                // tile's have m = inf: exponent -inf, weight 0.
                auto exponents = [&](int c, float (&e)[8]) {   // of rows 8 c .. 8 c + 7
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int n = 8 * c + 2 * i;
                        const uint64_t nm = kKeep ? kept_nm[n / 2] : reinterpret_cast<const uint64_t*>(g_negm)[n / 2];
                        const uint64_t s2 = f2_pack(__uint_as_float(sr[n]), __uint_as_float(sr[n + 1]));
                        f2_unpack(kFp8 ? f2_add(s2, nm) : f2_fma(s2, sc2, nm), e[2 * i], e[2 * i + 1]);
                    }
                };
                float kept_e[8];
                bool grows = false;
                if (x > 0) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int c = 0; c < NC / 8; ++c) {
                        float now[8];
                        float(&e)[8] = kKeep ? kept_e : now;
                        exponents(c, e);
                        mx = max3f(max3f(e[0], e[1], e[2]), max3f(e[3], e[4], e[5]), max3f(e[6], e[7], mx));
                    }
                    grows = mx > kRescaleThreshold + kWeightShift<kMmaF16>;
                }
                const bool renewed = x == 0 || named_barrier_or(bar, 128, grows);
                if (renewed) {
                    // new references, from the maxima over the warp's keys, then over the four warps
                    float mine_max = -INFINITY;
#pragma unroll
                    for (int n = 0; n < NC; ++n) {
                        const float wm = key_float(__reduce_max_sync(0xffffffffu, float_key(__uint_as_float(sr[n]))));
                        if (n == lane) mine_max = wm;
                    }
                    if (lane < NC) g_row[quarter * N + lane] = mine_max;
                    named_barrier_sync(bar, 128);
                    if (tid < NC) {
                        const float old = x > 0 ? -g_negm[tid] : kNoMax;
                        const float mx = fmaxf(fmaxf(g_row[tid], g_row[N + tid]),
                                               fmaxf(g_row[2 * N + tid], g_row[3 * N + tid]));
                        const float mt = fmaxf(old, (kFp8 ? mx : sc * mx) - kWeightShift<kMmaF16>);
                        g_negm[tid] = tid < rows ? -mt : -INFINITY;
                        g_fac[tid] = tid < rows ? ex2_approx(old - mt) : 0.f;
                    }
                    named_barrier_sync(bar, 128);
                    if (x > 0) {   // sums and O^T columns, once P V of the block before is in
                        ok = ok && wait_warp<kFp8>(&pv_done[(blk - 1) & 1], ((blk - 1) >> 1) & 1, s_abort);
                        tc_fence_after();
#pragma unroll
                        for (int n = 0; n < NC / 2; ++n) l[n] = f2_mul(l[n], reinterpret_cast<const uint64_t*>(g_fac)[n]);
#pragma unroll 1
                        for (int c = 0; c < C::HALVES * NC / W; ++c) {
                            const uint32_t at = t_O + c / (NC / W) * N + W * (c % (NC / W));
                            uint32_t o[W];
                            tmem_ld_cols<W>(at, o);
                            tmem_ld_wait();
                            reg_fence(o);
#pragma unroll
                            for (int n = 0; n < W; ++n)
                                o[n] = __float_as_uint(__uint_as_float(o[n]) * g_fac[(W * c + n) % NC]);
                            if constexpr (W == 8) tmem_st8(at, o);
                            else tmem_st16(at, o);
                        }
                        tmem_st_wait();
                    }
                }
                if (kKeep && renewed) {
#pragma unroll
                    for (int n = 0; n < NC / 2; ++n) kept_nm[n] = reinterpret_cast<const uint64_t*>(g_negm)[n];
                    exponents(0, kept_e);
                }
                // P^T: this key's N weights, rounded to the storage type for the
                // product with V; the sum takes them unrounded
                if (blk >= 2) ok = ok && wait_warp_soon<kFp8>(&pv_done[blk & 1], ((blk >> 1) & 1) ^ 1, s_abort);
                uint8_t* row = sP + (blk & 1) * C::P_BYTES + tid * 128;
#pragma unroll
                for (int c = 0; c < NC / 8; ++c) {
                    float now[8];
                    float(&e)[8] = kKeep ? kept_e : now;
                    if (!kKeep) exponents(c, e);
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p0 = ex2_approx(e[2 * i]);
                        const float p1 = ex2_approx(e[2 * i + 1]);
                        if constexpr (kFp8) l[4 * c + i] = f2_fma(f2_pack(p0, p1), off2, l[4 * c + i]);
                        else l[4 * c + i] = f2_add(l[4 * c + i], f2_pack(p0, p1));
                        w[i] = pack_h2<kMmaF16>(p0, p1);
                    }
                    *reinterpret_cast<uint4*>(row + (((c0 / 8 + c) ^ (tid & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (!kFp8 && (k0 < s.klo || k0 + kTileRows > s.khi)) {
                    // V rows of keys outside [klo, khi) become zero.  Their slots'
                    // fills before this one must have landed, or the parity would
                    // be theirs: with a tile in two slots that takes P V of the
                    // block before, else that of two blocks before (above).
                    if (C::CHUNKS == 2 && blk > 0)
                        ok = ok && wait_warp<kFp8>(&pv_done[(blk - 1) & 1], ((blk - 1) >> 1) & 1, s_abort);
                    for (int c = 0; c < C::CHUNKS; ++c) {   // (each group clears all of them)
                        const int f = C::CHUNKS * blk + c;
                        ok = ok && wait_warp<kFp8>(&v_full[f % C::NV], (f / C::NV) & 1, s_abort);
                        if (ok && (key < s.klo || key >= s.khi)) {
                            for (int cb = 0; cb < C::CCB; ++cb) {
                                uint4* vr = reinterpret_cast<uint4*>(sV + (f % C::NV) * C::SLOT + cb * C::CB_BYTES +
                                                                     tid * 128);
#pragma unroll
                                for (int e = 0; e < 8; ++e) vr[e] = make_uint4(0u, 0u, 0u, 0u);
                            }
                        }
                    }
                }
                if (threadIdx.x == 0) s_kind[blk & 1] = x == 0 ? kFirst : 0;
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive_warp(&p_full[blk & 1]);
            }
            // ---- the segment's result: sums over all keys, O = acc / l ----
            float ls[NC];
#pragma unroll
            for (int n = 0; n < NC / 2; ++n) f2_unpack(l[n], ls[2 * n], ls[2 * n + 1]);
            const int col = warp_sum_scatter<NC>(ls, lane);
            if ((lane & (32 / NC - 1)) == 0) g_row[quarter * N + col] = ls[0];
            named_barrier_sync(bar, 128);
            if (tid < NC) {
                const float sum = (g_row[tid] + g_row[N + tid]) + (g_row[2 * N + tid] + g_row[3 * N + tid]);
                g_fac[tid] = sum == 0.f ? 0.f : 1.f / sum;
                if (tid < rows) {
                    const float lse2 = sum == 0.f ? -INFINITY : log2f(sum) - g_negm[tid];
                    const int n = c0 + tid;
                    if (s.out >= 0) {
                        piece_lse[static_cast<size_t>(s.out) * piece_rows + n] = lse2;
                    } else {
                        const int tok = n / G;
                        p.LSE[static_cast<size_t>(s.hk * G + n - tok * G) * p.lq.total + s.q_start + tok] =
                            lse2 * kLn2;
                    }
                }
            }
            blk0 += nblk;
            if (!s.none) {
                const int last = blk0 - 1;
                ok = ok && wait_warp<kFp8>(&pv_done[last & 1], (last >> 1) & 1, s_abort);
                tc_fence_after();
            }
            named_barrier_sync(bar, 128);
            // Row n of lane d: consecutive lanes, consecutive columns of a row.
            // A piece's rows are D floats apart, the output's H D after the last
            // head of a token.
            const int tok0 = c0 / G, g0 = c0 - tok0 * G;   // of the group's first row
            const size_t out0 = s.out >= 0 ? (static_cast<size_t>(s.out) * piece_rows + c0) * D
                                           : ((static_cast<size_t>(s.q_start) + tok0) * p.lq.H + s.hk * G + g0) * D;
            const size_t skip = s.out >= 0 ? 0 : static_cast<size_t>(p.lq.H - G) * D;
#pragma unroll 1
            for (int h = 0; h < C::HALVES; ++h) {
                size_t at = out0 + h * 128 + tid;
                int g = g0;
#pragma unroll 1
                for (int c = 0; c < NC / W; ++c) {
                    if (W * c >= rows) break;
                    uint32_t o[W];
                    if (!s.none) {
                        tmem_ld_cols<W>(t_O + h * N + W * c, o);
                        tmem_ld_wait();
                        reg_fence(o);
                    } else {
#pragma unroll
                        for (int n = 0; n < W; ++n) o[n] = 0u;
                    }
                    if (D >= 128 || tid < D) {
#pragma unroll
                        for (int n = 0; n < W; ++n) {
                            if (W * c + n < rows) {
                                const float y = __uint_as_float(o[n]) * g_fac[W * c + n];
                                if (s.out >= 0)
                                    piece_o[at] = y;
                                else
                                    static_cast<uint16_t*>(p.O)[at] =
                                        static_cast<uint16_t>(pack_h2<kF16>(y, 0.f));
                            }
                            at += D;
                            if (++g == G) {
                                g = 0;
                                at += skip;
                            }
                        }
                    }
                    __syncwarp();
                }
            }
            // O^T is read: the next segment's first P V, which overwrites it,
            // waits for P^T of these threads.
            tc_fence_before();
        }
        if (ok) {   // tell the P V warp
            if (threadIdx.x == 0) s_kind[blk0 & 1] = kStop;
            mbar_arrive_warp(&p_full[blk0 & 1]);
        }
    }

    // ---- a cluster's pieces become its tile's result ----
    if (p.cluster > 1) {
        const int rank = cta % p.cluster, tile = cta / p.cluster;
        const int b = tile / p.Hkv, hk = tile - b * p.Hkv;
        const Request r = request_of(p, b);
        const int share = (r.units + p.cluster - 1) / p.cluster;
        const bool whole = share >= r.units;   // written by rank 0
        // pieces without a key, for CTAs that had no block
        if (rank * share >= r.units && threadIdx.x < N) s_lse[threadIdx.x] = -INFINITY;
        cluster_sync();
        for (int n = rank * (C::THREADS / 32) + warp; n < r.n * p.G && !whole;
             n += p.cluster * (C::THREADS / 32)) {
            float w = lane < p.cluster ? ld_cluster(&s_lse[n], lane) : -INFINITY;
            float M = w;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            M = __shfl_sync(0xffffffffu, M, 0);
            w = M == -INFINITY ? 0.f : ex2_approx(w - M);
            float sum = w;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            sum = __shfl_sync(0xffffffffu, sum, 0);
            constexpr int PER = D / 32;
            const float* src = reinterpret_cast<const float*>(kFp8 ? sW : sK) + n * D + lane * PER;
            float2 x[8][PER / 2];   // all pieces' loads before the first is used
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < p.cluster) {
#pragma unroll
                    for (int e = 0; e < PER / 2; ++e) x[i][e] = ld_cluster2(src + 2 * e, i);
                }
            float acc[PER];
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[e] = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float wi = __shfl_sync(0xffffffffu, w, i);
                if (i < p.cluster && wi != 0.f) {   // else no key, or no piece at all
#pragma unroll
                    for (int e = 0; e < PER / 2; ++e) {
                        acc[2 * e] += wi * x[i][e].x;
                        acc[2 * e + 1] += wi * x[i][e].y;
                    }
                }
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const int tok = n / p.G, head = hk * p.G + n - tok * p.G;
            uint32_t* dst = reinterpret_cast<uint32_t*>(
                static_cast<uint16_t*>(p.O) + ((static_cast<size_t>(r.start) + tok) * p.lq.H + head) * D + lane * PER);
#pragma unroll
            for (int e = 0; e < PER / 2; ++e) dst[e] = pack_h2<kF16>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
            if (lane == 0)
                p.LSE[static_cast<size_t>(head) * p.lq.total + r.start + tok] =
                    sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
        }
        cluster_sync();   // no CTA leaves while another reads its piece
    }

    // ---- teardown ----
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == C::S_WARP) tmem_dealloc(tmem, C::TMEM_COLS);
    if (threadIdx.x == 0 && *s_abort && p.dev_status != nullptr)
        atomicCAS(p.dev_status, 0, static_cast<int>(ATTN_ERR_DEVICE_TIMEOUT));
    if (blockIdx.x == 0) paged_report(p);
}

template <int D, bool kF16, int N, bool kFp8>
cudaError_t launch_decode_t(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                            const PagedParams& p, cudaStream_t stream) {
    using C = DecodeCfg<D, N, kFp8>;
    auto kern = attn_decode_kernel<D, kF16, N, kFp8>;
    static std::atomic<unsigned long long> smem_ready{0};
    const cudaError_t e = enable_smem_per_device(kern, C::SMEM, smem_ready);
    if (e != cudaSuccess) return e;
    return launch_overlapped_cluster(kern, static_cast<unsigned>(p.tiles), C::THREADS, C::SMEM, p.cluster, true, stream,
                                     tq, tk, tv, p);
}

template <int D, bool kF16, bool kFp8 = false>
cudaError_t launch_decode_n(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                            const PagedParams& p, cudaStream_t stream) {
    switch (p.slot_rows) {
        case 16: return launch_decode_t<D, kF16, 16, kFp8>(tq, tk, tv, p, stream);
        case 32: return launch_decode_t<D, kF16, 32, kFp8>(tq, tk, tv, p, stream);
        case 64: return launch_decode_t<D, kF16, 64, kFp8>(tq, tk, tv, p, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace gbattn
