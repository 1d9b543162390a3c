// attn_paged.cu — launches of the paged attention kernel (attn_paged_kernel.cuh)
// at head dim 64, and the kernel that joins pieces; head dims 128 and 256 compile
// beside it in attn_paged_d128.cu and attn_paged_d256.cu.
#include "attn_paged_kernel.cuh"

namespace gbattn {
namespace {

// Joins the pieces of split tiles.  Row r of a tile has n pieces (O_i, lse2_i)
// over disjoint key sets: with M = max lse2_i and w_i = exp2(lse2_i - M),
// O = sum w_i O_i / sum w_i and LSE = (M + log2 sum w_i) ln 2.  The pieces were
// written by the launch before and come from L2, so the time is that of
// dependent loads: each warp asks for the O_i of up to kBatch pieces before it
// knows their weights.  A row takes one warp, or (kPerRow) the eight of a CTA,
// which share its pieces: for few tiles, where one long context can be in as many
// pieces as there are CTAs (76 pieces a row: 9 -> 6 us).  Where there are only a
// few pieces a row, kBatch = 4 leaves registers for more CTAs at a time.  The order of the sums is
// fixed either way.  Most CTAs find nothing to join and leave, so there should
// not be many of them: 6000 took 15 us to come and go.
template <int D, bool kF16, int kPerRow, int kBatch>
__global__ void __launch_bounds__(kPerRow > 1 ? 32 * kPerRow : 128) paged_join_kernel(const PagedParams p) {
    grid_dep_wait();
    grid_dep_launch_dependents();
    constexpr int PER = D / 32;   // floats of a lane
    constexpr int kWarps = kPerRow > 1 ? kPerRow : 4;
    __shared__ float s_acc[kPerRow][D];
    __shared__ float s_sum[kPerRow];
    const PieceDesc t = p.desc[blockIdx.x];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = warp % kPerRow;
    constexpr int kRows = kWarps / kPerRow;   // of a CTA at a time
    const int rows = t.n == 0 ? 0 : t.ntok * p.G;
    // u: (token, head of the group); the same for all warps of a row
    for (int u = blockIdx.y * kRows + warp / kPerRow; u < rows; u += gridDim.y * kRows) {
        const int tok = u / p.G, g = u - tok * p.G;
        const int row = tok / p.tile_tokens * kTileRows + (tok % p.tile_tokens) * p.G + g;
        auto piece_row = [&](int i) {
            const int slot = i == 0 ? t.slot0 : t.slot1 + (i - 1) * t.step;
            return static_cast<size_t>(slot) * p.slot_rows + row;
        };
        float M = -INFINITY, m0 = 0.f, acc[PER], sum = 0.f;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] = 0.f;
        for (int i0 = part; i0 < t.n || i0 == part; i0 += kBatch * kPerRow) {
            float2 x[kBatch][PER / 2];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int i = i0 + k * kPerRow;
                const float2* src = reinterpret_cast<const float2*>(p.part_o + piece_row(i) * D) + lane * (PER / 2);
#pragma unroll
                for (int e = 0; e < PER / 2; ++e) x[k][e] = i < t.n ? src[e] : make_float2(0.f, 0.f);
            }
            // lane k: the log-sum-exp, then the weight, of piece i0 + k kPerRow
            const int mine = i0 + lane * kPerRow;
            const float lse_mine = lane < kBatch && mine < t.n ? p.part_lse[piece_row(mine)] : -INFINITY;
            if (i0 == part) {   // first batch: the maximum over all pieces
                for (int i = lane; i < t.n; i += 32) M = fmaxf(M, p.part_lse[piece_row(i)]);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
                m0 = M == -INFINITY ? 0.f : M;
            }
            const float w_mine = ex2_approx(lse_mine - m0);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const float w = __shfl_sync(0xffffffffu, w_mine, k);
                sum += w;
#pragma unroll
                for (int e = 0; e < PER / 2; ++e) {
                    acc[2 * e] += w * x[k][e].x;
                    acc[2 * e + 1] += w * x[k][e].y;
                }
            }
        }
        if constexpr (kPerRow > 1) {
#pragma unroll
            for (int e = 0; e < PER; ++e) s_acc[part][lane * PER + e] = acc[e];
            if (lane == 0) s_sum[part] = sum;
            __syncthreads();
            sum = 0.f;
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[e] = 0.f;
#pragma unroll
            for (int w = 0; w < kPerRow; ++w) {
                sum += s_sum[w];
#pragma unroll
                for (int e = 0; e < PER; ++e) acc[e] += s_acc[w][lane * PER + e];
            }
            __syncthreads();   // the next row's turn
            if (part != 0) continue;
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int head = t.hk * p.G + g;
        const size_t out_row = (static_cast<size_t>(t.q_start) + t.tok0 + tok) * p.lq.H + head;
        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.O) + out_row * D) + lane * (PER / 2);
#pragma unroll
        for (int e = 0; e < PER / 2; ++e) dst[e] = pack_h2<kF16>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
        if (lane == 0)
            p.LSE[static_cast<size_t>(head) * p.lq.total + t.q_start + t.tok0 + tok] =
                sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
    }
}

template <int D, bool kF16>
cudaError_t launch_join_t(cudaLaunchConfig_t& cfg, int descs, int rows, JoinKind kind, const PagedParams& p) {
    const int groups = kind == kJoinFewRows ? rows : (rows + 3) / 4;
    cfg.gridDim = dim3(static_cast<unsigned>(descs), static_cast<unsigned>(groups < 16 ? groups : 16));
    cfg.blockDim = dim3(kind == kJoinFewRows ? 256 : 128);
    switch (kind) {
        case kJoinFewRows: return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, kF16, 8, 10>, p);
        case kJoinFewPieces: return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, kF16, 1, 4>, p);
        case kJoinMany: return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, kF16, 1, 10>, p);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_paged_join(const PagedParams& p, int descs, int rows, JoinKind kind, int d, bool f16,
                              cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    switch (d) {
        case 64: return f16 ? launch_join_t<64, true>(cfg, descs, rows, kind, p)
                            : launch_join_t<64, false>(cfg, descs, rows, kind, p);
        case 128: return f16 ? launch_join_t<128, true>(cfg, descs, rows, kind, p)
                             : launch_join_t<128, false>(cfg, descs, rows, kind, p);
        case 256: return f16 ? launch_join_t<256, true>(cfg, descs, rows, kind, p)
                             : launch_join_t<256, false>(cfg, descs, rows, kind, p);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_paged_tiles(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const PagedParams& p, int d, bool f16, cudaStream_t stream) {
    switch (d) {
        case 64: return launch_paged_f<64, 2, false>(tq, tk, tv, p, f16, stream);
        case 128: return launch_paged_tiles_d128(tq, tk, tv, p, f16, stream);
        case 256: return launch_paged_tiles_d256(tq, tk, tv, p, f16, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gbattn
