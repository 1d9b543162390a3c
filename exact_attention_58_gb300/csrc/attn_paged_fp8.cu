// attn_paged_fp8.cu — attention of new tokens over a paged cache held in e4m3.
#include "fp8.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace gbattn {
namespace {

constexpr float kLn2f = 0.69314718055994530942f;

// One warp per query token and head: the online softmax over its keys, one key
// at a time, D / 32 head-dim elements a lane.
template <int D, bool kF16>
__global__ void __launch_bounds__(256) attn_paged_fp8_kernel(const PagedParams p, const Fp8Cache c) {
    grid_dep_wait();
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31;
    const long long units = static_cast<long long>(p.B) * p.lq.N * p.lq.H;
    if (blockIdx.x == 0) paged_report(p);
    for (long long x = blockIdx.x * 8ll + (threadIdx.x >> 5); x < units; x += gridDim.x * 8ll) {
        const int h = static_cast<int>(x % p.lq.H);
        const long long y = x / p.lq.H;
        const int i = static_cast<int>(y % p.lq.N), b = static_cast<int>(y / p.lq.N);
        const SeqSpan sq = seq_span(p.lq, b, nullptr, false);
        if (i >= sq.len) continue;
        const int L = paged_keys(p, b), hk = h / p.G;
        int lo, hi;
        key_range(p, i, i, L - sq.len, L, lo, hi);
        const size_t t = static_cast<size_t>(sq.start) + i;
        const uint16_t* q = static_cast<const uint16_t*>(c.Q) + t * c.q_token_stride + h * c.q_head_stride + lane * PER;
        float qf[PER], o[PER], m = -INFINITY, l = 0.f;
        for (int e = 0; e < PER; ++e) {
            qf[e] = h2lo_to_f32<kF16>(q[e]);
            o[e] = 0.f;
        }
        const int32_t* table = p.page_table + static_cast<size_t>(b) * p.max_pages;
        for (int j = lo; j < hi; ++j) {
            const int col = j / p.page_size, row = j - col * p.page_size;
            const int page = table[col];
            const bool in = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
            if (!in && p.dev_status != nullptr) atomicCAS(p.dev_status, 0, static_cast<int>(ATTN_ERR_INVALID_ARG));
            float ks = 1.f, vs = 1.f, kf[PER], vf[PER], s = 0.f;
            const long long at = in ? page * c.page_stride + hk * c.head_stride + row * c.token_stride + lane * PER : 0;
            if (in) {
                const uint32_t kb = __float_as_uint(c.k_scale[static_cast<size_t>(page) * p.Hkv + hk]);
                const uint32_t vb = __float_as_uint(c.v_scale[static_cast<size_t>(page) * p.Hkv + hk]);
                if ((bad_scale(kb) || bad_scale(vb)) && p.dev_status != nullptr)
                    atomicCAS(p.dev_status, 0, static_cast<int>(ATTN_ERR_INVALID_ARG));
                ks = exp2_int(scale_exponent(kb));
                vs = exp2_int(scale_exponent(vb));
            }
            for (int e = 0; e < PER; e += 2) {
                const uint32_t kk = in ? e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(c.k + at + e)) : 0u;
                const uint32_t vv = in ? e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(c.v + at + e)) : 0u;
                kf[e] = f16lo_to_f32(kk);
                kf[e + 1] = f16hi_to_f32(kk);
                vf[e] = f16lo_to_f32(vv) * vs;
                vf[e + 1] = f16hi_to_f32(vv) * vs;
            }
            for (int e = 0; e < PER; ++e) s += qf[e] * kf[e];
            for (int x2 = 16; x2 > 0; x2 >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x2);
            s *= ks * p.scale_log2;
            const float mn = fmaxf(m, s), a = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(s - mn);
            m = mn;
            l = l * a + w;
            for (int e = 0; e < PER; ++e) o[e] = o[e] * a + w * vf[e];
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t* out = static_cast<uint16_t*>(p.O) + (t * p.lq.H + h) * D + lane * PER;
        for (int e = 0; e < PER; ++e) out[e] = static_cast<uint16_t>(pack_h2<kF16>(o[e] * inv, 0.f));
        if (lane == 0)
            p.LSE[static_cast<size_t>(h) * p.lq.total + t] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2f;
    }
}

}  // namespace

cudaError_t launch_paged_fp8(const PagedParams& p, const Fp8Cache& c, int d, bool f16, cudaStream_t stream) {
    const long long units = (static_cast<long long>(p.B) * p.lq.N * p.lq.H + 7) / 8;
    const unsigned grid = static_cast<unsigned>(units < kSMs * 8 ? units : kSMs * 8);
    auto go = [&](auto kern) { return launch_overlapped(kern, grid, 256, 0, stream, p, c); };
    switch (d) {
        case 64: return f16 ? go(attn_paged_fp8_kernel<64, true>) : go(attn_paged_fp8_kernel<64, false>);
        case 128: return f16 ? go(attn_paged_fp8_kernel<128, true>) : go(attn_paged_fp8_kernel<128, false>);
        case 256: return f16 ? go(attn_paged_fp8_kernel<256, true>) : go(attn_paged_fp8_kernel<256, false>);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gbattn
