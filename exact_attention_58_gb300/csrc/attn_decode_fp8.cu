// attn_decode_fp8.cu — launches of the decode attention kernel over a cache of
// e4m3 (attn_decode_kernel.cuh) at head dim 64; head dims 128 and 256 compile
// beside it in attn_decode_fp8_d128.cu and attn_decode_fp8_d256.cu.
#include "attn_decode_kernel.cuh"

namespace gbattn {

cudaError_t launch_paged_decode_fp8(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                    const PagedParams& p, int d, bool f16, cudaStream_t stream) {
    switch (d) {
        case 64: return f16 ? launch_decode_n<64, true, true>(tq, tk, tv, p, stream)
                            : launch_decode_n<64, false, true>(tq, tk, tv, p, stream);
        case 128: return launch_paged_decode_fp8_d128(tq, tk, tv, p, f16, stream);
        case 256: return launch_paged_decode_fp8_d256(tq, tk, tv, p, f16, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gbattn
