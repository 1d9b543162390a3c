// attn_decode.cu — launches of the decode kernel (attn_decode_kernel.cuh) at
// head dims 64 and 128; head dim 256 compiles beside it in attn_decode_d256.cu.
#include "attn_decode_kernel.cuh"

namespace gbattn {

cudaError_t launch_paged_decode(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                const PagedParams& p, int d, bool f16, cudaStream_t stream) {
    switch (d) {
        case 64: return f16 ? launch_decode_n<64, true>(tq, tk, tv, p, stream)
                            : launch_decode_n<64, false>(tq, tk, tv, p, stream);
        case 128: return f16 ? launch_decode_n<128, true>(tq, tk, tv, p, stream)
                             : launch_decode_n<128, false>(tq, tk, tv, p, stream);
        case 256: return launch_paged_decode_d256(tq, tk, tv, p, f16, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gbattn
