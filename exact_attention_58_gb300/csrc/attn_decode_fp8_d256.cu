// attn_decode_fp8_d256.cu — the decode attention kernel over a cache of e4m3 at
// head dim 256.
#include "attn_decode_kernel.cuh"

namespace gbattn {

cudaError_t launch_paged_decode_fp8_d256(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                         const PagedParams& p, bool f16, cudaStream_t stream) {
    return f16 ? launch_decode_n<256, true, true>(tq, tk, tv, p, stream)
               : launch_decode_n<256, false, true>(tq, tk, tv, p, stream);
}

}  // namespace gbattn
