// attn_paged_fp8.cu — launches of the paged attention kernel (attn_paged_kernel.cuh)
// over a cache of e4m3.
#include "attn_paged_kernel.cuh"

namespace gbattn {

cudaError_t launch_paged_tiles_fp8(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                   const PagedParams& p, int d, bool f16, cudaStream_t stream) {
    switch (d) {
        case 64: return launch_paged_8<64, 2>(tq, tk, tv, p, f16, stream);
        case 128: return launch_paged_8<128, 2>(tq, tk, tv, p, f16, stream);
        case 256: return launch_paged_8<256, 1>(tq, tk, tv, p, f16, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gbattn
