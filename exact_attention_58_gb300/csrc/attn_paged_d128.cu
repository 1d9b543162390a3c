// attn_paged_d128.cu — the paged attention kernel at head dim 128;
// compiles in parallel with attn_paged.cu.
#include "attn_paged_kernel.cuh"

namespace gbattn {

cudaError_t launch_paged_tiles_d128(const CUtensorMap& tq, const CUtensorMap& tk,
                                    const CUtensorMap& tv, const PagedParams& p, bool f16,
                                    cudaStream_t stream) {
    return p.fine ? launch_paged_f<128, 2, true>(tq, tk, tv, p, f16, stream)
                  : launch_paged_f<128, 2, false>(tq, tk, tv, p, f16, stream);
}

}  // namespace gbattn
