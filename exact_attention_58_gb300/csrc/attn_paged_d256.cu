// attn_paged_d256.cu — the paged attention kernel at head dim 256 (one query tile per CTA);
// compiles in parallel with attn_paged.cu.
#include "attn_paged_kernel.cuh"

namespace gbattn {

cudaError_t launch_paged_tiles_d256(const CUtensorMap& tq, const CUtensorMap& tk,
                                    const CUtensorMap& tv, const PagedParams& p, bool f16,
                                    cudaStream_t stream) {
    return p.fine ? launch_paged_f<256, 1, true>(tq, tk, tv, p, f16, stream)
                  : launch_paged_f<256, 1, false>(tq, tk, tv, p, f16, stream);
}

}  // namespace gbattn
