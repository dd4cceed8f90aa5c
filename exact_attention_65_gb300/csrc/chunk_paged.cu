// Forward of the new tokens of each request over a paged cache
// (attn_chunk_paged): the kernel of fwd_packed.cuh with K and V tiles gathered
// from pages.
#include "fwd_packed.cuh"

namespace exattn {

cudaError_t launch_chunk_paged(int d, bool bf16, const CUtensorMap &tq, const CUtensorMap &tk,
                               const CUtensorMap &tv, const PackArgs &a, cudaStream_t stream) {
    return launch_pack<true>(d, bf16, tq, tk, tv, a, stream);
}

}  // namespace exattn
