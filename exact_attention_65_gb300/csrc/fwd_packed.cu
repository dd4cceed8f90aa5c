// Forward over prompts packed one behind the other (attn_fwd_packed): the
// kernel of fwd_packed.cuh with K and V read from packed tensors.
#include "fwd_packed.cuh"

namespace exattn {

cudaError_t launch_fwd_packed(int d, bool bf16, const CUtensorMap &tq, const CUtensorMap &tk,
                              const CUtensorMap &tv, const PackArgs &a, cudaStream_t stream) {
    return launch_pack<false>(d, bf16, tq, tk, tv, a, stream);
}

}  // namespace exattn
