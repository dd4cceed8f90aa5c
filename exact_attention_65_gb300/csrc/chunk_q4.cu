// The new tokens of each request over a cache held in 4 bits
// (attn_chunk_paged_q4): the packed forward's two-tile form with warps that
// widen K and V (fwd_packed.cuh).
#include "fwd_packed.cuh"

namespace exattn {
namespace {

template <int D>
cudaError_t launch_q4(bool bf16, const CUtensorMap &tq, const PackArgs &a, cudaStream_t stream) {
    return bf16 ? launch_pack_t<D, true, true, false, true>(tq, tq, tq, a, stream)
                : launch_pack_t<D, false, true, false, true>(tq, tq, tq, a, stream);
}

}  // namespace

cudaError_t launch_chunk_q4(int d, bool bf16, const CUtensorMap &tq, const PackArgs &a, cudaStream_t stream) {
    switch (d) {
        case 16: return launch_q4<16>(bf16, tq, a, stream);
        case 32: return launch_q4<32>(bf16, tq, a, stream);
        case 64: return launch_q4<64>(bf16, tq, a, stream);
        case 128: return launch_q4<128>(bf16, tq, a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace exattn
