// The new tokens of each request over a cache held in 4 bits
// (attn_chunk_paged_q4): the packed forward's two-tile form with warps that
// widen K and V (fwd_packed.cuh).
#include "fwd_packed.cuh"

namespace exattn {
namespace {

template <int D, bool BF16>
cudaError_t launch_t(const CUtensorMap &tq, const PackArgs &a, bool early, cudaStream_t stream) {
    using G = PackGeom<D, false>;
    const auto kernel = pack_kernel<D, BF16, true, false, true>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && !attr_set[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    // Behind the few-row kernel, whose sequences are others: CTAs start where its
    // have finished, and wait for the rest of it at their end only.
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.ctas));
    cfg.blockDim = dim3(PackThreads<true>::COUNT);
    cfg.dynamicSmemBytes = G::SMEM_BYTES;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, tq, tq, tq, a);
}

template <int D>
cudaError_t launch_d(bool bf16, const CUtensorMap &tq, const PackArgs &a, bool early, cudaStream_t stream) {
    return bf16 ? launch_t<D, true>(tq, a, early, stream) : launch_t<D, false>(tq, a, early, stream);
}

}  // namespace

cudaError_t launch_chunk_q4(int d, bool bf16, const CUtensorMap &tq, const PackArgs &a, bool early,
                            cudaStream_t stream) {
    switch (d) {
        case 16: return launch_d<16>(bf16, tq, a, early, stream);
        case 32: return launch_d<32>(bf16, tq, a, early, stream);
        case 64: return launch_d<64>(bf16, tq, a, early, stream);
        case 128: return launch_d<128>(bf16, tq, a, early, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace exattn
