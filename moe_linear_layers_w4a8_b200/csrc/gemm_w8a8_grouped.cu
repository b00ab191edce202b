// Instantiations and launch of the grouped W8A8 GEMM kernel.
#include <atomic>
#include <cuda_runtime.h>

#include "gemm_w8a8_grouped.cuh"

namespace w4a8 {

template <int BN, bool GATEUP>
static int launch_w8a8_grouped_t(const CUtensorMap& tmap_w, const CUtensorMap& tmap_x, const W8GroupedParams& p,
                                 int grid, cudaStream_t stream) {
    using C = W8GCfg<BN>;
    auto kern = w8a8_grouped_kernel<BN, GATEUP>;
    static std::atomic<uint64_t> attr_done{0};
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    if (!(attr_done.load() & bit)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
            return 6;
        attr_done.fetch_or(bit);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kW8GThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, tmap_w, tmap_x, p) != cudaSuccess) return 6;
    return cudaGetLastError() == cudaSuccess ? 0 : 6;
}

int launch_w8a8_grouped(int bn, bool gate_up, const CUtensorMap& tmap_w, const CUtensorMap& tmap_x,
                        const W8GroupedParams& p, int grid, cudaStream_t stream) {
#define W4A8_W8G(B)                                                                              \
    case B:                                                                                      \
        return gate_up ? launch_w8a8_grouped_t<B, true>(tmap_w, tmap_x, p, grid, stream)         \
                       : launch_w8a8_grouped_t<B, false>(tmap_w, tmap_x, p, grid, stream);
    switch (bn) {
        W4A8_W8G(16) W4A8_W8G(32) W4A8_W8G(64) W4A8_W8G(128)
    }
#undef W4A8_W8G
    return 2;
}

}  // namespace w4a8
