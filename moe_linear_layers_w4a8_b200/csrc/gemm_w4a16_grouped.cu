// Instantiations and launch of the grouped W4A16 GEMM kernels.
#include <atomic>
#include <cuda_runtime.h>

#include "gemm_w4a16_grouped.cuh"

namespace w4a8 {

template <int BN, bool SYM>
static int launch_w4a16_grouped_t(const CUtensorMap (&tmap_x)[3], const CUtensorMap& tmap_s,
                                  const CUtensorMap& tmap_z, const W16GroupedParams& p, int grid, cudaStream_t stream) {
    using C = W16GCfg<BN>;
    auto kern = w4a16_grouped_kernel<BN, SYM>;
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
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, tmap_x[0], tmap_x[1], tmap_x[2], tmap_s, tmap_z, p) != cudaSuccess) return 6;
    return cudaGetLastError() == cudaSuccess ? 0 : 6;
}

int launch_w4a16_grouped(int bn, bool sym, const CUtensorMap (&tx)[3], const CUtensorMap& ts, const CUtensorMap& tz,
                         const W16GroupedParams& p, int grid, cudaStream_t stream) {
#define W4A8_W16G(B)                                                                   \
    case B:                                                                            \
        return sym ? launch_w4a16_grouped_t<B, true>(tx, ts, tz, p, grid, stream)      \
                   : launch_w4a16_grouped_t<B, false>(tx, ts, tz, p, grid, stream);
    switch (bn) {
        W4A8_W16G(16) W4A8_W16G(32) W4A8_W16G(64) W4A8_W16G(128) W4A8_W16G(192)
    }
#undef W4A8_W16G
    return 2;
}

}  // namespace w4a8
