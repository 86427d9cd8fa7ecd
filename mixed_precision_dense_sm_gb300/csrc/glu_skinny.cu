// glu_skinny.cu -- instances of the weight-streaming gated layer.
#include "device_limits.h"
#include "launch.h"

namespace gemm103 {

template <int BN, int KC>
static cudaError_t launch(const GluSkinnyLaunch& l) {
    auto kern = glu_skinny_kernel<BN, KC>;
    static DeviceLimits limit;
    const cudaError_t set = limit.raise(Skinny<BN, KC>::kSmem, [&] {
        // room for two CTAs per SM
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                                                   cudaSharedmemCarveoutMaxShared);
        return e != cudaSuccess ? e
                                : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       static_cast<int>(Skinny<BN, KC>::kSmem));
    });
    if (set != cudaSuccess) return set;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(l.p.splits);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(l.grid, 1, 1);
    cfg.blockDim = dim3(kSkinnyThreads, 1, 1);
    cfg.dynamicSmemBytes = Skinny<BN, KC>::kSmem;
    cfg.stream = l.stream;
    cfg.attrs = attr;
    cfg.numAttrs = l.p.splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, l.tmW, l.tmX, l.p);
}

cudaError_t launch_glu_skinny(const GluSkinnyLaunch& l) {
    if (l.kc == 1) {
        switch (l.block_n) {
            case 16: return launch<16, 1>(l);
            case 32: return launch<32, 1>(l);
            case 64: return launch<64, 1>(l);
            case 128: return launch<128, 1>(l);
        }
    } else {
        switch (l.block_n) {
            case 16: return launch<16, 2>(l);
            case 32: return launch<32, 2>(l);
            case 64: return launch<64, 2>(l);
        }
    }
    return cudaErrorInvalidValue;
}

}  // namespace gemm103
