// norm_inst.cuh -- instantiates the norm kernels for one pair of types
// (NORM_XT, NORM_ZT) behind plain launchers.
#pragma once
#include "device_limits.h"
#include "norm_launch.h"

#define NORM_CAT2(a, b) a##b
#define NORM_CAT(a, b) NORM_CAT2(a, b)

namespace gemm103 {
namespace nrm {

template <typename K>
static cudaError_t launch_kernel(K kern, const Launch& l, DeviceLimits& limit) {
    const cudaError_t e = limit.raise(l.smem, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(l.smem));
    });
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(l.grid, 1, 1);
    cfg.blockDim = dim3(l.threads, 1, 1);
    cfg.dynamicSmemBytes = l.smem;
    cfg.stream = l.stream;
    cfg.attrs = attr;
    cfg.numAttrs = l.p.cluster == 2 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, l.p);
}

template <int TT, int C, bool VEC, int KIND>
static cudaError_t forward_c(const Launch& l) {
    static DeviceLimits limit;
    return launch_kernel(forward_kernel<NORM_XT, NORM_ZT, TT, C, VEC, KIND>, l, limit);
}

template <int TT, int C, bool VEC, bool BIAS, int KIND>
static cudaError_t backward_c(const Launch& l) {
    static DeviceLimits limit;
    return launch_kernel(backward_kernel<NORM_XT, NORM_ZT, TT, C, VEC, BIAS, KIND>, l, limit);
}

// Threads per row and chunks per thread: one chunk for rows of up to 256
// columns (a warp each) and for few rows (norm.cu), else two.  Rows of vectors
// have the threads compiled in; the others share a kernel per C.
template <int KIND>
static cudaError_t forward_k(const Launch& l) {
    if (!l.p.vec) return l.chunks8 == 1 ? forward_c<0, 1, false, KIND>(l) : forward_c<0, 2, false, KIND>(l);
    if (l.chunks8 == 1) {
        return l.p.T == 32    ? forward_c<32, 1, true, KIND>(l)
               : l.p.T == 512 ? forward_c<512, 1, true, KIND>(l)
                              : forward_c<0, 1, true, KIND>(l);
    }
    switch (l.p.T) {
        case 32: return forward_c<32, 2, true, KIND>(l);
        case 64: return forward_c<64, 2, true, KIND>(l);
        case 128: return forward_c<128, 2, true, KIND>(l);
        case 256: return forward_c<256, 2, true, KIND>(l);
        case 384: return forward_c<384, 2, true, KIND>(l);
        case 512: return forward_c<512, 2, true, KIND>(l);
        default: return cudaErrorInvalidValue;
    }
}

// The kinds that are compiled in: RMSNorm without biases, LayerNorm with them,
// each with the same norm behind the block or none.
cudaError_t NORM_CAT(forward_, NORM_SUFFIX)(const Launch& l) {
    const Params& p = l.p;
    if (p.Z && p.Y && !p.token_gate) {
        const bool bs = p.i_bs >= 0, bpre = p.i_bpre >= 0;
        if (!bs && !bpre && p.pre == kRms && p.post == kRms) return forward_k<kRmsRms>(l);
        if (!bs && !bpre && p.pre == kRms && p.post == kNone) return forward_k<kRmsPlain>(l);
        if (bs && bpre && p.pre == kLayer && p.post == kLayer) return forward_k<kLayerLayer>(l);
        if (!bs && bpre && p.pre == kLayer && p.post == kNone) return forward_k<kLayerPlain>(l);
    }
    return forward_k<kAnyKind>(l);
}

template <bool BIAS, int KIND>
static cudaError_t backward_k(const Launch& l) {
    if (!l.p.vec) return backward_c<0, 1, false, BIAS, KIND>(l);
    if (l.chunks8 == 1) return backward_c<32, 1, true, BIAS, KIND>(l);
    switch (l.p.T) {
        case 32: return backward_c<32, 2, true, BIAS, KIND>(l);
        case 64: return backward_c<64, 2, true, BIAS, KIND>(l);
        case 128: return backward_c<128, 2, true, BIAS, KIND>(l);
        case 256: return backward_c<256, 2, true, BIAS, KIND>(l);
        case 384: return backward_c<384, 2, true, BIAS, KIND>(l);
        case 512: return backward_c<512, 2, true, BIAS, KIND>(l);
        default: return cudaErrorInvalidValue;
    }
}

// The same kinds (the biases' gradients standing for the biases).  Rows that
// are not vectors and take two chunks per thread run the kernel with all four sums (fewer
// kernels; the two that are not wanted are not added up).
cudaError_t NORM_CAT(backward_, NORM_SUFFIX)(const Launch& l) {
    const Params& p = l.p;
    if (!p.vec && l.chunks8 == 2) return backward_c<0, 2, false, true, kAnyKind>(l);
    if (p.Z && p.dY && p.dXO && p.dX && p.dZ && !p.token_gate) {
        if (!l.bias && p.pre == kRms && p.post == kRms) return backward_k<false, kRmsRms>(l);
        if (!l.bias && p.pre == kRms && p.post == kNone) return backward_k<false, kRmsPlain>(l);
        if (l.bias && p.pre == kLayer && p.post == kLayer) return backward_k<true, kLayerLayer>(l);
        if (l.bias && p.pre == kLayer && p.post == kNone) return backward_k<true, kLayerPlain>(l);
    }
    return l.bias ? backward_k<true, kAnyKind>(l) : backward_k<false, kAnyKind>(l);
}

}  // namespace nrm
}  // namespace gemm103
