// norm_launch.h -- internal interface between norm.cu and the translation
// units that instantiate the norm kernels for one pair of types each.
#pragma once
#include <cuda_runtime.h>

#include "norm_kern.cuh"

namespace gemm103 {
namespace nrm {

struct Launch {
    Params p;
    int grid, threads;          // threads per CTA: a multiple of p.T
    int chunks8;                // C: chunks of 8 elements per thread (1 or 2)
    bool bias;                  // backward: the sums of dY and q are wanted
    size_t smem;
    cudaStream_t stream;
};

// Types of (X, Z): 0 = F16, 1 = BF16, 2 = F32, as gemm_dtype_t.
cudaError_t forward_f16_f16(const Launch& l);
cudaError_t forward_bf16_bf16(const Launch& l);
cudaError_t forward_f32_f32(const Launch& l);
cudaError_t forward_f32_f16(const Launch& l);
cudaError_t forward_f32_bf16(const Launch& l);
cudaError_t backward_f16_f16(const Launch& l);
cudaError_t backward_bf16_bf16(const Launch& l);
cudaError_t backward_f32_f32(const Launch& l);
cudaError_t backward_f32_f16(const Launch& l);
cudaError_t backward_f32_bf16(const Launch& l);

}  // namespace nrm
}  // namespace gemm103
