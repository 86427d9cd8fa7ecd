// norm_bf16_bf16.cu -- norm kernels, residual stream and block types bf16_bf16.
#define NORM_XT __nv_bfloat16
#define NORM_ZT __nv_bfloat16
#define NORM_SUFFIX bf16_bf16
#include "norm_inst.cuh"
