// norm_f32_bf16.cu -- norm kernels, residual stream and block types f32_bf16.
#define NORM_XT float
#define NORM_ZT __nv_bfloat16
#define NORM_SUFFIX f32_bf16
#include "norm_inst.cuh"
