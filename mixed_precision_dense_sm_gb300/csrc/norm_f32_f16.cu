// norm_f32_f16.cu -- norm kernels, residual stream and block types f32_f16.
#define NORM_XT float
#define NORM_ZT __half
#define NORM_SUFFIX f32_f16
#include "norm_inst.cuh"
