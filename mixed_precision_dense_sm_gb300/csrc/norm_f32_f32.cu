// norm_f32_f32.cu -- norm kernels, residual stream and block types f32_f32.
#define NORM_XT float
#define NORM_ZT float
#define NORM_SUFFIX f32_f32
#include "norm_inst.cuh"
