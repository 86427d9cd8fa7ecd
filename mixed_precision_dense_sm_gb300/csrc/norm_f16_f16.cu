// norm_f16_f16.cu -- norm kernels, residual stream and block types f16_f16.
#define NORM_XT __half
#define NORM_ZT __half
#define NORM_SUFFIX f16_f16
#include "norm_inst.cuh"
