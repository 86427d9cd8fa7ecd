// kern_glu_f16.cu -- gated linear layer, f16 output.
#define KERN_OUT_T __half
#define KERN_SUFFIX f16
#define KERN_ES 2
#define KERN_GLU
#include "kern_inst.cuh"
