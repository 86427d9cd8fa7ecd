// kern_glu_f32.cu -- gated linear layer, f32 output.
#define KERN_OUT_T float
#define KERN_SUFFIX f32
#define KERN_ES 2
#define KERN_GLU
#include "kern_inst.cuh"
