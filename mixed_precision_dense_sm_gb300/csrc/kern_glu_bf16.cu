// kern_glu_bf16.cu -- gated linear layer, bf16 output.
#define KERN_OUT_T __nv_bfloat16
#define KERN_SUFFIX bf16
#define KERN_ES 2
#define KERN_GLU
#include "kern_inst.cuh"
