// ortho_launch.h -- internal interface between the orthogonalised update's entry
// point (api.cu, which owns the handle) and its kernels (ortho.cu).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "ortho_sm103.h"

namespace gemm103 {

struct OrthoCall {
    int64_t batch, rows, cols;
    const void* G;
    int64_t ldg, stride_g;
    int32_t g_dtype;
    void* O;
    int64_t ldo, stride_o;
    const ortho_update_t* opt;
    // of the handle
    decltype(&cuTensorMapEncodeTiled) encode;
    uint8_t* ws;                       // behind the counters
    int sms;
    int* err;
    uint64_t wait_limit_ns;
    uint32_t debug_flags;
    cudaStream_t stream;
};

int64_t ortho_bytes(int64_t batch, int64_t rows, int64_t cols);
gemm_status_t ortho_enqueue(const OrthoCall& c);

}  // namespace gemm103
