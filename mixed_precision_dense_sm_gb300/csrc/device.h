// device.h -- what the handle-less entry points ask of the current device.
#pragma once
#include <cuda_runtime.h>

namespace gemm103 {

// SMs of the current device; 0 if it is not sm_103, -1 on a CUDA error.
inline int device_sms() {
    int dev = 0, major = 0, minor = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return -1;
    }
    return major == 10 && minor == 3 ? sms : 0;
}

}  // namespace gemm103
