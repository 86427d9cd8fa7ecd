// device_limits.h -- what the launchers set or look up once: per device, as the
// runtime's function attributes are.
#pragma once
#include <cstddef>
#include <mutex>

#include <cuda_runtime.h>

namespace gemm103 {

constexpr int kMaxDevices = 64;

// A value of each device, zero at first.
template <typename T>
class PerDevice {
public:
    // The current device's; NULL beyond kMaxDevices.
    T* current() {
        int dev = -1;
        if (cudaGetDevice(&dev) != cudaSuccess) cudaGetLastError();
        return dev >= 0 && dev < kMaxDevices ? &v_[dev] : nullptr;
    }

private:
    T v_[kMaxDevices] = {};
};

// A kernel's dynamic shared-memory limit: raised on a device only when a launch
// needs more than that device has been given (a host call worth avoiding on every
// launch of a kernel of microseconds).
class DeviceLimits {
public:
    // Runs set() where `bytes` is above the current device's limit; its status.
    template <typename Set>
    cudaError_t raise(size_t bytes, Set set) {
        std::lock_guard<std::mutex> g(mu_);
        size_t* to = to_.current();
        if (to != nullptr && bytes <= *to) return cudaSuccess;
        const cudaError_t e = set();
        if (e == cudaSuccess && to != nullptr) *to = bytes;
        return e;
    }

private:
    std::mutex mu_;
    PerDevice<size_t> to_;
};

}  // namespace gemm103
