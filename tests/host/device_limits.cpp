// What a kernel is given once is given once per device.
#include <cstdio>
#include <thread>
#include <vector>

#include "device_limits.h"

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
    gemm103::DeviceLimits l;
    int calls = 0;
    auto set = [&]() -> cudaError_t { ++calls; return cudaSuccess; };
    CHECK(l.raise(50000, set) == cudaSuccess && calls == 1);
    CHECK(l.raise(50000, set) == cudaSuccess && l.raise(40000, set) == cudaSuccess && calls == 1);
    CHECK(l.raise(60000, set) == cudaSuccess && calls == 2);
    fake::device = 1;                                          // it knows nothing of this yet
    CHECK(l.raise(50000, set) == cudaSuccess && calls == 3);
    CHECK(l.raise(50000, set) == cudaSuccess && calls == 3);
    fake::device = 0;
    CHECK(l.raise(60000, set) == cudaSuccess && calls == 3);
    // a failure is not remembered as done
    fake::device = 2;
    CHECK(l.raise(50000, [&]() -> cudaError_t { return cudaErrorInvalidValue; }) == cudaErrorInvalidValue);
    CHECK(l.raise(50000, set) == cudaSuccess && calls == 4);
    // devices beyond the table: every time
    fake::device = gemm103::kMaxDevices;
    CHECK(l.raise(50000, set) == cudaSuccess && l.raise(50000, set) == cudaSuccess && calls == 6);
    fake::device = 3;
    int n = 0;                                                 // (set() runs under the lock)
    std::vector<std::thread> ts;
    for (int i = 0; i < 8; ++i)
        ts.emplace_back([&] { for (int k = 0; k < 1000; ++k) l.raise(100, [&]() -> cudaError_t { ++n; return cudaSuccess; }); });
    for (auto& t : ts) t.join();
    CHECK(n == 1);

    gemm103::PerDevice<int> v;
    fake::device = 0;
    CHECK(v.current() != nullptr && *v.current() == 0);
    *v.current() = 5;
    fake::device = 1;
    CHECK(*v.current() == 0);
    fake::device = 0;
    CHECK(*v.current() == 5);
    fake::device = gemm103::kMaxDevices;
    CHECK(v.current() == nullptr);
    return 0;
}
