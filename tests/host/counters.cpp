// The counters are zero when reserve() and clear_counters() return: the streams
// of the calls that use them need not wait for the legacy stream.
#include <cstdio>

#include "workspace.h"

static bool zero(const void* p, size_t n) {
    for (size_t i = 0; i < n; ++i)
        if (static_cast<const unsigned char*>(p)[i] != 0) return false;
    return true;
}
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
    constexpr size_t kHeader = 64;
    gemm103::Workspace w(kHeader);
    cudaStream_t s;
    cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking);
    CHECK(w.reserve(1000, s) && zero(w.data(), kHeader));
    CHECK(w.reserve(10000, s) && zero(w.data(), kHeader));
    std::memset(w.data(), 1, kHeader);
    CHECK(w.clear_counters() && zero(w.data(), kHeader));
    CHECK(fake::mode == cudaStreamCaptureModeGlobal);
    // a capture under way on another thread's stream forbids neither
    cudaStream_t other;
    cudaStreamCreateWithFlags(&other, cudaStreamNonBlocking);
    other->capturing = true;
    CHECK(w.reserve(100000, s) && zero(w.data(), kHeader));
    std::memset(w.data(), 1, kHeader);
    CHECK(w.clear_counters() && zero(w.data(), kHeader));
    CHECK(fake::mode == cudaStreamCaptureModeGlobal && fake::streams.size() == 3);
    w.release();
    CHECK(fake::memory.empty());
    return 0;
}
