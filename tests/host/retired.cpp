// After a kernel gave up, the counters of every buffer are cleared: also of those
// that captured graphs still address.
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
    CHECK(w.reserve(0, s) && w.data() == nullptr);
    CHECK(w.reserve(1000, s) && w.bytes() >= 1000);
    void* eager = w.data();
    CHECK(w.reserve(1100, s) && w.data() == eager);           // it has room to spare
    s->capturing = true;
    CHECK(w.reserve(900, s) && w.data() == eager);            // a graph holds it from here on
    CHECK(w.reserve(5000, s));
    void* first = w.data();
    CHECK(first != eager && zero(first, kHeader));
    s->capturing = false;
    CHECK(w.reserve(50000, s));
    void* second = w.data();
    CHECK(second != first && fake::memory.size() == 3);       // both are still in graphs
    for (void* p : {eager, first, second}) std::memset(p, 1, kHeader);
    std::memset(static_cast<char*>(first) + kHeader, 2, 8);
    cudaDeviceSynchronize();
    CHECK(w.clear_counters());
    cudaDeviceSynchronize();
    for (void* p : {eager, first, second}) CHECK(zero(p, kHeader));
    CHECK(static_cast<char*>(first)[kHeader] == 2);
    CHECK(w.reserve(500000, s) && fake::memory.size() == 3);  // `second` was in no graph: freed
    fake::fail_alloc = true;
    CHECK(!w.reserve(5000000, s) && w.data() == nullptr);
    fake::fail_alloc = false;
    CHECK(w.reserve(10, s));
    w.release();
    CHECK(fake::memory.empty() && w.data() == nullptr);
    return 0;
}
