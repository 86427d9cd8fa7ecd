// Recovery from a kernel that gave up: done once the device has been waited for,
// which a capture under way prevents; then it is to be tried again.
#include <cstdio>

#include "workspace.h"

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
    constexpr size_t kHeader = 64;
    gemm103::Workspace w(kHeader);
    CHECK(w.recover());                                       // nothing to clear
    cudaStream_t s;
    cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking);
    CHECK(w.reserve(1000, s));
    unsigned char* p = static_cast<unsigned char*>(w.data());
    // the last kernel on the buffer, still running, counts on
    s->queue.push_back([=] { p[5] = 7; });
    s->capturing = true;
    CHECK(!w.recover());
    CHECK(fake::mode == cudaStreamCaptureModeGlobal);
    s->capturing = false;
    CHECK(w.recover() && p[5] == 0 && s->queue.empty());
    w.release();
    return 0;
}
