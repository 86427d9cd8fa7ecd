// A stand-in for the CUDA runtime on the host: what the library's host-only parts
// call of it, on host memory.  Work that the real runtime only enqueues is
// enqueued here, and done when something waits for it, so a missing wait shows.
#pragma once
#include <cstddef>
#include <cstdlib>
#include <cstring>
#include <deque>
#include <functional>
#include <map>
#include <set>

typedef int cudaError_t;
constexpr cudaError_t cudaSuccess = 0, cudaErrorInvalidValue = 1, cudaErrorMemoryAllocation = 2,
                      cudaErrorStreamCaptureUnsupported = 900;
typedef struct FakeStream* cudaStream_t;
enum cudaStreamCaptureStatus { cudaStreamCaptureStatusNone, cudaStreamCaptureStatusActive };
enum cudaStreamCaptureMode { cudaStreamCaptureModeGlobal, cudaStreamCaptureModeThreadLocal, cudaStreamCaptureModeRelaxed };
constexpr unsigned cudaStreamNonBlocking = 1;

struct FakeStream {
    std::deque<std::function<void()>> queue;
    bool capturing = false;
};

namespace fake {
inline FakeStream legacy;
inline std::set<FakeStream*> streams{&legacy};
inline std::map<void*, size_t> memory;
inline cudaStreamCaptureMode mode = cudaStreamCaptureModeGlobal;
inline int device = 0, devices = 1;
inline bool fail_alloc = false;

inline FakeStream* of(cudaStream_t s) { return s ? s : &legacy; }
inline void drain(FakeStream* s) {
    while (!s->queue.empty()) {
        s->queue.front()();
        s->queue.pop_front();
    }
}
inline void drain_all() {
    for (FakeStream* s : streams) drain(s);
}
inline bool any_capture() {
    for (FakeStream* s : streams)
        if (s->capturing) return true;
    return false;
}
// Calls that a capture under way forbids unless the thread is in relaxed mode.
inline bool unsafe() { return any_capture() && mode != cudaStreamCaptureModeRelaxed; }
}  // namespace fake

inline cudaError_t cudaGetLastError() { return cudaSuccess; }
inline cudaError_t cudaGetDevice(int* d) { *d = fake::device; return cudaSuccess; }
inline cudaError_t cudaStreamIsCapturing(cudaStream_t s, cudaStreamCaptureStatus* st) {
    *st = fake::of(s)->capturing ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
    return cudaSuccess;
}
inline cudaError_t cudaThreadExchangeStreamCaptureMode(cudaStreamCaptureMode* m) {
    const cudaStreamCaptureMode old = fake::mode;
    fake::mode = *m;
    *m = old;
    return cudaSuccess;
}
inline cudaError_t cudaMalloc(void** p, size_t n) {
    if (fake::unsafe()) return cudaErrorStreamCaptureUnsupported;
    if (fake::fail_alloc) return cudaErrorMemoryAllocation;
    *p = std::malloc(n);
    std::memset(*p, 0xA5, n);                 // what was there before
    fake::memory[*p] = n;
    return cudaSuccess;
}
// (waits for the device, as the real one does)
inline cudaError_t cudaFree(void* p) {
    if (fake::memory.erase(p) != 1) std::abort();
    fake::drain_all();
    std::free(p);
    return cudaSuccess;
}
inline cudaError_t cudaMemsetAsync(void* p, int v, size_t n, cudaStream_t s) {
    if (fake::memory.count(p) != 1 || n > fake::memory[p]) return cudaErrorInvalidValue;
    if (s == nullptr && fake::any_capture()) return cudaErrorStreamCaptureUnsupported;
    fake::of(s)->queue.push_back([=] { std::memset(p, v, n); });
    return cudaSuccess;
}
// Device memory: asynchronous, on the legacy stream, which non-blocking streams do not wait for.
inline cudaError_t cudaMemset(void* p, int v, size_t n) { return cudaMemsetAsync(p, v, n, nullptr); }
inline cudaError_t cudaStreamCreateWithFlags(cudaStream_t* s, unsigned) {
    *s = new FakeStream;
    fake::streams.insert(*s);
    return cudaSuccess;
}
inline cudaError_t cudaStreamDestroy(cudaStream_t s) {
    fake::drain(s);
    fake::streams.erase(s);
    delete s;
    return cudaSuccess;
}
inline cudaError_t cudaStreamSynchronize(cudaStream_t s) {
    if (fake::of(s)->capturing) return cudaErrorStreamCaptureUnsupported;
    fake::drain(fake::of(s));
    return cudaSuccess;
}
inline cudaError_t cudaDeviceSynchronize() {
    if (fake::any_capture()) return cudaErrorStreamCaptureUnsupported;
    fake::drain_all();
    return cudaSuccess;
}
