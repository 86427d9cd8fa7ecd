// workspace.h -- the device buffer behind a handle, and those it has outgrown.
#pragma once
#include <cstddef>
#include <new>

#include <cuda_runtime.h>

namespace gemm103 {

// A buffer that grows on demand.  It begins with `header` bytes of tile counters,
// zero when it is made and zero again after every call that uses it.  A buffer
// that a captured graph may still address, and any buffer outgrown under capture,
// where nothing can wait for its users, is kept until release().
class Workspace {
public:
    explicit Workspace(size_t header) : header_(header) {}
    void* data() const { return p_; }
    size_t bytes() const { return bytes_; }

    // At least `bytes` for a call on `stream`; false: out of memory.
    bool reserve(size_t bytes, cudaStream_t stream) {
        if (bytes == 0) return true;
        cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
        if (cudaStreamIsCapturing(stream, &cap) != cudaSuccess) cudaGetLastError();
        const bool capturing = cap != cudaStreamCaptureStatusNone;
        if (bytes <= bytes_) {
            captured_ = captured_ || capturing;
            return true;
        }
        const Relaxed relaxed;
        if (p_ != nullptr && (captured_ || capturing)) {
            Retired* r = new (std::nothrow) Retired;
            if (r == nullptr) return false;
            r->p = p_;
            r->next = retired_;
            retired_ = r;
        } else if (p_ != nullptr) {
            cudaFree(p_);         // implicit device synchronisation: no user of the old buffer remains
        }
        bytes_ = 0;
        captured_ = capturing;
        const size_t some = bytes + (bytes >> 2), want = some > header_ ? some : header_;
        p_ = make(want);
        if (p_ == nullptr) return false;
        bytes_ = want;
        return true;
    }

    // After a kernel gave up: waits for the device and clears the counters.  False
    // where it cannot, as while a stream is captured: to be tried again.
    bool recover() {
        if (cudaDeviceSynchronize() != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        return clear_counters();
    }

    // Zeroes the counters of every buffer, the outgrown ones too, once nothing
    // runs on them: a kernel that gave up may have left them half-counted, in the
    // buffer that its graph was captured with.
    bool clear_counters() {
        const Relaxed relaxed;
        bool ok = p_ == nullptr || zero(p_);
        for (Retired* r = retired_; r != nullptr; r = r->next) ok = zero(r->p) && ok;
        return ok;
    }

    void release() {
        if (p_ != nullptr) cudaFree(p_);
        p_ = nullptr;
        bytes_ = 0;
        while (retired_ != nullptr) {
            Retired* r = retired_;
            retired_ = r->next;
            cudaFree(r->p);
            delete r;
        }
    }

private:
    struct Retired {
        void* p;
        Retired* next;
    };

    // Calls that a capture under way, this thread's or another's, would forbid:
    // the graph does not hold what they do.
    struct Relaxed {
        cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
        Relaxed() { cudaThreadExchangeStreamCaptureMode(&mode); }
        ~Relaxed() { cudaThreadExchangeStreamCaptureMode(&mode); }
    };

    // The counters at p as zero before it returns: on a stream of its own (cudaMemset
    // would return early, on the legacy stream, which non-blocking streams do not
    // wait for).
    bool zero(void* p) const {
        cudaStream_t s;
        cudaError_t e = cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking);
        if (e == cudaSuccess) {
            e = cudaMemsetAsync(p, 0, header_, s);
            if (e == cudaSuccess) e = cudaStreamSynchronize(s);
            cudaStreamDestroy(s);
        }
        if (e != cudaSuccess) cudaGetLastError();
        return e == cudaSuccess;
    }

    // A buffer of `want` bytes whose counters are zero.
    void* make(size_t want) const {
        void* p = nullptr;
        if (cudaMalloc(&p, want) != cudaSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        if (zero(p)) return p;
        cudaFree(p);
        return nullptr;
    }

    size_t header_;
    void* p_ = nullptr;
    size_t bytes_ = 0;
    bool captured_ = false;       // a captured graph may hold p_'s address
    Retired* retired_ = nullptr;  // outgrown
};

}  // namespace gemm103
