// grad.cu -- the global gradient norm over many tensors, and clipping by it
// (include/grad_sm103.h).
//
// Two kernels.  norm_partial_kernel reads every element once: the tensors are
// cut into chunks of 8192 or 16384 elements, numbered through all of a launch's
// tensors, and CTA b takes chunks b, b + grid, ...; each CTA leaves one FP64
// partial sum.  apply_kernel adds the partial sums (every CTA the same way:
// a few hundred FP64 values out of L2, cheaper than a third launch or a
// grid-wide wait), CTA 0 writes the norm, and each CTA scales its chunks.  The
// second pass walks the chunks in the opposite order, each SM those it had in
// the first (the grids are multiples of the SMs), and what the first pass read
// last it marked to stay in L2 (kKeepBytes).  Bound by HBM: two reads and one write of the
// gradients (one read where nothing is scaled in place, or where they fit in
// L2).  120M bf16 elements: 115 us; three passes over them at copy speed are 106.
//
// Squares are summed in FP32 over one batch of a thread (kVecs 16-byte
// vectors: 16 or 32 elements) and then in FP64: one FP64 add per batch, as
// FP64 arithmetic is scarce here.  A batch whose FP32 sum lies in
// [2^-90, 2^127) lost at most 32 squares below 2^-126 -- under 2^-31 of it --
// so it is kept; any other batch that is not all zeros is summed again in
// FP64, where the square of no FP32, BF16 or FP16 value overflows or
// underflows.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "device.h"
#include "f32x2.cuh"
#include "grad_sm103.h"
#include "ptx.cuh"

namespace {

using namespace gemm103;

constexpr int kThreads = 256;
constexpr int kSumCtas = 6;                    // per SM, all resident at once
constexpr int kApplyCtas = 3;                  // (4 would spill: 122 against 112 us for 120M bf16)
constexpr int kVecs = 4;                       // 16-byte vectors per thread and batch
// Elements per chunk; the smaller where the larger would give an SM fewer than
// four (60 FP32 tensors of 900k elements in all: 14.5 us by 16384, 12.4 by
// 8192, 18.6 by 2048).
constexpr int32_t kMostChunk = 16384, kLeastChunk = 8192;
// About this much of what is read last is kept in L2 for the second pass, the
// rest makes room for it (0 to 100 MB measured: 115, 112, 115 us at 0, 64, 96 MB).
constexpr int64_t kKeepBytes = 64 << 20;
constexpr int kPerLaunch = GRAD_TENSORS_PER_LAUNCH;

template <int CAP>
struct Tensors {
    const void* src[CAP];
    void* dst[CAP];
    int64_t size[CAP];
    int32_t first_chunk[CAP + 1];              // chunks before tensor t; [count] = all
    uint8_t dtype[CAP];
    int32_t count;
    int32_t chunk;                             // elements per chunk
};

struct ApplyParams {
    const double* partials;
    int32_t num_partials;
    float max_norm, inv_scale;
    float* norm;
    int32_t write_norm;
};

// Tensor that holds chunk `c` (the last t with first_chunk[t] <= c).
template <int CAP>
__device__ __forceinline__ int find_tensor(const Tensors<CAP>& t, int32_t c) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first_chunk[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <typename T>
union Vec16 {
    uint4 u;
    T e[16 / sizeof(T)];
};

// A batch again in FP64, from memory: rare, and out of line so that it costs
// the fast path no registers.
template <typename T>
__device__ __noinline__ double batch_again(const uint4* v, int32_t i, int32_t nvec) {
    double d = 0.0;
    for (int q = 0; q < kVecs; ++q) {
        const int32_t k = i + q * kThreads;
        if (k >= nvec) break;
        Vec16<T> w;
        w.u = v[k];
        #pragma unroll
        for (int e = 0; e < static_cast<int>(16 / sizeof(T)); ++e) {
            const double x = static_cast<double>(to_f<T>(w.e[e]));
            d = fma(x, x, d);
        }
    }
    return d;
}

// The sum of squares of a batch (see above): vectors i, i + kThreads, ... of v.
template <typename T>
__device__ __forceinline__ double batch_sum(const uint4 (&r)[kVecs], const uint4* v, int32_t i,
                                            int32_t nvec) {
    constexpr int kPer = 16 / sizeof(T);
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    #pragma unroll
    for (int q = 0; q < kVecs; ++q) {
        Vec16<T> w;
        w.u = r[q];
        #pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const float x = to_f<T>(w.e[e]);
            s[e & 3] = fmaf(x, x, s[e & 3]);
        }
    }
    const float t = (s[0] + s[1]) + (s[2] + s[3]);
    if (t >= 0x1p-90f && t < 0x1p127f) return static_cast<double>(t);
    uint32_t any = 0;
    #pragma unroll
    for (int q = 0; q < kVecs; ++q) any |= r[q].x | r[q].y | r[q].z | r[q].w;
    return any == 0 ? 0.0 : batch_again<T>(v, i, nvec);
}

// Elements of a chunk before its first 16-byte boundary (at most n).
template <typename T>
__device__ __forceinline__ int32_t head_of(const T* p, int32_t n) {
    const int32_t h = static_cast<int32_t>(((16u - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) /
                                           sizeof(T));
    return h < n ? h : n;
}

// 16 bytes with an L2 policy.
__device__ __forceinline__ uint4 load_hint(const uint4* p, uint64_t policy) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p), "l"(policy));
    return r;
}

template <typename T>
__device__ __forceinline__ double chunk_sum(const T* p, int32_t n, uint64_t policy) {
    constexpr int kPer = 16 / sizeof(T);
    const int32_t head = head_of(p, n);
    const int32_t nvec = (n - head) / kPer;
    const uint4* v = reinterpret_cast<const uint4*>(p + head);
    double acc = 0.0;
    for (int32_t i = threadIdx.x; i < nvec; i += kVecs * kThreads) {
        uint4 r[kVecs];
        #pragma unroll
        for (int q = 0; q < kVecs; ++q) {
            const int32_t k = i + q * kThreads;
            r[q] = k < nvec ? load_hint(v + k, policy) : make_uint4(0u, 0u, 0u, 0u);
        }
        acc += batch_sum<T>(r, v, i, nvec);
    }
    // the elements before and behind the vectors: at most 14
    const int32_t tail0 = head + nvec * kPer;
    const int32_t loose = head + (n - tail0);
    if (static_cast<int32_t>(threadIdx.x) < loose) {
        const int32_t k = static_cast<int32_t>(threadIdx.x) < head ? threadIdx.x
                                                                   : tail0 + threadIdx.x - head;
        const double x = static_cast<double>(to_f<T>(p[k]));
        acc = fma(x, x, acc);
    }
    return acc;
}

// Sum over the CTA in a fixed order; every thread gets it.
__device__ __forceinline__ double cta_sum(double v, double* red) {
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
    #pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) t += red[w];
    return t;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kSumCtas)
    norm_partial_kernel(const __grid_constant__ Tensors<CAP> t, double* __restrict__ partials) {
    __shared__ double red[kThreads / 32];
    grid_dependency_wait();
    grid_dependents_launch();
    const int32_t chunks = t.first_chunk[t.count];
    double acc = 0.0;
    const uint64_t last = l2_policy_evict_last(), early = l2_policy_evict_first();
    for (int32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int k = find_tensor(t, c);
        const int64_t behind = static_cast<int64_t>(chunks - c) * t.chunk * (t.dtype[k] == GEMM_F32 ? 4 : 2);
        const uint64_t pol = behind <= kKeepBytes ? last : early;
        const int64_t at = static_cast<int64_t>(c - t.first_chunk[k]) * t.chunk;
        const int64_t left = t.size[k] - at;
        const int32_t n = static_cast<int32_t>(left < t.chunk ? left : t.chunk);
        if (t.dtype[k] == GEMM_F32)
            acc += chunk_sum(static_cast<const float*>(t.src[k]) + at, n, pol);
        else if (t.dtype[k] == GEMM_BF16)
            acc += chunk_sum(static_cast<const __nv_bfloat16*>(t.src[k]) + at, n, pol);
        else
            acc += chunk_sum(static_cast<const __half*>(t.src[k]) + at, n, pol);
    }
    const double s = cta_sum(acc, red);
    if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

template <typename T>
__device__ __forceinline__ uint4 scale_vec(uint4 u, float f) {
    Vec16<T> w;
    w.u = u;
    #pragma unroll
    for (int e = 0; e < static_cast<int>(16 / sizeof(T)); ++e) w.e[e] = from_f<T>(to_f<T>(w.e[e]) * f);
    return w.u;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T* p, T* o, int32_t n, float f) {
    constexpr int kPer = 16 / sizeof(T);
    // vectors only where source and destination reach a 16-byte boundary together
    const bool same = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15u) == 0;
    if (!same) {
        for (int32_t i = threadIdx.x; i < n; i += kThreads) o[i] = from_f<T>(to_f<T>(p[i]) * f);
        return;
    }
    const int32_t head = head_of(p, n);
    const int32_t nvec = (n - head) / kPer;
    const uint4* v = reinterpret_cast<const uint4*>(p + head);
    uint4* w = reinterpret_cast<uint4*>(o + head);
    for (int32_t i = threadIdx.x; i < nvec; i += kVecs * kThreads) {
        uint4 r[kVecs];
        #pragma unroll
        for (int q = 0; q < kVecs; ++q) {
            const int32_t k = i + q * kThreads;
            if (k < nvec) r[q] = __ldcs(v + k);
        }
        #pragma unroll
        for (int q = 0; q < kVecs; ++q) {
            const int32_t k = i + q * kThreads;
            if (k < nvec) __stcs(w + k, scale_vec<T>(r[q], f));
        }
    }
    const int32_t tail0 = head + nvec * kPer;
    const int32_t loose = head + (n - tail0);
    if (static_cast<int32_t>(threadIdx.x) < loose) {
        const int32_t k = static_cast<int32_t>(threadIdx.x) < head ? threadIdx.x
                                                                   : tail0 + threadIdx.x - head;
        o[k] = from_f<T>(to_f<T>(p[k]) * f);
    }
}

// By a factor that FP32 holds as a subnormal, if at all: the products may be
// normal numbers all the same, so they are made in FP64.  Rare, and out of line as
// batch_again is.
template <typename T>
__device__ __noinline__ void chunk_scale_far(const T* p, T* o, int32_t n, double f) {
    for (int32_t i = threadIdx.x; i < n; i += kThreads)
        o[i] = from_f<T>(static_cast<float>(static_cast<double>(to_f<T>(p[i])) * f));
}

template <typename T>
__device__ __forceinline__ void chunk_apply(const void* p, void* o, int64_t at, int32_t n, double f) {
    const T* src = static_cast<const T*>(p) + at;
    T* dst = static_cast<T*>(o) + at;
    if (f < 0x1p-126) chunk_scale_far(src, dst, n, f);
    else chunk_scale(src, dst, n, static_cast<float>(f));
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kApplyCtas)
    apply_kernel(const __grid_constant__ Tensors<CAP> t, const ApplyParams a) {
    __shared__ double red[kThreads / 32];
    grid_dependency_wait();
    grid_dependents_launch();
    double acc = 0.0;
    for (int32_t i = threadIdx.x; i < a.num_partials; i += kThreads) acc += a.partials[i];
    const double norm = sqrt(cta_sum(acc, red)) * static_cast<double>(a.inv_scale);
    // the caller, who decides by the stored norm, and the clipping agree on what is finite
    const float stored = static_cast<float>(norm);
    if (a.write_norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = stored;
    double f = static_cast<double>(a.inv_scale);
    if (isfinite(stored) && norm > static_cast<double>(a.max_norm))
        f *= static_cast<double>(a.max_norm) / norm;
    const int32_t chunks = t.first_chunk[t.count];
    // this CTA's chunks, the last one first
    const int32_t mine = chunks > static_cast<int32_t>(blockIdx.x)
                             ? (chunks - 1 - static_cast<int32_t>(blockIdx.x)) / static_cast<int32_t>(gridDim.x)
                             : -1;
    for (int32_t r = mine; r >= 0; --r) {
        const int32_t c = static_cast<int32_t>(blockIdx.x) + r * static_cast<int32_t>(gridDim.x);
        const int k = find_tensor(t, c);
        if (static_cast<float>(f) == 1.0f && t.dst[k] == t.src[k]) continue;
        const int64_t at = static_cast<int64_t>(c - t.first_chunk[k]) * t.chunk;
        const int64_t left = t.size[k] - at;
        const int32_t n = static_cast<int32_t>(left < t.chunk ? left : t.chunk);
        if (t.dtype[k] == GEMM_F32) chunk_apply<float>(t.src[k], t.dst[k], at, n, f);
        else if (t.dtype[k] == GEMM_BF16) chunk_apply<__nv_bfloat16>(t.src[k], t.dst[k], at, n, f);
        else chunk_apply<__half>(t.src[k], t.dst[k], at, n, f);
    }
}

bool dtype_ok(int32_t t) { return t == GEMM_F16 || t == GEMM_BF16 || t == GEMM_F32; }
int64_t esize(int32_t t) { return t == GEMM_F32 ? 4 : 2; }

int64_t launches_for(int64_t count) { return (count + kPerLaunch - 1) / kPerLaunch; }

int64_t workspace_for(int64_t count, int32_t sms) {
    const int64_t l = launches_for(count);
    return (l < 1 ? 1 : l) * static_cast<int64_t>(sms) * kSumCtas * 8;
}

// CTAs write the outputs while others still read gradients: the outputs have to
// be apart from each other, and from every gradient but their own (where they
// may be that gradient itself).  With the starts and the ends of the gradients
// sorted, those that meet [s, e) are the starts before e less the ends up to s.
gemm_status_t check_overlap(int64_t count, const void* const* grads, void* const* outs,
                            const int64_t* sizes, const int32_t* dtypes) {
    if (count < 2 && (outs == nullptr || count == 0 || outs[0] == grads[0])) return GEMM_OK;
    uintptr_t* mem = new (std::nothrow) uintptr_t[4 * count];
    if (mem == nullptr) return GEMM_ERR_ALLOC;
    uintptr_t* gs = mem;                     // gradients' starts and ends
    uintptr_t* ge = mem + count;
    uintptr_t* os = mem + 2 * count;         // outputs', sorted apart: disjoint intervals keep their order
    uintptr_t* oe = mem + 3 * count;
    int64_t n = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (sizes[i] == 0) continue;
        const uintptr_t bytes = static_cast<uintptr_t>(sizes[i] * esize(dtypes[i]));
        gs[n] = reinterpret_cast<uintptr_t>(grads[i]);
        ge[n] = gs[n] + bytes;
        os[n] = outs ? reinterpret_cast<uintptr_t>(outs[i]) : gs[n];
        oe[n] = os[n] + bytes;
        ++n;
    }
    std::sort(gs, gs + n);
    std::sort(ge, ge + n);
    std::sort(os, os + n);
    std::sort(oe, oe + n);
    bool ok = true;
    for (int64_t i = 0; i + 1 < n; ++i) ok = ok && oe[i] <= os[i + 1];
    for (int64_t i = 0; i < count && ok; ++i) {
        if (sizes[i] == 0) continue;
        const uintptr_t s = reinterpret_cast<uintptr_t>(outs ? outs[i] : grads[i]);
        const uintptr_t e = s + static_cast<uintptr_t>(sizes[i] * esize(dtypes[i]));
        const int64_t meet = (std::lower_bound(gs, gs + n, e) - gs) - (std::upper_bound(ge, ge + n, s) - ge);
        ok = meet == (s == reinterpret_cast<uintptr_t>(grads[i]) ? 1 : 0);
    }
    delete[] mem;
    return ok ? GEMM_OK : GEMM_ERR_INVALID_VALUE;
}

cudaLaunchConfig_t config(int grid, cudaStream_t stream, cudaLaunchAttribute* attr) {
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

struct Call {
    int64_t count;
    const void* const* grads;
    void* const* outs;
    const int64_t* sizes;
    const int32_t* dtypes;
    float max_norm, inv_scale;
    float* norm;
    double* partials;
    int sms;
    cudaStream_t stream;
};

// Tensors [first, first + n) of the call that are not empty.
template <int CAP>
void fill(Tensors<CAP>& t, const Call& c, int64_t first, int64_t n) {
    int32_t chunk = 0;
    t.count = 0;
    for (int64_t i = first; i < first + n; ++i) {
        if (c.sizes[i] == 0) continue;
        const int k = t.count++;
        t.src[k] = c.grads[i];
        t.dst[k] = c.outs ? c.outs[i] : const_cast<void*>(c.grads[i]);
        t.size[k] = c.sizes[i];
        t.dtype[k] = static_cast<uint8_t>(c.dtypes[i]);
        t.first_chunk[k] = chunk;
        chunk += static_cast<int32_t>((c.sizes[i] + t.chunk - 1) / t.chunk);
    }
    t.first_chunk[t.count] = chunk;
}

// Two capacities: a launch copies its parameters, and 64 tensors (2 KB) go out
// faster than 512 (15 KB).
template <int CAP>
cudaError_t run(const Call& c) {
    Tensors<CAP> t;
    const int64_t parts = c.count > 0 ? (c.count + CAP - 1) / CAP : 1;
    int32_t partials = 0;
    cudaLaunchAttribute attr;
    for (int pass = 0; pass < 2; ++pass) {
        for (int64_t l = 0; l < parts; ++l) {
            const int64_t first = l * CAP;
            const int64_t n = c.count - first < CAP ? c.count - first : CAP;
            int64_t total = 0;
            for (int64_t i = first; i < first + n; ++i) total += c.sizes[i];
            t.chunk = kMostChunk;
            while (t.chunk > kLeastChunk && total / t.chunk < 4 * c.sms) t.chunk /= 2;
            fill(t, c, first, n);
            const int32_t chunks = t.first_chunk[t.count];
            const int most = c.sms * (pass == 0 ? kSumCtas : kApplyCtas);
            int grid = chunks < most ? chunks : most;
            if (pass == 0) {
                if (grid == 0) continue;
                cudaLaunchConfig_t cfg = config(grid, c.stream, &attr);
                const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_partial_kernel<CAP>, t,
                                                         c.partials + partials);
                if (e != cudaSuccess) return e;
                partials += grid;
            } else {
                // nothing to scale: only the norm is written, by one CTA
                bool in_place = true;
                for (int32_t k = 0; k < t.count; ++k) in_place = in_place && t.dst[k] == t.src[k];
                if (in_place && c.inv_scale == 1.0f && std::isinf(c.max_norm)) t.first_chunk[t.count] = 0, grid = 0;
                if (grid == 0) {
                    if (l > 0) continue;
                    grid = 1;
                }
                const ApplyParams a{c.partials, partials, c.max_norm, c.inv_scale, c.norm,
                                    l == 0 ? 1 : 0};
                cudaLaunchConfig_t cfg = config(grid, c.stream, &attr);
                const cudaError_t e = cudaLaunchKernelEx(&cfg, apply_kernel<CAP>, t, a);
                if (e != cudaSuccess) return e;
            }
        }
    }
    return cudaSuccess;
}

}  // namespace

extern "C" {

int64_t grad_clip_workspace(int64_t count, int32_t num_sms) {
    if (count < 0 || count > (1ll << 40) || num_sms < 0) return -1;
    if (num_sms == 0) {
        const int s = device_sms();
        if (s <= 0) return -1;
        num_sms = s;
    }
    return workspace_for(count, num_sms);
}

gemm_status_t grad_clip(int64_t count, const void* const* grads, void* const* outs,
                        const int64_t* sizes, const int32_t* dtypes, float max_norm,
                        float inv_scale, float* norm, void* workspace, int64_t workspace_bytes,
                        gemm_stream_t stream) {
    if (count < 0 || (count > 0 && (grads == nullptr || sizes == nullptr || dtypes == nullptr)))
        return GEMM_ERR_INVALID_VALUE;
    if (!(max_norm > 0.0f) || !(inv_scale > 0.0f) || std::isinf(inv_scale))
        return GEMM_ERR_INVALID_VALUE;
    if (norm == nullptr || (reinterpret_cast<uintptr_t>(norm) & 3u) != 0)
        return GEMM_ERR_INVALID_VALUE;
    for (int64_t i = 0; i < count; ++i) {
        if (sizes[i] < 0 || sizes[i] > (1ll << 40) || !dtype_ok(dtypes[i]))
            return GEMM_ERR_INVALID_VALUE;
        if (sizes[i] == 0) continue;
        const uintptr_t m = static_cast<uintptr_t>(esize(dtypes[i])) - 1;
        const void* o = outs ? outs[i] : grads[i];
        if (grads[i] == nullptr || o == nullptr || (reinterpret_cast<uintptr_t>(grads[i]) & m) != 0 ||
            (reinterpret_cast<uintptr_t>(o) & m) != 0)
            return GEMM_ERR_INVALID_VALUE;
    }
    // chunk numbers are 32-bit within a launch
    for (int64_t l = 0; l * kPerLaunch < count; ++l) {
        int64_t chunks = 0;
        for (int64_t i = l * kPerLaunch; i < count && i < (l + 1) * kPerLaunch; ++i)
            chunks += (sizes[i] + kLeastChunk - 1) / kLeastChunk;
        if (chunks > (1ll << 30)) return GEMM_ERR_INVALID_VALUE;
    }
    // in place, with nothing to scale: only the norm is written
    bool norm_only = inv_scale == 1.0f && std::isinf(max_norm);
    for (int64_t i = 0; outs != nullptr && norm_only && i < count; ++i)
        norm_only = sizes[i] == 0 || outs[i] == grads[i];
    const gemm_status_t st = norm_only ? GEMM_OK : check_overlap(count, grads, outs, sizes, dtypes);
    if (st != GEMM_OK) return st;
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0)
        return GEMM_ERR_INVALID_VALUE;
    const int sms = device_sms();
    if (sms < 0) return GEMM_ERR_LAUNCH;
    if (sms == 0) return GEMM_ERR_NOT_SUPPORTED;
    if (workspace_bytes < workspace_for(count, sms)) return GEMM_ERR_INVALID_VALUE;
    const Call c{count, grads, outs, sizes, dtypes, max_norm, inv_scale, norm,
                 static_cast<double*>(workspace), sms,
                 reinterpret_cast<cudaStream_t>(stream)};
    const cudaError_t e = count <= 64 ? run<64>(c) : run<kPerLaunch>(c);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

}  // extern "C"
