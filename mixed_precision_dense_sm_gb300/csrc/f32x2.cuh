// f32x2.cuh -- FP32 arithmetic on pairs, and conversions between FP32 and the
// storage types: single elements, elements of a type chosen at run time, and
// pairs of 16-bit elements.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace gemm103 {

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) {
    return __bfloat162float(v);
}
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// p[i] = v rounded to type 0 = F16, 1 = BF16, 2 = F32.
__device__ __forceinline__ void store_elem(void* p, int32_t dtype, int64_t i, float v) {
    if (dtype == 2) static_cast<float*>(p)[i] = v;
    else if (dtype == 1) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// Two FP32 values in a 64-bit register: the packed FP32 instructions do two
// lanes' work in one issue slot.  The element kernels here convert 16-bit
// data and do a dozen or more FP32 operations per element, so issue slots, not
// HBM, bound them in scalar form.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 mk2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ F2 mk2(float x) { return mk2(x, x); }
__device__ __forceinline__ void get2(F2 a, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ float sum2(F2 a) {
    float lo, hi;
    get2(a, lo, hi);
    return lo + hi;
}

// A pair of 16-bit elements (low half first) as FP32, and back, rounded.
template <typename E> __device__ __forceinline__ F2 unpack2(uint32_t w);
template <> __device__ __forceinline__ F2 unpack2<__nv_bfloat16>(uint32_t w) {
    return mk2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <> __device__ __forceinline__ F2 unpack2<__half>(uint32_t w) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return mk2(f.x, f.y);
}
template <typename E> __device__ __forceinline__ uint32_t pack2(F2 a);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(F2 a) {
    float lo, hi;
    get2(a, lo, hi);
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(F2 a) {
    float lo, hi;
    get2(a, lo, hi);
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace gemm103
