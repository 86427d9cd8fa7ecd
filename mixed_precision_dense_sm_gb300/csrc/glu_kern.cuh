// glu_kern.cuh -- the element kernels of the gated linear layer
// (include/glu_sm103.h): the gate where there is no product to fuse it into
// (K == 0), and the backward pass's dP with the sums of its columns.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "epilogue_ops.cuh"
#include "ptx.cuh"

namespace gemm103 {

// act(x) and act'(x) of 8 values, the choice made outside the element loops:
//   SiLU  s = 1 / (1 + e^-x):  x s,  s (1 + x (1 - s))
//   GELU  Phi = erfc(-x / sqrt 2) / 2:  x Phi,  Phi + x e^(-x^2 / 2) / sqrt(2 pi)
//   ReLU  max(x, 0),  1 for x > 0 else 0
__device__ __forceinline__ void act_and_slope8(int act, const float (&x)[8], float (&a)[8],
                                               float (&d)[8]) {
    if (act == kActSilu) {
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float s = __fdividef(1.0f, 1.0f + __expf(-x[e]));
            a[e] = x[e] * s;
            d[e] = s * fmaf(x[e], 1.0f - s, 1.0f);
        }
    } else if (act == kActGelu) {
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float h = 0.5f * erfc_nr(fabsf(x[e]) * 0.70710678118654752f);
            const float phi = x[e] >= 0.0f ? 1.0f - h : h;
            a[e] = x[e] * phi;
            // e^(-x^2/2) is 0 in FP32 beyond |x| = 15, where x times it would be inf * 0 for x = inf
            const float g = fabsf(x[e]) < 15.0f
                                ? x[e] * __expf(-0.5f * x[e] * x[e]) * 0.39894228040143268f : 0.0f;
            d[e] = phi + g;
        }
    } else if (act == kActRelu) {
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
            a[e] = relu(x[e]);
            d[e] = x[e] > 0.0f ? 1.0f : 0.0f;
        }
    } else {
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
            a[e] = x[e];
            d[e] = 1.0f;
        }
    }
}

template <typename T> __device__ __forceinline__ float glu_to_f(T v);
template <> __device__ __forceinline__ float glu_to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float glu_to_f<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float glu_to_f<__nv_bfloat16>(__nv_bfloat16 v) {
    return __bfloat162float(v);
}
template <typename T> __device__ __forceinline__ T glu_from_f(float v);
template <> __device__ __forceinline__ float glu_from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half glu_from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 glu_from_f<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// K == 0: P = [G U] is the bias (0 where there is none), H = act(G) * U.
template <typename OutT>
__global__ void __launch_bounds__(256)
    glu_gate_kernel(const void* bias, int32_t bias_dtype, int32_t act, OutT* __restrict__ H,
                    int64_t ldh, OutT* P, int64_t ldp, int64_t M, int64_t F) {
    const int64_t total = M * F;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t r = i / F, c = i - r * F;
        const float g = bias ? load_bias_elem(bias, bias_dtype, c) : 0.0f;
        const float u = bias ? load_bias_elem(bias, bias_dtype, F + c) : 0.0f;
        if (P != nullptr) {
            P[r * ldp + c] = glu_from_f<OutT>(g);
            P[r * ldp + F + c] = glu_from_f<OutT>(u);
        }
        H[r * ldh + c] = glu_from_f<OutT>(activate(act, g) * u);
    }
}

struct GluBackParams {
    const void* dH; int64_t lddh;
    const void* P; int64_t ldp;
    void* dP; int64_t lddp;
    int64_t M;
    int64_t F;
    int32_t act;
    int32_t vec;             // rows of dH, P, dP and their halves 16-byte aligned, F a multiple of 8
    int64_t slab_rows;       // rows per CTA (blockIdx.y)
    float* partials;         // [slabs][2F] column sums of dP, or NULL
};

constexpr int kGluBackWarps = 8;

template <typename T>
union GluVec {
    uint4 u[sizeof(T) / 2];
    T e[8];
};

// 8 elements at p + base + e * step; 0 past column F.
template <typename T>
__device__ __forceinline__ void glu_load8(const T* p, bool vec, int64_t base, int64_t F, float (&o)[8]) {
    if (vec) {
        if (base >= F) {
            #pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = 0.0f;
            return;
        }
        GluVec<T> v;
        #pragma unroll
        for (int q = 0; q < static_cast<int>(sizeof(T) / 2); ++q)
            v.u[q] = __ldcs(reinterpret_cast<const uint4*>(p + base) + q);
        #pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = glu_to_f<T>(v.e[e]);
    } else {
        #pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = base + e * 32 < F ? glu_to_f<T>(p[base + e * 32]) : 0.0f;
    }
}

template <typename T>
__device__ __forceinline__ void glu_store8(T* p, bool vec, int64_t base, int64_t F, const float (&v)[8]) {
    if (vec) {
        if (base >= F) return;
        GluVec<T> w;
        #pragma unroll
        for (int e = 0; e < 8; ++e) w.e[e] = glu_from_f<T>(v[e]);
        #pragma unroll
        for (int q = 0; q < static_cast<int>(sizeof(T) / 2); ++q)
            reinterpret_cast<uint4*>(p + base)[q] = w.u[q];
    } else {
        #pragma unroll
        for (int e = 0; e < 8; ++e)
            if (base + e * 32 < F) p[base + e * 32] = glu_from_f<T>(v[e]);
    }
}

// dG = dH U act'(G), dU = dH act(G).  A CTA covers 256 columns of each half
// (8 per lane) by slab_rows rows, its warps taking the rows in turn; bound by
// HBM: 3 reads and 2 writes per element of H.  A thread reads P's elements
// before it writes dP's, so dP may be P.  Column sums of the FP32 values: per
// thread over its rows, then over the warps in order, then over the slabs by
// glu_dbias_kernel.  The stores of dP are kept in L2 (the products read it next).
template <typename T, typename PT, bool SUMS>
__global__ void __launch_bounds__(32 * kGluBackWarps)
    glu_back_kernel(const __grid_constant__ GluBackParams p) {
    __shared__ float red[SUMS ? kGluBackWarps : 1][SUMS ? 512 : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool vec = p.vec != 0;
    const int64_t col0 = static_cast<int64_t>(blockIdx.x) * 256;
    const int64_t base = col0 + (vec ? lane * 8 : lane);
    const int64_t row0 = static_cast<int64_t>(blockIdx.y) * p.slab_rows;
    int64_t row1 = row0 + p.slab_rows;
    if (row1 > p.M) row1 = p.M;
    grid_dependency_wait();
    float sg[8], su[8];
    #pragma unroll
    for (int e = 0; e < 8; ++e) sg[e] = su[e] = 0.0f;
    #pragma unroll 2
    for (int64_t r = row0 + warp; r < row1; r += kGluBackWarps) {
        float h[8], g[8], u[8];
        const PT* prow = static_cast<const PT*>(p.P) + r * p.ldp;
        T* drow = static_cast<T*>(p.dP) + r * p.lddp;
        glu_load8<T>(static_cast<const T*>(p.dH) + r * p.lddh, vec, base, p.F, h);
        glu_load8<PT>(prow, vec, base, p.F, g);
        glu_load8<PT>(prow + p.F, vec, base, p.F, u);
        float a[8], d[8];
        act_and_slope8(p.act, g, a, d);
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
            g[e] = h[e] * u[e] * d[e];
            u[e] = h[e] * a[e];
            if constexpr (SUMS) {
                sg[e] += g[e];
                su[e] += u[e];
            }
        }
        glu_store8<T>(drow, vec, base, p.F, g);
        glu_store8<T>(drow + p.F, vec, base, p.F, u);
    }
    if constexpr (SUMS) {
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = vec ? lane * 8 + e : lane + e * 32;
            red[warp][c] = sg[e];
            red[warp][256 + c] = su[e];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < 512; c += 32 * kGluBackWarps) {
            const int64_t col = col0 + (c & 255);
            if (col >= p.F) continue;
            float t = 0.0f;
            #pragma unroll
            for (int w = 0; w < kGluBackWarps; ++w) t += red[w][c];
            p.partials[static_cast<int64_t>(blockIdx.y) * 2 * p.F + (c < 256 ? 0 : p.F) + col] = t;
        }
    }
}

// dbias = sum over the slabs, in order.
static __global__ void __launch_bounds__(256)
    glu_dbias_kernel(const float* __restrict__ partials, int32_t slabs, int64_t cols, void* dbias,
                     int32_t dtype) {
    grid_dependency_wait();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (c >= cols) return;
    float t = 0.0f;
    #pragma unroll 8
    for (int32_t s = 0; s < slabs; ++s) t += partials[static_cast<int64_t>(s) * cols + c];
    if (dtype == 2) static_cast<float*>(dbias)[c] = t;
    else if (dtype == 1) static_cast<__nv_bfloat16*>(dbias)[c] = __float2bfloat16_rn(t);
    else static_cast<__half*>(dbias)[c] = __float2half_rn(t);
}

}  // namespace gemm103
