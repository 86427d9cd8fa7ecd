// glu_kern.cuh -- the element kernels of the gated linear layer
// (include/glu_sm103.h): the gate where there is no product to fuse it into
// (K == 0), and the backward pass's dP with the sums of its columns.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "epilogue_ops.cuh"
#include "f32x2.cuh"
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
            P[r * ldp + c] = from_f<OutT>(g);
            P[r * ldp + F + c] = from_f<OutT>(u);
        }
        H[r * ldh + c] = from_f<OutT>(activate(act, g) * u);
    }
}

struct GluBackParams {
    const void* dH; int64_t lddh;
    const void* P; int64_t ldp;
    void* dP; int64_t lddp;
    void* dPa; int64_t ldpa;  // a second copy of dP in aligned rows, zeros behind column 2F, or NULL
    int64_t M;
    int64_t F;
    int32_t act;
    int64_t slab_rows;       // rows per CTA (blockIdx.y)
    float* partials;         // [slabs][2F] column sums of dP, or NULL
};

constexpr int kGluBackWarps = 8;
constexpr int kGluBackRows = 2;     // rows whose loads a warp has in flight together

// 8 elements of a row as they lie in memory (VEC: consecutive; else 32 apart).
template <typename T, bool VEC>
struct Raw8 {
    union {
        uint4 u[sizeof(T) / 2];
        T e[8];
    };
    // the loads; element i is at p + base + i (VEC) or p + base + 32 i
    __device__ __forceinline__ void load(const T* p, int64_t base, int64_t F) {
        if constexpr (VEC) {
            if (base < F) {
                #pragma unroll
                for (int q = 0; q < static_cast<int>(sizeof(T) / 2); ++q)
                    u[q] = __ldcs(reinterpret_cast<const uint4*>(p + base) + q);
            }
        } else {
            #pragma unroll
            for (int i = 0; i < 8; ++i)
                if (base + i * 32 < F) e[i] = p[base + i * 32];
        }
    }
    __device__ __forceinline__ void store(T* p, int64_t base, int64_t F) const {
        if constexpr (VEC) {
            if (base < F) {
                #pragma unroll
                for (int q = 0; q < static_cast<int>(sizeof(T) / 2); ++q)
                    reinterpret_cast<uint4*>(p + base)[q] = u[q];
            }
        } else {
            #pragma unroll
            for (int i = 0; i < 8; ++i)
                if (base + i * 32 < F) p[base + i * 32] = e[i];
        }
    }
};

// dG = dH U act'(G), dU = dH act(G).  A CTA covers 256 columns of each half
// (8 per lane) by slab_rows rows, its warps taking the rows in turn; bound by
// HBM (3 reads and 2 writes per element of H; 8192 x 14336 bf16 195 us, 6.0
// TB/s) once enough loads are in flight:
// each warp issues those of kGluBackRows rows before it works on them.  A
// thread reads P's elements before it writes dP's, so dP may be P.  Column
// sums of the FP32 values: per thread over its rows, then over the warps in
// order, then over the slabs by glu_dbias_kernel.
template <typename T, typename PT, bool VEC, bool SUMS>
__global__ void __launch_bounds__(32 * kGluBackWarps, VEC ? 4 : 2)
    glu_back_kernel(const __grid_constant__ GluBackParams p) {
    __shared__ float red[SUMS ? kGluBackWarps : 1][SUMS ? 512 : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col0 = static_cast<int64_t>(blockIdx.x) * 256;
    const int64_t base = col0 + (VEC ? lane * 8 : lane);
    const int64_t row0 = static_cast<int64_t>(blockIdx.y) * p.slab_rows;
    int64_t row1 = row0 + p.slab_rows;
    if (row1 > p.M) row1 = p.M;
    grid_dependency_wait();
    grid_dependents_launch();
    float sg[SUMS ? 8 : 1], su[SUMS ? 8 : 1];
    if constexpr (SUMS) {
        #pragma unroll
        for (int e = 0; e < 8; ++e) sg[e] = su[e] = 0.0f;
    }
    for (int64_t r = row0 + warp; r < row1; r += kGluBackWarps * kGluBackRows) {
        Raw8<T, VEC> h[kGluBackRows];
        Raw8<PT, VEC> gu[kGluBackRows][2];
        #pragma unroll
        for (int k = 0; k < kGluBackRows; ++k) {
            const int64_t rk = r + k * kGluBackWarps;
            if (rk < row1) {
                const PT* prow = static_cast<const PT*>(p.P) + rk * p.ldp;
                h[k].load(static_cast<const T*>(p.dH) + rk * p.lddh, base, p.F);
                gu[k][0].load(prow, base, p.F);
                gu[k][1].load(prow + p.F, base, p.F);
            }
        }
        #pragma unroll
        for (int k = 0; k < kGluBackRows; ++k) {
            const int64_t rk = r + k * kGluBackWarps;
            if (rk >= row1) break;
            float g[8], a[8], d[8];
            #pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = to_f<PT>(gu[k][0].e[e]);
            act_and_slope8(p.act, g, a, d);
            Raw8<T, VEC> og, ou;
            #pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = to_f<T>(h[k].e[e]);
                const float dg = x * to_f<PT>(gu[k][1].e[e]) * d[e], du = x * a[e];
                og.e[e] = from_f<T>(dg);
                ou.e[e] = from_f<T>(du);
                if constexpr (SUMS) {
                    sg[e] += dg;                       // (columns past F are not looked at)
                    su[e] += du;
                }
            }
            T* drow = static_cast<T*>(p.dP) + rk * p.lddp;
            og.store(drow, base, p.F);
            ou.store(drow + p.F, base, p.F);
            if (!VEC && p.dPa != nullptr) {
                T* arow = static_cast<T*>(p.dPa) + rk * p.ldpa;
                og.store(arow, base, p.F);
                ou.store(arow + p.F, base, p.F);
                if (blockIdx.x == 0)
                    for (int64_t c = 2 * p.F + lane; c < p.ldpa; c += 32) arow[c] = from_f<T>(0.0f);
            }
        }
    }
    if constexpr (SUMS) {
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = VEC ? lane * 8 + e : lane + e * 32;
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

// dbias = sum over the slabs: 32 columns per CTA, 32 lines of threads that
// take the slabs in turn and are added in line order.
static __global__ void __launch_bounds__(1024)
    glu_dbias_kernel(const float* partials, int32_t slabs, int64_t cols, void* dbias,
                     int32_t dtype) {
    __shared__ float red[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + tx;
    grid_dependency_wait();
    grid_dependents_launch();
    float t = 0.0f;
    if (c < cols) {
        #pragma unroll 4
        for (int32_t s = ty; s < slabs; s += 32) t += partials[static_cast<int64_t>(s) * cols + c];
    }
    red[ty][tx] = t;
    __syncthreads();
    if (ty != 0 || c >= cols) return;
    t = 0.0f;
    #pragma unroll
    for (int y = 0; y < 32; ++y) t += red[y][tx];
    store_elem(dbias, dtype, c, t);
}

// -------------------------------------------------------- a few tokens (decode)

struct GluDotParams {
    const void* X; int64_t ldx;
    const void* W; int64_t ldw;
    void* H; int64_t ldh;
    void* P; int64_t ldp;
    const void* bias;
    int32_t bias_dtype, act, h_dtype;
    int32_t F, K;
};

constexpr int kGluDotThreads = 256;
constexpr int kGluDotCtas = 4;          // per SM
constexpr int kGluDotAhead = 4;         // 256-element pieces of both rows in flight per warp

// The gated layer of MT tokens (1 or 2): bound by the stream of W.  A warp
// takes one gate row and its up row at a time, 16 bytes per lane and load,
// kGluDotAhead pieces of both rows in flight; X (a few KB) comes from L1.
// Against the tensor-core path there is no tile to fill, no pipeline to start
// and no split of K to join: what a problem of a few microseconds spends its
// time on.  FP32 sums in pairs, joined over the lanes by a butterfly.
// K is a multiple of 8; rows of X and W are 16-byte aligned.  X is read by plain
// loads: the kernel before this one, still running when this one begins, writes it.
// One token, bf16: 1024 -> 4096 6.3 us with the launch, 2.5 us of which are W's 17
// MB; W not in L2, one call after another, 4096 -> 8192 22.0 us, 6.1 TB/s.
template <typename T, int MT>
__global__ void __launch_bounds__(kGluDotThreads, kGluDotCtas)
    glu_dot_kernel(const __grid_constant__ GluDotParams p) {
    const int lane = threadIdx.x & 31;
    const int32_t warp = static_cast<int32_t>(blockIdx.x) * (kGluDotThreads / 32) +
                         static_cast<int32_t>(threadIdx.x >> 5);
    const int32_t warps = static_cast<int32_t>(gridDim.x) * (kGluDotThreads / 32);
    const T* X = static_cast<const T*>(p.X);
    grid_dependency_wait();
    grid_dependents_launch();
    for (int32_t f = warp; f < p.F; f += warps) {
        const T* wg = static_cast<const T*>(p.W) + static_cast<int64_t>(f) * p.ldw;
        const T* wu = wg + static_cast<int64_t>(p.F) * p.ldw;
        F2 ag[MT], au[MT];
        #pragma unroll
        for (int m = 0; m < MT; ++m) ag[m] = au[m] = mk2(0.0f);
        // (unsigned: K may end less than a step below 2^31)
        const uint32_t K = static_cast<uint32_t>(p.K);
        for (uint32_t k0 = lane * 8; k0 < K; k0 += 256 * kGluDotAhead) {
            uint4 g[kGluDotAhead], u[kGluDotAhead];
            #pragma unroll
            for (int i = 0; i < kGluDotAhead; ++i) {
                const uint32_t k = k0 + i * 256;
                const bool in = k < K;
                g[i] = in ? __ldcs(reinterpret_cast<const uint4*>(wg + k)) : make_uint4(0u, 0u, 0u, 0u);
                u[i] = in ? __ldcs(reinterpret_cast<const uint4*>(wu + k)) : make_uint4(0u, 0u, 0u, 0u);
            }
            #pragma unroll
            for (int i = 0; i < kGluDotAhead; ++i) {
                const uint32_t k = k0 + i * 256;
                if (k >= K) break;
                const uint32_t gw[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
                const uint32_t uw[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
                #pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const uint4 x = *reinterpret_cast<const uint4*>(X + m * p.ldx + k);
                    const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const F2 xv = unpack2<T>(xw[q]);
                        ag[m] = fma2(unpack2<T>(gw[q]), xv, ag[m]);
                        au[m] = fma2(unpack2<T>(uw[q]), xv, au[m]);
                    }
                }
            }
        }
        float mine_g = 0.0f, mine_u = 0.0f;              // lane m keeps token m's sums
        #pragma unroll
        for (int m = 0; m < MT; ++m) {
            float sg = sum2(ag[m]), su = sum2(au[m]);
            #pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                sg += __shfl_xor_sync(0xffffffffu, sg, o);
                su += __shfl_xor_sync(0xffffffffu, su, o);
            }
            if (lane == m) {
                mine_g = sg;
                mine_u = su;
            }
        }
        if (lane < MT) {
            if (p.bias != nullptr) {
                mine_g += load_bias_elem(p.bias, p.bias_dtype, f);
                mine_u += load_bias_elem(p.bias, p.bias_dtype, static_cast<int64_t>(p.F) + f);
            }
            if (p.P != nullptr) {
                store_elem(p.P, p.h_dtype, lane * p.ldp + f, mine_g);
                store_elem(p.P, p.h_dtype, lane * p.ldp + p.F + f, mine_u);
            }
            store_elem(p.H, p.h_dtype, lane * p.ldh + f, activate(p.act, mine_g) * mine_u);
        }
    }
}

}  // namespace gemm103
