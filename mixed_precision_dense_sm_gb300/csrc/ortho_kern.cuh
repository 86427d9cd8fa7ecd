// ortho_kern.cuh -- the products of the orthogonalised update
// (include/ortho_sm103.h) on tcgen05, with their epilogues.
//
// The workspace holds every matrix in the wide orientation (n x m, n <= m), both
// sides padded with zeros to multiples of 64: products of zeros are zeros, so the
// padding keeps itself and only the last epilogue looks at the true sizes.
// Everything is FP16 times a power of two, kScale = 2^11: entries of X are as small
// as 1 / sqrt(n m), near FP16's subnormals without it, and up to 32 is held.
//
// One step is three products:
//   kGram  A = X X^T            upper tiles only; each is stored twice, as it is
//   kPoly  B = b A + c A A      and mirrored
//   kStep  X = a X + B X        X = hi + lo; the product reads hi, from one of two
//   kLast  O = scale (...)      buffers to the other, lo stays in place
// Operands come as boxes of 128 rows by two K chunks (32 KB) through 4-D maps (64
// elements, rows, chunk, matrix).  In the first two both operands are K-major; in
// kStep the right one is X with K along its rows (MN-major), a box of the same map.
//
// Two kernels.  ortho_pair_kernel: persistent, 256 x 256 tiles on CTA pairs, double-
// buffered accumulators, for many tiles.  ortho_tile_kernel: one 128 x 128 tile per
// cluster, whose 1 to 8 CTAs split K and add up through distributed shared memory,
// for few tiles.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace gemm103 {

enum : int { kGram = 0, kPoly = 1, kStep = 2, kLast = 3 };

constexpr float kOrthoScale = 2048.0f;
constexpr int kOrthoStages = 3;
constexpr uint32_t kOrthoBox = 32768;                // 128 rows x 128 bytes x 2 chunks
constexpr uint32_t kOrthoStage = 2 * kOrthoBox;      // A's and B's
constexpr uint32_t kOrthoSmem = kOrthoStages * kOrthoStage + 1024 + 256;
constexpr int kOrthoPairThreads = 320;               // warp 0 TMA, 1 MMA, 2-9 epilogue
constexpr int kOrthoTileThreads = 192;               // warp 0 TMA, 1 MMA, 2-5 epilogue

struct OrthoParams {
    int32_t batch, tiles, tiles_i;      // matrices; tiles of each; tiles along its rows
    int32_t k_blocks;                   // pairs of K chunks
    int32_t np, mp;                     // padded sides
    int32_t splits, log_width;          // ortho_tile_kernel: CTAs per tile; log2(128 / splits)
    float a, b, c;
    const __half* ah;                   // kPoly: A
    __half* out;                        // kGram: A, kPoly: B
    const __half* hi;                   // kStep, kLast
    __half* lo;
    __half* hi_out;                     // kStep
    __nv_bfloat16* O;                   // kLast
    int64_t ldo, stride_o;
    int32_t n, m, tall, vec;            // true sides (wide); O transposed; O's rows are vectors
    float scale;
    int* err;
    uint64_t wait_limit_ns;
    uint32_t debug_flags;
};

struct OrthoTile {
    int32_t b, i, j;
};

// Work item -> matrix and tile.  Symmetric products: the upper tiles (i <= j), by
// columns.  Others: by columns, so that the tiles of a wave share few columns of X.
template <int MODE>
__device__ __forceinline__ OrthoTile ortho_tile(const OrthoParams& p, int32_t item) {
    OrthoTile t;
    t.b = item / p.tiles;
    const int32_t k = item - t.b * p.tiles;
    if constexpr (MODE == kGram || MODE == kPoly) {
        int32_t j = static_cast<int32_t>((sqrtf(8.0f * static_cast<float>(k) + 1.0f) - 1.0f) * 0.5f);
        while (j * (j + 1) / 2 > k) --j;
        while ((j + 1) * (j + 2) / 2 <= k) ++j;
        t.j = j;
        t.i = k - j * (j + 1) / 2;
    } else {
        t.j = k / p.tiles_i;
        t.i = k - t.j * p.tiles_i;
    }
    return t;
}

__device__ __forceinline__ void half8(uint4 u, float* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}

// What the epilogue reads of 16 columns: A (kPoly), or hi and lo.
template <int MODE>
struct OrthoIn {
    uint4 u[MODE == kGram ? 1 : MODE == kPoly ? 2 : 4];
};
template <int MODE>
__device__ __forceinline__ bool ortho_inside(const OrthoParams& p, int32_t row, int32_t col) {
    return row < p.np && col < (MODE == kGram || MODE == kPoly ? p.np : p.mp);
}
template <int MODE>
__device__ __forceinline__ OrthoIn<MODE> ortho_read(const OrthoParams& p, int32_t b, int32_t row, int32_t col) {
    OrthoIn<MODE> in = {};
    if constexpr (MODE == kPoly) {
        const uint4* s = reinterpret_cast<const uint4*>(p.ah + (static_cast<int64_t>(b) * p.np + row) * p.np + col);
        in.u[0] = s[0], in.u[1] = s[1];
    } else if constexpr (MODE != kGram) {
        const int64_t at = (static_cast<int64_t>(b) * p.np + row) * p.mp + col;
        const uint4* h = reinterpret_cast<const uint4*>(p.hi + at);
        const uint4* l = reinterpret_cast<const uint4*>(p.lo + at);
        in.u[0] = h[0], in.u[1] = h[1], in.u[2] = l[0], in.u[3] = l[1];
    }
    return in;
}

// 16 columns of one row: sums v (of scaled products) to the result, and out.
// `mirror`: also to the transposed place.
template <int MODE>
__device__ __forceinline__ void ortho_finish(const OrthoParams& p, int32_t b, int32_t row, int32_t col,
                                             const OrthoIn<MODE>& in, float (&v)[16], bool mirror) {
    constexpr float kDown = 1.0f / kOrthoScale;
    if constexpr (MODE == kGram || MODE == kPoly) {
        if constexpr (MODE == kPoly) {
            float x[16];
            half8(in.u[0], x);
            half8(in.u[1], x + 8);
            const float c = p.c * kDown;
            #pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = fmaf(p.b, x[i], c * v[i]);
        } else {
            #pragma unroll
            for (int i = 0; i < 16; ++i) v[i] *= kDown;
        }
        __half* base = p.out + static_cast<int64_t>(b) * p.np * p.np;
        alignas(16) __half h[16];
        #pragma unroll
        for (int i = 0; i < 16; ++i) h[i] = __float2half_rn(v[i]);
        uint4* d = reinterpret_cast<uint4*>(base + static_cast<int64_t>(row) * p.np + col);
        d[0] = reinterpret_cast<const uint4*>(h)[0];
        d[1] = reinterpret_cast<const uint4*>(h)[1];
        if (mirror) {
            // (the lanes' rows are neighbours: 64 contiguous bytes per store)
            __half* t = base + static_cast<int64_t>(col) * p.np + row;
            #pragma unroll
            for (int i = 0; i < 16; ++i) t[static_cast<int64_t>(i) * p.np] = h[i];
        }
    } else {
        float x[16], y[8];
        half8(in.u[0], x);
        half8(in.u[1], x + 8);
        #pragma unroll
        for (int q = 0; q < 2; ++q) {
            half8(in.u[2 + q], y);
            #pragma unroll
            for (int i = 0; i < 8; ++i) x[8 * q + i] += y[i];
        }
        #pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = fmaf(p.a, x[i], v[i] * kDown);
        if constexpr (MODE == kStep) {
            alignas(16) __half h[16], l[16];
            #pragma unroll
            for (int i = 0; i < 16; ++i) {
                h[i] = __float2half_rn(v[i]);
                l[i] = __float2half_rn(v[i] - __half2float(h[i]));
            }
            const int64_t at = (static_cast<int64_t>(b) * p.np + row) * p.mp + col;
            uint4* d = reinterpret_cast<uint4*>(p.hi_out + at);
            d[0] = reinterpret_cast<const uint4*>(h)[0];
            d[1] = reinterpret_cast<const uint4*>(h)[1];
            d = reinterpret_cast<uint4*>(p.lo + at);
            d[0] = reinterpret_cast<const uint4*>(l)[0];
            d[1] = reinterpret_cast<const uint4*>(l)[1];
        } else {
            if (row >= p.n) return;
            const float s = p.scale * kDown;
            alignas(16) __nv_bfloat16 o[16];
            #pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float2bfloat16_rn(v[i] * s);
            __nv_bfloat16* base = p.O + b * p.stride_o;
            if (p.tall) {
                #pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (col + i < p.m) base[(col + i) * p.ldo + row] = o[i];
            } else if (p.vec && col + 16 <= p.m) {
                uint4* d = reinterpret_cast<uint4*>(base + row * p.ldo + col);
                d[0] = reinterpret_cast<const uint4*>(o)[0];
                d[1] = reinterpret_cast<const uint4*>(o)[1];
            } else {
                #pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (col + i < p.m) base[row * p.ldo + col + i] = o[i];
            }
        }
    }
}

__device__ __forceinline__ void ortho_give_up(const OrthoParams& p, volatile int* abort_flag) {
    *abort_flag = 1;
    if (p.err) atomicCAS(p.err, 0, 1);
}

// Bounded wait that also gives up once another role of the CTA has.  CLUSTER: for
// plain arrivals from the peer CTA.
template <bool CLUSTER = false>
__device__ __forceinline__ bool ortho_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                           const OrthoParams& p) {
    const uint32_t a = smem_addr(bar);
    auto done = [&] { return CLUSTER ? mbar_try_wait_cluster(a, parity) : mbar_try_wait(a, parity); };
    if (done()) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 1;; ++i) {
        if (done()) return true;
        if ((i & 63u) == 0 && (*abort_flag || global_timer_ns() - t0 > p.wait_limit_ns)) break;
    }
    ortho_give_up(p, abort_flag);
    return false;
}

// The MMAs of one stage (128 of K) into d.
template <int MODE, bool PAIR>
__device__ __forceinline__ void ortho_mma(uint32_t d, uint32_t sa, bool first) {
    constexpr bool kMN = MODE == kStep || MODE == kLast;      // B's K along its rows
    constexpr uint32_t kSide = PAIR ? 256 : 128;
    constexpr uint32_t idesc = instr_desc(0, false, kMN, kSide, kSide);
    const uint32_t sb = sa + kOrthoBox;
    #pragma unroll
    for (uint32_t kk = 0; kk < 8; ++kk) {
        const uint32_t km = (kk >> 2) * 16384u + (kk & 3u) * 32u;
        const uint64_t ad = smem_desc_sw128(sa + km, 16u, 1024u);
        const uint64_t bd = kMN ? smem_desc_sw128(sb + kk * 2048u, 16384u, 1024u)
                                : smem_desc_sw128(sb + km, 16u, 1024u);
        const uint32_t acc = first && kk == 0 ? 0u : 1u;
        if constexpr (PAIR) tc_mma_f16_pair(d, ad, bd, idesc, acc);
        else tc_mma_f16(d, ad, bd, idesc, acc);
    }
}

// ------------------------------------------------------------------- CTA pairs

template <int MODE>
__global__ void __launch_bounds__(kOrthoPairThreads, 1)
    ortho_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ OrthoParams p) {
    constexpr bool kMN = MODE == kStep || MODE == kLast;
    constexpr bool kSym = MODE == kGram || MODE == kPoly;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOrthoStages * kOrthoStage);
    uint64_t* empty = full + kOrthoStages;
    uint64_t* acc_full = empty + kOrthoStages;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    __shared__ volatile int abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int32_t pairs = static_cast<int32_t>(gridDim.x >> 1), items = p.batch * p.tiles;
    const int32_t mine = static_cast<int32_t>(blockIdx.x >> 1);

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < kOrthoStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 16);                 // 8 epilogue warps of both CTAs
        }
        mbar_init(drain, 1);
        fence_barrier_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t keep = l2_policy_evict_last();
            uint32_t armed = 0;
            bool ok = true;
            for (int32_t item = mine; item < items && ok; item += pairs) {
                const OrthoTile t = ortho_tile<MODE>(p, item);
                const int32_t r0 = t.i * 256 + static_cast<int32_t>(rank) * 128;
                const int32_t c0 = t.j * 256 + static_cast<int32_t>(rank) * 128;
                for (int32_t kb = 0; kb < p.k_blocks; ++kb, ++armed) {
                    const uint32_t s = armed % kOrthoStages, round = armed / kOrthoStages;
                    ok = ortho_wait(&empty[s], (round & 1u) ^ 1u, &abort_flag, p);
                    if (!ok) break;
                    uint8_t* sa = smem + s * kOrthoStage;
                    const uint32_t fb = map_to_rank(smem_addr(&full[s]), 0);
                    // the even CTA's barrier counts the bytes of both
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kOrthoStage);
                    if ((p.debug_flags & 1u) && armed == 0 && blockIdx.x == 0) continue;   // test hook: no load
                    tma_load_4d_pair(sa, &tmA, fb, 0, r0, kb * 2, t.b, keep);
                    if constexpr (kMN) tma_load_4d_pair(sa + kOrthoBox, &tmB, fb, 0, kb * 128, c0 >> 6, t.b, keep);
                    else tma_load_4d_pair(sa + kOrthoBox, &tmB, fb, 0, c0, kb * 2, t.b, keep);
                }
            }
            grid_dependents_launch();
            // every load issued into the pair has landed before it ends
            if (rank == 0) {
                for (uint32_t s = 0; s < kOrthoStages; ++s) {
                    if (armed <= s) break;
                    if (!mbar_wait(&full[s], ((armed - 1 - s) / kOrthoStages) & 1u, p.wait_limit_ns))
                        ortho_give_up(p, &abort_flag);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            uint32_t used = 0, acc_i = 0;
            bool ok = true;
            const uint32_t base = smem_addr(smem);
            for (int32_t item = mine; item < items && ok; item += pairs, ++acc_i) {
                const uint32_t buf = acc_i & 1u;
                if (!ortho_wait<true>(&acc_empty[buf], ((acc_i >> 1) & 1u) ^ 1u, &abort_flag, p)) break;
                tc_fence_after_sync();
                for (int32_t kb = 0; kb < p.k_blocks; ++kb, ++used) {
                    const uint32_t s = used % kOrthoStages, round = used / kOrthoStages;
                    ok = ortho_wait(&full[s], round & 1u, &abort_flag, p);
                    if (!ok) break;
                    tc_fence_after_sync();
                    ortho_mma<MODE, true>(tmem + buf * 256u, base + s * kOrthoStage, kb == 0);
                    tc_commit_pair_multicast(&empty[s], 3);
                }
                if (ok) tc_commit_pair_multicast(&acc_full[buf], 3);
            }
            // all MMAs issued have completed, also when the loop was left early
            tc_commit_pair(drain);
            if (!mbar_wait(drain, 0, p.wait_limit_ns)) ortho_give_up(p, &abort_flag);
        }
    } else {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        uint32_t acc_i = 0;
        for (int32_t item = mine; item < items; item += pairs, ++acc_i) {
            const OrthoTile t = ortho_tile<MODE>(p, item);
            const uint32_t buf = acc_i & 1u;
            const int32_t row = t.i * 256 + static_cast<int32_t>(rank) * 128 + quarter * 32 + lane;
            if (!ortho_wait(&acc_full[buf], (acc_i >> 1) & 1u, &abort_flag, p)) break;
            tc_fence_after_sync();
            const uint32_t taddr = tmem + buf * 256u + (static_cast<uint32_t>(quarter * 32) << 16);
            #pragma unroll 1
            for (int c = half * 128; c < half * 128 + 128; c += 32) {
                __syncwarp();
                const int32_t col = t.j * 256 + c;
                OrthoIn<MODE> in[2];
                #pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (ortho_inside<MODE>(p, row, col + 16 * q)) in[q] = ortho_read<MODE>(p, t.b, row, col + 16 * q);
                uint32_t r[32];
                tmem_ld_32x32b_x32(taddr + c, r);
                tmem_ld_wait();
                #pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (!ortho_inside<MODE>(p, row, col + 16 * q)) continue;
                    float v[16];
                    #pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(r[16 * q + k]);
                    ortho_finish<MODE>(p, t.b, row, col + 16 * q, in[q], v, kSym && t.i != t.j);
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_addr(&acc_empty[buf]), 0));
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();                                   // the peer is through with our memory
    tc_fence_after_sync();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ------------------------------------------------------- one tile per cluster

template <int MODE>
__global__ void __launch_bounds__(kOrthoTileThreads, 1)
    ortho_tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ OrthoParams p) {
    constexpr bool kMN = MODE == kStep || MODE == kLast;
    constexpr bool kSym = MODE == kGram || MODE == kPoly;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOrthoStages * kOrthoStage);
    uint64_t* empty = full + kOrthoStages;
    uint64_t* done = empty + kOrthoStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    __shared__ volatile int abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t S = p.splits;
    const uint32_t rank = S > 1 ? cluster_ctarank() : 0u;
    const OrthoTile t = ortho_tile<MODE>(p, static_cast<int32_t>(blockIdx.x) / S);
    const int32_t kb0 = static_cast<int32_t>(rank) * p.k_blocks / S;
    const int32_t kb1 = static_cast<int32_t>(rank + 1) * p.k_blocks / S;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < kOrthoStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        fence_barrier_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 128);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();
    grid_dependents_launch();

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t keep = l2_policy_evict_last();
            uint32_t armed = 0;
            for (int32_t kb = kb0; kb < kb1; ++kb, ++armed) {
                const uint32_t s = armed % kOrthoStages, round = armed / kOrthoStages;
                if (!ortho_wait(&empty[s], (round & 1u) ^ 1u, &abort_flag, p)) break;
                uint8_t* sa = smem + s * kOrthoStage;
                mbar_arrive_expect_tx(&full[s], kOrthoStage);
                if ((p.debug_flags & 1u) && armed == 0 && blockIdx.x == 0) continue;   // test hook: no load
                tma_load_4d(sa, &tmA, &full[s], 0, t.i * 128, kb * 2, t.b, keep);
                if constexpr (kMN) tma_load_4d(sa + kOrthoBox, &tmB, &full[s], 0, kb * 128, t.j * 2, t.b, keep);
                else tma_load_4d(sa + kOrthoBox, &tmB, &full[s], 0, t.j * 128, kb * 2, t.b, keep);
            }
            // every load has landed before the memory is written again or the CTA ends
            for (uint32_t s = 0; s < kOrthoStages; ++s) {
                if (armed <= s) break;
                if (!mbar_wait(&full[s], ((armed - 1 - s) / kOrthoStages) & 1u, p.wait_limit_ns))
                    ortho_give_up(p, &abort_flag);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t used = 0;
            const uint32_t base = smem_addr(smem);
            for (int32_t kb = kb0; kb < kb1; ++kb, ++used) {
                const uint32_t s = used % kOrthoStages, round = used / kOrthoStages;
                if (!ortho_wait(&full[s], round & 1u, &abort_flag, p)) break;
                tc_fence_after_sync();
                ortho_mma<MODE, false>(tmem, base + s * kOrthoStage, used == 0);
                tc_commit(&empty[s]);
            }
            tc_commit(done);
            if (!mbar_wait(done, 0, p.wait_limit_ns)) ortho_give_up(p, &abort_flag);
        }
    }
    // Every CTA of the cluster is through with its stages: their memory becomes the
    // exchange buffer [source][four columns of mine][row] of float4s.
    tc_fence_before_sync();
    __syncthreads();
    if (S > 1) cluster_sync_all();
    tc_fence_after_sync();
    const int quarter = warp & 3;
    const int r_in = quarter * 32 + lane;
    const int32_t row = t.i * 128 + r_in;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    if (S > 1) {
        const int32_t log4 = p.log_width - 2;                // log2 of the fours of columns each CTA finishes
        float4* xbuf = reinterpret_cast<float4*>(smem);
        if (warp >= 2) {
            const bool any = kb1 > kb0;                      // (a CTA without a K block adds zeros)
            #pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(taddr + c, r);
                tmem_ld_wait();
                #pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const int32_t c4 = (c + j) >> 2;
                    const uint32_t q = static_cast<uint32_t>(c4 >> log4);
                    float4* at = xbuf + ((static_cast<int32_t>(rank) << log4) + (c4 & ((1 << log4) - 1))) * 128 + r_in;
                    const float4 v = any ? make_float4(__uint_as_float(r[j]), __uint_as_float(r[j + 1]),
                                                       __uint_as_float(r[j + 2]), __uint_as_float(r[j + 3]))
                                         : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (q == rank) *at = v;
                    else
                        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         map_to_rank(smem_addr(at), q)),
                                     "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                                     : "memory");
                }
            }
        }
        __syncthreads();
        cluster_sync_all();
        if (warp >= 2 && !abort_flag) {
            const int32_t col0 = t.j * 128 + (static_cast<int32_t>(rank) << p.log_width);
            #pragma unroll 1
            for (int32_t u = 0; u < (1 << p.log_width) / 16; ++u) {
                const int32_t col = col0 + u * 16;
                if (!ortho_inside<MODE>(p, row, col)) continue;
                const OrthoIn<MODE> in = ortho_read<MODE>(p, t.b, row, col);
                float v[16];
                #pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = 0.0f;
                #pragma unroll 2
                for (int32_t s = 0; s < S; ++s) {
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 f = xbuf[((s << log4) + u * 4 + q) * 128 + r_in];
                        v[4 * q] += f.x, v[4 * q + 1] += f.y, v[4 * q + 2] += f.z, v[4 * q + 3] += f.w;
                    }
                }
                ortho_finish<MODE>(p, t.b, row, col, in, v, kSym && t.i != t.j);
            }
        }
    } else if (warp >= 2 && !abort_flag) {
        #pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
            __syncwarp();
            const int32_t col = t.j * 128 + c;
            OrthoIn<MODE> in[2];
            #pragma unroll
            for (int q = 0; q < 2; ++q)
                if (ortho_inside<MODE>(p, row, col + 16 * q)) in[q] = ortho_read<MODE>(p, t.b, row, col + 16 * q);
            uint32_t r[32];
            tmem_ld_32x32b_x32(taddr + c, r);
            tmem_ld_wait();
            #pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (!ortho_inside<MODE>(p, row, col + 16 * q)) continue;
                float v[16];
                #pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(r[16 * q + k]);
                ortho_finish<MODE>(p, t.b, row, col + 16 * q, in[q], v, kSym && t.i != t.j);
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 1) tmem_dealloc(tmem, 128);
}

}  // namespace gemm103
