// glu_skinny.cuh -- the gated linear layer of up to 128 tokens
// (include/glu_sm103.h): a weight-streaming kernel.
//
// Swapped as the GEMM's skinny path is: the weights fill the tensor core's 128
// rows (64 of the gate, the same 64 of the up projection), the tokens are the
// MMA's N (16, 32, 64 or 128).  What differs is the split of K.  A problem of few
// tiles is split over the S CTAs of a cluster, each streaming its own range of
// K, and the sums meet through distributed shared memory: every CTA sends each
// other one the columns (tokens) which that one finishes, one exchange of 64 KB
// at most and two cluster barriers, where stream-K goes through global memory,
// a counter and a second pass over tensor memory (4 to 5 us of a problem of
// 10).  Two CTAs share an SM, so one's set-up and epilogue hide behind the
// other's stream, and S = 1 suffices once there are about as many tiles as SMs:
// HBM, which bounds all of this, divides itself evenly over the CTAs.  W not in
// L2, one call after another: 16 tokens, 4096 -> 14336, 39.2 us, 6.0 TB/s; 4096 ->
// 4096, 14.0 us, 4.8 TB/s; 64 tokens, 2048 -> 10240, 23.0 us, 3.6 TB/s.  (Of more
// tokens and tiles the GEMM's persistent tiles are faster: glu_plan says where.)
#pragma once
#include <cstdint>
#include <cuda.h>

#include "epilogue_ops.cuh"
#include "f32x2.cuh"
#include "ptx.cuh"

namespace gemm103 {

constexpr int kSkinnyThreads = 192;      // warp 0 TMA, warp 1 MMA, warps 2-5 epilogue
constexpr uint32_t kSkinnyATile = 16384; // one K chunk of 128 rows

struct GluSkinnyParams {
    int32_t M, F;                        // tokens, output columns
    int32_t k_blocks;                    // of KC chunks
    int32_t splits;                      // CTAs per tile (the cluster's size): 1, 2, 4, 8, at most BN / 4
    int32_t log_per;                     // log2(BN / splits): tokens each CTA finishes
    uint32_t idesc;
    void* H; int64_t ldh;
    void* P; int64_t ldp;
    const void* bias;
    int32_t bias_dtype, act, h_dtype;
    int* err;
    uint64_t wait_limit_ns;
    uint32_t debug_flags;
};

template <int BN, int KC>
struct Skinny {
    static constexpr uint32_t kA = KC * kSkinnyATile;
    static constexpr uint32_t kStage = kA + KC * BN * 128u;
    static constexpr uint32_t kExchange = 128u * BN * 4u;
    // the exchange takes the stages' memory; stages for two CTAs per SM
    static constexpr int kStages = static_cast<int>((112u * 1024u - 2048u) / kStage);
    static constexpr uint32_t kSmem = (kStages * kStage > kExchange ? kStages * kStage : kExchange) + 1024u + 128u;
};

// Bounded wait that also gives up once another role has.
__device__ __forceinline__ bool skinny_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                            const GluSkinnyParams& p) {
    const uint32_t a = smem_addr(bar);
    if (mbar_try_wait(a, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(a, parity)) return true;
        if ((i & 63u) == 0 && (*abort_flag || global_timer_ns() - t0 > p.wait_limit_ns)) break;
    }
    *abort_flag = 1;
    if (p.err) atomicCAS(p.err, 0, 1);
    return false;
}

template <int BN, int KC>
__global__ void __launch_bounds__(kSkinnyThreads)
    glu_skinny_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                      const __grid_constant__ GluSkinnyParams p) {
    constexpr uint32_t kTmemCols = BN < 32 ? 32 : BN;
    using Cfg = Skinny<BN, KC>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* tail = smem + (Cfg::kSmem - 1024u - 128u);
    uint64_t* full = reinterpret_cast<uint64_t*>(tail);
    uint64_t* empty = full + Cfg::kStages;
    uint64_t* done = empty + Cfg::kStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    static_assert((2 * Cfg::kStages + 2) * 8 <= 128, "barriers fit behind the stages");
    __shared__ volatile int abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t S = p.splits;
    const uint32_t rank = S > 1 ? cluster_ctarank() : 0u;
    const int32_t tile = static_cast<int32_t>(blockIdx.x) / S;
    const int32_t kb0 = static_cast<int32_t>((static_cast<int64_t>(rank) * p.k_blocks) / S);
    const int32_t kb1 = static_cast<int32_t>((static_cast<int64_t>(rank + 1) * p.k_blocks) / S);

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < Cfg::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        fence_barrier_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();
    grid_dependents_launch();

    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            const uint64_t once = l2_policy_evict_first(), keep = l2_policy_evict_last();
            uint32_t armed = 0;
            for (int32_t kb = kb0; kb < kb1 && ok; ++kb, ++armed) {
                const uint32_t s = armed % Cfg::kStages, round = armed / Cfg::kStages;
                ok = skinny_wait(&empty[s], (round & 1u) ^ 1u, &abort_flag, p);
                if (!ok) break;
                uint8_t* a = smem + s * Cfg::kStage;
                mbar_arrive_expect_tx(&full[s], Cfg::kStage);
                if ((p.debug_flags & 1u) && armed == 0 && blockIdx.x == 0) continue;   // test hook: no load
                if constexpr (KC == 1) {
                    tma_load_3d(a, &tmW, &full[s], kb * 64, tile * 64, 0, once);
                    tma_load_2d(a + Cfg::kA, &tmX, &full[s], kb * 64, 0, keep);
                } else {
                    tma_load_4d(a, &tmW, &full[s], 0, tile * 64, 0, kb * KC, once);
                    tma_load_3d(a + Cfg::kA, &tmX, &full[s], 0, 0, kb * KC, keep);
                }
            }
            // wind-down: every load issued has landed before the memory is
            // written again (the exchange) or the CTA ends
            for (uint32_t s = 0; s < Cfg::kStages; ++s) {
                if (armed <= s) break;
                const uint32_t round = (armed - 1 - s) / Cfg::kStages;
                if (!mbar_wait(&full[s], round & 1u, p.wait_limit_ns)) {
                    abort_flag = 1;
                    if (p.err) atomicCAS(p.err, 0, 1);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t i = 0;
            const uint32_t base = smem_addr(smem);
            for (int32_t kb = kb0; kb < kb1; ++kb, ++i) {
                const uint32_t s = i % Cfg::kStages, round = i / Cfg::kStages;
                if (!skinny_wait(&full[s], round & 1u, &abort_flag, p)) break;
                tc_fence_after_sync();
                const uint32_t sa = base + s * Cfg::kStage, sb = sa + Cfg::kA;
                #pragma unroll
                for (int kk = 0; kk < KC * 4; ++kk) {
                    const uint64_t ad = smem_desc_sw128(sa + (kk >> 2) * kSkinnyATile + (kk & 3) * 32u, 16u, 1024);
                    const uint64_t bd = smem_desc_sw128(sb + (kk >> 2) * (BN * 128u) + (kk & 3) * 32u, 16u, 1024);
                    tc_mma_f16(tmem, ad, bd, p.idesc, (i > 0 || kk > 0) ? 1u : 0u);
                }
                tc_commit(&empty[s]);
            }
            // all MMAs issued have completed (also when the loop was left early)
            tc_commit(done);
            if (!mbar_wait(done, 0, p.wait_limit_ns)) {
                abort_flag = 1;
                if (p.err) atomicCAS(p.err, 0, 1);
            }
        }
    }
    // Every CTA of the cluster is through with its stages: their memory becomes
    // the exchange buffer [source rank][four tokens of mine][row], float4s of
    // four tokens: a warp's store and load are 512 contiguous bytes.
    tc_fence_before_sync();
    __syncthreads();
    if (S > 1) cluster_sync_all();
    tc_fence_after_sync();
    const int32_t per4 = 1 << (p.log_per - 2);       // fours of tokens each CTA finishes
    float4* xbuf = reinterpret_cast<float4*>(smem);
    if (warp >= 2) {
        const int quarter = warp & 3;
        const uint32_t row = quarter * 32 + lane;
        const bool any = kb1 > kb0;                  // (a CTA without a k-block adds zeros)
        #pragma unroll 1
        for (int c = 0; c < BN; c += 32) {
            if (c >= p.M) break;
            uint32_t r[32];
            tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c, r);
            tmem_ld_wait();
            #pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const int32_t t4 = (c + j) >> 2;
                if (c + j >= p.M || c + j >= BN) break;
                const uint32_t q = static_cast<uint32_t>(t4 >> (p.log_per - 2));
                float4* at = xbuf + (rank * per4 + (t4 & (per4 - 1))) * 128 + row;
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
    tc_fence_before_sync();
    __syncthreads();
    if (S > 1) cluster_sync_all();
    // This CTA's tokens: thread = output column (64 of them) and every third
    // (with warps 0 and 1: all 192 threads) four of tokens; the sources are
    // added in rank order.
    if (!abort_flag) {
        const int n_in = static_cast<int>(threadIdx.x) & 63;
        const int32_t n = tile * 64 + n_in;
        if (n < p.F) {
            float bg = 0.0f, bu = 0.0f;
            if (p.bias != nullptr) {
                bg = load_bias_elem(p.bias, p.bias_dtype, n);
                bu = load_bias_elem(p.bias, p.bias_dtype, static_cast<int64_t>(p.F) + n);
            }
            for (int32_t i = static_cast<int32_t>(threadIdx.x) >> 6; i < per4; i += kSkinnyThreads / 64) {
                const int64_t t = (static_cast<int64_t>(rank) * per4 + i) * 4;
                if (t >= p.M) break;
                float g[4] = {bg, bg, bg, bg}, u[4] = {bu, bu, bu, bu};
                #pragma unroll 2
                for (int32_t s = 0; s < S; ++s) {
                    const float4* src = xbuf + (s * per4 + i) * 128 + n_in;
                    const float4 a = src[0], b = src[64];
                    g[0] += a.x; g[1] += a.y; g[2] += a.z; g[3] += a.w;
                    u[0] += b.x; u[1] += b.y; u[2] += b.z; u[3] += b.w;
                }
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (t + k >= p.M) break;
                    if (p.P != nullptr) {
                        store_elem(p.P, p.h_dtype, (t + k) * p.ldp + n, g[k]);
                        store_elem(p.P, p.h_dtype, (t + k) * p.ldp + p.F + n, u[k]);
                    }
                    store_elem(p.H, p.h_dtype, (t + k) * p.ldh + n, activate(p.act, g[k]) * u[k]);
                }
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace gemm103
