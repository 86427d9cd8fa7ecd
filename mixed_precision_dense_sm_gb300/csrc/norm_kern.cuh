// norm_kern.cuh -- the norms before and after a block, fused with its gate,
// residual scale and residual add (include/norm_sm103.h): forward and
// backward row kernels, and the backward's sum over rows.
//
// Each matrix element is read once and written once.  A row belongs to a group
// of T threads of a CTA (a warp for narrow rows, the whole CTA for wide ones);
// each thread owns C chunks of 8 elements.  A thread copies its own elements of
// the next row to shared memory with cp.async while the group works on the
// current one, into a ring of slots that only this thread reads: no barrier
// guards the copies, and no registers hold loads in flight.  What the group
// shares are the sums of a row: halving in each warp, one shared-memory
// exchange, one barrier.  A CTA takes a chunk of consecutive rows that see the
// same row of the gate, so the weights, the gate and the scale fold into
// vectors that it converts to FP32 in shared memory once.
//
// 8192 x 4096 bf16, RMSNorm on both sides, a gate per channel.  Forward: 49 us,
// 5.4 TB/s; issue slots 57 % and DRAM 61 % busy.  Backward: 72 us and 6 for the
// sums, 5.2 TB/s; bound by its instructions, 39 per element (16-bit pairs are
// unpacked again in each of its passes over a row), and the latency of shared
// memory at the 16 warps per SM that its registers leave: issue slots 47 %
// busy.  One exchange per row in place of two (the post-norm's sums, from
// products known before the pre-norm's size) costs more products than it saves:
// 93 us for 84, both without the kinds compiled in.
//
// Rows that are not 16-byte aligned, or N not a multiple of 8, go element by
// element: a thread's 8 elements are then 32 apart, so a warp's accesses stay
// contiguous.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "f32x2.cuh"
#include "ptx.cuh"

namespace gemm103 {
namespace nrm {

enum : int { kNone = 0, kRms = 1, kLayer = 2 };
constexpr int kMaxStages = 3;
// What a kernel has compiled in: the norms on both sides, that every matrix is
// there and that the gate is not per token (or nothing of this).  Fewer
// instructions and longer runs of them without a branch: 8192 x 4096 bf16,
// RMSNorm on both sides, backward, 84 us not compiled in, 76 compiled in.
enum : int { kAnyKind = 0, kRmsRms = 1, kRmsPlain = 2, kLayerLayer = 3, kLayerPlain = 4 };
__host__ __device__ constexpr int kind_pre(int kind) { return kind <= kRmsPlain ? kRms : kLayer; }
__host__ __device__ constexpr int kind_post(int kind) {
    return kind == kRmsRms ? kRms : kind == kLayerLayer ? kLayer : kNone;
}
constexpr int kBackThreads = 512;    // of a backward CTA: 128 registers each, one CTA per SM

struct Params {
    // forward: X, Z in, XO, Y out; backward: X = XO, Z, dY, dXO in, dX, dZ out
    const void* X; int64_t ldx;
    const void* Z; int64_t ldz;
    void* XO; int64_t ldxo;
    void* Y; int64_t ldy;
    const void* dY; int64_t lddy;
    const void* dXO; int64_t lddxo;
    void* dX; int64_t lddx;
    void* dZ; int64_t lddz;
    const void* wpre; const void* bpre; const void* wpost; const void* bpost;
    const void* gate; int64_t ld_gate;
    int32_t vec_dtype;
    int32_t vec_aligned;        // weights, biases and gate rows are 16-byte aligned
    int32_t vec;                // rows are 16-byte aligned and N a multiple of 8
    int32_t pre, post;
    float scale, eps, inv_n;
    int64_t M;
    int32_t N;
    int32_t T;                  // threads per row
    int32_t stages;             // slots of the ring
    uint32_t slot_bytes;        // of one row of one group
    // Row-invariant vectors, kept in shared memory as FP32 (their numbers
    // there, -1 where absent): ws multiplies the post-norm (scale gate wpost,
    // or wpost for token gates), bs is added to it (scale gate bpost, or bpost)
    int32_t i_ws, i_bs, i_wpre, i_bpre, n_par;
    // rows are cut into chunks, one CTA (or pair) each, that lie in one group
    // of the gate (token gates, gate_rows == 1, count as one group)
    int64_t chunk_group_rows;   // rows of a gate group (M where rows do not share one)
    int32_t chunks_per_group;
    int64_t chunk_rows;
    int32_t token_gate;         // the gate's row changes with every row
    int32_t cluster;            // CTAs that share a row (1 or 2), each half its columns
    // backward
    float* partials;            // [4][chunks][N]: sums of dY xhat, q zhat, dY, q (the last two: BIAS)
    int64_t part_stride;        // chunks * N
    void* dgate;                // written directly for token gates
    int32_t grad_dtype;
};

// ------------------------------------------------------------------ elements

// 8 consecutive or strided elements as 4 pairs.
typedef F2 F8[4];

__device__ __forceinline__ void set8(F8& o, float x) {
    #pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = mk2(x);
}

__device__ __forceinline__ void set8(F8& o, float4 a, float4 b) {
    o[0] = mk2(a.x, a.y);
    o[1] = mk2(a.z, a.w);
    o[2] = mk2(b.x, b.y);
    o[3] = mk2(b.z, b.w);
}
__device__ __forceinline__ float4 join2(F2 a, F2 b) {
    float4 r;
    get2(a, r.x, r.y);
    get2(b, r.z, r.w);
    return r;
}

// Where a thread's 8 elements of chunk c lie in the row: element e at
// base + e with VEC (all 8 of them inside the row or none), else at
// base + 32 e.
template <bool VEC>
struct Spot {
    int32_t base;
    __device__ __forceinline__ int32_t at(int e) const { return VEC ? base + e : base + 32 * e; }
    __device__ __forceinline__ bool in(int e, int32_t N) const { return VEC ? base < N : at(e) < N; }
    // whether there is anything to do for the chunk
    __device__ __forceinline__ bool some(int32_t N) const { return base < N; }
};

template <bool VEC>
__device__ __forceinline__ Spot<VEC> spot_of(int T, int t, int c, int32_t first = 0) {
    return {first + (VEC ? (c * T + t) * 8 : (c * T + (t & ~31)) * 8 + (t & 31))};
}

// 8 elements of a vector parameter (weight, bias, gate row) of type dtype; 0
// past column N.
template <bool VEC>
__device__ __forceinline__ void load_param8(const void* v, int32_t dtype, bool wide, Spot<VEC> s,
                                            int32_t N, F8& o) {
    if (VEC && wide) {
        if (dtype == 2) {
            const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(v) + s.base);
            set8(o, p[0], p[1]);
        } else {
            const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(v) + s.base);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
            #pragma unroll
            for (int q = 0; q < 4; ++q)
                o[q] = dtype == 1 ? unpack2<__nv_bfloat16>(w[q]) : unpack2<__half>(w[q]);
        }
        return;
    }
    float f[8];
    if (dtype == 2) {
        #pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = s.in(e, N) ? static_cast<const float*>(v)[s.at(e)] : 0.0f;
    } else {
        uint16_t u[8];
        #pragma unroll
        for (int e = 0; e < 8; ++e)
            u[e] = s.in(e, N) ? static_cast<const uint16_t*>(v)[s.at(e)] : static_cast<uint16_t>(0);
        #pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = dtype == 1 ? __bfloat162float(__ushort_as_bfloat16(u[e])) : __half2float(__ushort_as_half(u[e]));
    }
    #pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = mk2(f[2 * q], f[2 * q + 1]);
}

// o *= parameter, where there is one.
template <bool VEC>
__device__ __forceinline__ void scale_by(F8& o, const void* v, int32_t dtype, bool wide, Spot<VEC> s,
                                         int32_t N) {
    if (v == nullptr) return;
    F8 w;
    load_param8<VEC>(v, dtype, wide, s, N, w);
    #pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = mul2(o[q], w[q]);
}

// Elements past column N as 0 (a chunk with VEC has none).
template <bool VEC>
__device__ __forceinline__ void mask8(F8& o, Spot<VEC> s, int32_t N) {
    if constexpr (!VEC) {
        #pragma unroll
        for (int q = 0; q < 4; ++q) {
            float lo, hi;
            get2(o[q], lo, hi);
            o[q] = mk2(s.in(2 * q, N) ? lo : 0.0f, s.in(2 * q + 1, N) ? hi : 0.0f);
        }
    }
}

// o - mean, 0 past column N.
template <bool VEC>
__device__ __forceinline__ void center8(F8& o, float mean, Spot<VEC> s, int32_t N) {
    #pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = add2(o[q], mk2(-mean));
    mask8<VEC>(o, s, N);
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// Waits until at most `n` of this thread's copy groups are in flight.
__device__ __forceinline__ void cp_async_wait(int n) {
    switch (n) {
        case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    }
}

// A thread's chunk c in a slot: 8 elements, 16-byte pieces strided by the
// group's threads so that a warp's accesses are contiguous.
template <typename E>
__device__ __forceinline__ uint8_t* slot_at(uint8_t* slot, int T, int t, int c) {
    constexpr int kPieces = sizeof(E) / 2;            // 16-byte pieces per 8 elements
    return slot + (static_cast<uint32_t>(c * kPieces) * T + t) * 16u;
}

// Starts the copy of 8 elements of a row into this thread's part of a slot.
// Single 16-bit elements cannot be copied asynchronously: those are loaded by
// hold8 into registers while the previous row is worked on, and put8 writes
// them to the slot.
template <typename E, bool VEC>
__device__ __forceinline__ void fetch8(uint8_t* slot, int T, int t, int c, const E* row, Spot<VEC> s,
                                       int32_t N) {
    constexpr int kPieces = sizeof(E) / 2;
    uint8_t* d = slot_at<E>(slot, T, t, c);
    if constexpr (VEC) {
        if (s.base < N) {
            #pragma unroll
            for (int q = 0; q < kPieces; ++q)
                cp_async16(d + q * T * 16, row + s.base + q * (8 / kPieces));
        }
    } else if constexpr (sizeof(E) == 4) {
        // the elements past column N stay as they are: 0 (zero_ring)
        #pragma unroll
        for (int e = 0; e < 8; ++e)
            if (s.in(e, N)) cp_async4(d + (e / 4) * T * 16 + (e % 4) * 4, row + s.at(e));
    }
}

// 16-bit elements held in registers on the way to a slot (VEC false only).
template <typename E, bool VEC>
struct Held {
    static constexpr bool kUsed = !VEC && sizeof(E) == 2;
    uint32_t w[kUsed ? 4 : 1];
};

template <typename E, bool VEC>
__device__ __forceinline__ void hold8(Held<E, VEC>& h, const E* row, Spot<VEC> s, int32_t N) {
    if constexpr (Held<E, VEC>::kUsed) {
        const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
        #pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t lo = s.in(2 * q, N) ? r[s.at(2 * q)] : 0u;
            const uint32_t hi = s.in(2 * q + 1, N) ? r[s.at(2 * q + 1)] : 0u;
            h.w[q] = lo | hi << 16;
        }
    }
}

template <typename E, bool VEC>
__device__ __forceinline__ void put8(uint8_t* slot, int T, int t, int c, const Held<E, VEC>& h) {
    if constexpr (Held<E, VEC>::kUsed)
        *reinterpret_cast<uint4*>(slot_at<E>(slot, T, t, c)) = make_uint4(h.w[0], h.w[1], h.w[2], h.w[3]);
}

// This thread's parts of the group's ring as 0: what lies past column N in a
// chunk that has columns of the row is never copied and has to read as 0.
template <bool VEC>
__device__ __forceinline__ void zero_ring(uint8_t* ring, uint32_t bytes, int T, int t) {
    if constexpr (!VEC) {
        for (uint32_t i = t * 16u; i < bytes; i += T * 16u)
            *reinterpret_cast<uint4*>(ring + i) = make_uint4(0u, 0u, 0u, 0u);
    }
}

// The 8 elements of this thread's part of a slot as FP32.
template <typename E>
__device__ __forceinline__ void take8(uint8_t* slot, int T, int t, int c, F8& o) {
    const uint8_t* d = slot_at<E>(slot, T, t, c);
    if constexpr (sizeof(E) == 4) {
        set8(o, *reinterpret_cast<const float4*>(d), *reinterpret_cast<const float4*>(d + T * 16));
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(d);
        o[0] = unpack2<E>(u.x);
        o[1] = unpack2<E>(u.y);
        o[2] = unpack2<E>(u.z);
        o[3] = unpack2<E>(u.w);
    }
}

// Stores 8 elements rounded to E (the columns < N); with KEEP v becomes what
// was stored.
template <typename E, bool VEC, bool KEEP = false>
__device__ __forceinline__ void store8(E* row, Spot<VEC> s, int32_t N, F8& v) {
    if constexpr (sizeof(E) == 4) {
        if constexpr (VEC) {
            *reinterpret_cast<float4*>(row + s.base) = join2(v[0], v[1]);
            *reinterpret_cast<float4*>(row + s.base + 4) = join2(v[2], v[3]);
        } else {
            #pragma unroll
            for (int q = 0; q < 4; ++q) {
                float lo, hi;
                get2(v[q], lo, hi);
                if (s.in(2 * q, N)) row[s.at(2 * q)] = lo;
                if (s.in(2 * q + 1, N)) row[s.at(2 * q + 1)] = hi;
            }
        }
    } else {
        uint32_t w[4];
        #pragma unroll
        for (int q = 0; q < 4; ++q) {
            w[q] = pack2<E>(v[q]);
            if constexpr (KEEP) v[q] = unpack2<E>(w[q]);
        }
        if constexpr (VEC) {
            *reinterpret_cast<uint4*>(row + s.base) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            uint16_t* r = reinterpret_cast<uint16_t*>(row);
            #pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (s.in(2 * q, N)) r[s.at(2 * q)] = static_cast<uint16_t>(w[q] & 0xFFFFu);
                if (s.in(2 * q + 1, N)) r[s.at(2 * q + 1)] = static_cast<uint16_t>(w[q] >> 16);
            }
        }
    }
}

// The group of threads that shares a row: T threads of the CTA (a compile-time
// number for TT > 0); KR: the most values summed together.
template <int TT, int KR>
struct Group {
    static constexpr int kMost = KR;
    int T_, t, index;           // threads, this thread's number, the group's number
    float* red;                 // [2][KR][warps] exchange buffer of this group
    int parity;
    float* pair;                // [2][2][KR] exchange buffer of a CTA pair, or NULL
    uint32_t rank;              // this CTA's number in the pair
    __device__ __forceinline__ int T() const { return TT > 0 ? TT : T_; }
    __device__ __forceinline__ int warps() const { return T() >> 5; }
};

template <class G>
__device__ __forceinline__ void group_barrier(const G& g) {
    asm volatile("bar.sync %0, %1;" ::"r"(g.index + 1), "r"(g.T()) : "memory");
}

// Sums of v[0..K) over a warp by halving: at each step a lane keeps one half of
// the values it still has (the upper half where its bit is set) and gives the
// other away, so K values take about K + 3 exchanges instead of 5 K.  The lane
// ends with the sum of value warp_slot<K>(lane) in v[0].
template <int K, int O = 16, int L>
__device__ __forceinline__ void warp_halve(float (&v)[L], int lane) {
    constexpr int H = (K + 1) / 2;
    if constexpr (K > 1) {
        const bool up = (lane & O) != 0;
        #pragma unroll
        for (int k = 0; k < H; ++k) {
            const float hi = k + H < K ? v[k + H] : 0.0f;
            const float give = up ? v[k] : hi;
            v[k] = (up ? hi : v[k]) + __shfl_xor_sync(0xffffffffu, give, O);
        }
    } else {
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], O);
    }
    if constexpr (O > 1) warp_halve<H, O / 2>(v, lane);
}
// Number of the value that a lane ends with, -1 for none.
template <int K>
__host__ __device__ constexpr int warp_slot(int lane) {
    int first = 0, count = K, held = K;
    for (int o = 16; o > 0; o >>= 1) {
        if (held <= 1) break;
        const int h = (held + 1) / 2;
        if (lane & o) {
            first += h;
            count -= h;
        } else if (count > h) {
            count = h;
        }
        held = h;
    }
    return count > 0 ? first : -1;
}
// Lanes that end with each value.
template <int K>
struct WarpLanes {
    int at[K];
    bool all;
    __host__ __device__ constexpr WarpLanes() : at{}, all(true) {
        for (int k = 0; k < K; ++k) {
            at[k] = -1;
            for (int l = 31; l >= 0; --l)
                if (warp_slot<K>(l) == k) at[k] = l;
            all = all && at[k] >= 0;
        }
    }
};

// Sums of K values over the group, in the same order on every run; every
// thread gets them.  One barrier: consecutive sums use alternate buffers.
template <int K, class G>
__device__ __forceinline__ void group_sum(G& g, float (&v)[K]) {
    constexpr WarpLanes<K> lanes;
    static_assert(K <= G::kMost, "exchange buffer");
    static_assert(lanes.all, "every value ends somewhere");
    const int lane = static_cast<int>(threadIdx.x) & 31;
    warp_halve<K>(v, lane);
    if (g.T() == 32) {
        if constexpr (K > 1) {
            const float mine = v[0];
            #pragma unroll
            for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, mine, lanes.at[k]);
        }
        return;
    }
    float* r = g.red + g.parity * g.warps() * G::kMost;
    g.parity ^= 1;
    // (lanes that end with the same value write the same bits)
    const int slot = warp_slot<K>(lane);
    if (slot >= 0) r[slot * g.warps() + (g.t >> 5)] = v[0];
    group_barrier(g);
    #pragma unroll
    for (int k = 0; k < K; ++k) {
        const float* q = r + k * g.warps();
        if (g.warps() == 2) {
            v[k] = q[0] + q[1];
        } else {
            v[k] = 0.0f;
            #pragma unroll
            for (int w = 0; w < g.warps(); w += 4) {    // a multiple of 4
                const float4 x = *reinterpret_cast<const float4*>(q + w);
                v[k] += (x.x + x.y) + (x.z + x.w);
            }
        }
    }
    if (g.pair == nullptr) return;
    // the other half of the row: each CTA leaves its sums in both CTAs' shared
    // memory, and both add them in rank order.  The buffer of this parity is
    // written again only two sums on, behind the next sum's cluster barrier.
    float* x = g.pair + (g.parity * 2 + g.rank) * G::kMost;
    if (g.t == 0) {
        const uint32_t peer = map_to_rank(smem_addr(x), g.rank ^ 1u);
        #pragma unroll
        for (int k = 0; k < K; ++k) {
            x[k] = v[k];
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(peer + 4u * k), "f"(v[k])
                         : "memory");
        }
    }
    cluster_sync_all();
    const float* y = g.pair + g.parity * 2 * G::kMost;
    #pragma unroll
    for (int k = 0; k < K; ++k) v[k] = y[k] + y[G::kMost + k];
}

constexpr int kForwardSums = 4, kBackwardSums = 4;

template <class G>
__device__ __forceinline__ G make_group(const Params& p, uint8_t* smem) {
    G g;
    g.T_ = p.T;
    g.index = static_cast<int>(threadIdx.x) / g.T();
    g.t = static_cast<int>(threadIdx.x) - g.index * g.T();
    g.red = reinterpret_cast<float*>(smem) + g.index * (2 * G::kMost * g.warps());
    g.parity = 0;
    g.pair = nullptr;
    g.rank = 0;
    return g;
}

// The rows of chunk `b`: [row0, row1) inside one group of the gate.
__device__ __forceinline__ void chunk_span(const Params& p, int64_t b, int64_t& row0, int64_t& row1,
                                           int64_t& group) {
    group = b / p.chunks_per_group;
    const int64_t base = group * p.chunk_group_rows;
    int64_t end = base + p.chunk_group_rows;
    if (end > p.M) end = p.M;
    row0 = base + (b - group * p.chunks_per_group) * p.chunk_rows;
    row1 = row0 + p.chunk_rows;
    if (row1 > end) row1 = end;
}

__device__ __forceinline__ const void* gate_row(const Params& p, int64_t row) {
    return static_cast<const uint8_t*>(p.gate) + row * p.ld_gate * (p.vec_dtype == 2 ? 4 : 2);
}

// This thread's part of vector k in shared memory: as a slot of FP32 elements.
template <int C>
__device__ __forceinline__ uint8_t* par_at(uint8_t* par, int k, int T) {
    return par + static_cast<uint32_t>(k) * (C * 32u) * T;
}

// Fills the vectors in shared memory; every group reads them, the group
// numbered 0 writes them.
template <int C, bool VEC, class G>
__device__ __forceinline__ void fill_vectors(const Params& p, const G& g, uint8_t* par,
                                             int64_t group, int32_t col0) {
    if (g.index == 0) {
        const bool wide = p.vec_aligned != 0;
        #pragma unroll 1
        for (int c = 0; c < C; ++c) {
            const Spot<VEC> sp = spot_of<VEC>(g.T(), g.t, c, col0);
            if (!sp.some(p.N)) continue;
            auto put = [&](int k, const F8& v) {
                uint8_t* d = slot_at<float>(par_at<C>(par, k, g.T()), g.T(), g.t, c);
                *reinterpret_cast<float4*>(d) = join2(v[0], v[1]);
                *reinterpret_cast<float4*>(d + g.T() * 16) = join2(v[2], v[3]);
            };
            F8 gs, v;                               // scale * gate
            set8(gs, p.token_gate ? 1.0f : p.scale);
            if (p.gate != nullptr && !p.token_gate)
                scale_by<VEC>(gs, gate_row(p, group), p.vec_dtype, wide, sp, p.N);
            if (p.i_ws >= 0) {
                #pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = gs[q];
                scale_by<VEC>(v, p.wpost, p.vec_dtype, wide, sp, p.N);
                put(p.i_ws, v);
            }
            if (p.i_bs >= 0) {
                load_param8<VEC>(p.bpost, p.vec_dtype, wide, sp, p.N, v);
                #pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = mul2(v[q], gs[q]);
                put(p.i_bs, v);
            }
            if (p.i_wpre >= 0) {
                set8(v, 1.0f);
                scale_by<VEC>(v, p.wpre, p.vec_dtype, wide, sp, p.N);
                put(p.i_wpre, v);
            }
            if (p.i_bpre >= 0) {
                load_param8<VEC>(p.bpre, p.vec_dtype, wide, sp, p.N, v);
                put(p.i_bpre, v);
            }
        }
    }
    __syncthreads();
}

// 1 / sqrt(mean + eps): the hardware's approximation and one Newton step.
__device__ __forceinline__ float inv_size(float sum, const Params& p) {
    const float a = fmaf(sum, p.inv_n, p.eps);
    const float r = rsqrtf(a);
    return a < 3e38f ? r * fmaf(-0.5f * a * r, r, 1.5f) : r;     // (0 for infinity)
}

// ------------------------------------------------------------------- forward

// 1 / size of a row whose chunks are in v; v becomes v - mean for LayerNorm.
template <int C, bool VEC, class G>
__device__ __forceinline__ float norm_stats(G& g, const Params& p, int kind, int32_t col0,
                                            F8 (&v)[C]) {
    if (kind == kNone) return 1.0f;
    if (kind == kLayer) {
        F2 a = mk2(0.0f);
        #pragma unroll
        for (int c = 0; c < C; ++c)
            if (spot_of<VEC>(g.T(), g.t, c, col0).some(p.N)) {
                #pragma unroll
                for (int q = 0; q < 4; ++q) a = add2(a, v[c][q]);
            }
        float s[1] = {sum2(a)};
        group_sum(g, s);
        const float mean = s[0] * p.inv_n;
        #pragma unroll
        for (int c = 0; c < C; ++c) center8<VEC>(v[c], mean, spot_of<VEC>(g.T(), g.t, c, col0), p.N);
    }
    F2 a = mk2(0.0f);
    #pragma unroll
    for (int c = 0; c < C; ++c)
        if (spot_of<VEC>(g.T(), g.t, c, col0).some(p.N)) {
            #pragma unroll
            for (int q = 0; q < 4; ++q) a = fma2(v[c][q], v[c][q], a);
        }
    float s[1] = {sum2(a)};
    group_sum(g, s);
    return inv_size(s[0], p);
}

// One CTA (or a pair, for rows wider than kMaxColumnsPerCta) per chunk of rows,
// its groups taking the rows in turn.  (The bound of one CTA per SM keeps the
// compiler from spilling the narrowest rows' kernel to 32 registers: 33.5M bf16
// elements, N = 128, LayerNorm before 73 us without it and 59 with.  The others
// are left without: N = 5120 FP32, LayerNorm on both sides, 109 without, 150 with.)
template <typename XT, typename ZT, int TT, int C, bool VEC, int KIND>
__global__ void __launch_bounds__(1024, TT == 32 && C == 1 ? 1 : 0)
    forward_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(16) uint8_t smem[];
    auto g = make_group<Group<TT, kForwardSums>>(p, smem);
    const int T = g.T(), t = g.t;
    const int groups = static_cast<int>(blockDim.x) / T;
    uint8_t* par = smem + groups * g.warps() * (8 * kForwardSums);
    uint8_t* ring = par_at<C>(par, p.n_par, T) + static_cast<uint32_t>(g.index) * p.stages * p.slot_bytes;
    const uint32_t x_bytes = static_cast<uint32_t>(C) * 8u * sizeof(XT) * T;
    constexpr bool kAll = KIND != kAnyKind;
    constexpr bool kBiases = kAll && kind_pre(KIND) == kLayer;
    const bool has_z = kAll || p.Z != nullptr, has_y = kAll || p.Y != nullptr;
    const bool has_bs = kAll ? kBiases && kind_post(KIND) == kLayer : p.i_bs >= 0;
    const bool has_bpre = kAll ? kBiases : p.i_bpre >= 0;
    const bool token_gate = !kAll && p.token_gate;
    const int pre = kAll ? kind_pre(KIND) : p.pre, post = kAll ? kind_post(KIND) : p.post;
    const int32_t N = p.N;
    __shared__ float pair[4 * kForwardSums];
    int32_t col0 = 0;
    int64_t chunk = blockIdx.x;
    if (p.cluster == 2) {
        g.rank = cluster_ctarank();
        g.pair = pair;
        col0 = static_cast<int32_t>(g.rank) * T * C * 8;
        chunk >>= 1;
    }
    int64_t row0, row1, group;
    chunk_span(p, chunk, row0, row1, group);
    zero_ring<VEC>(ring, p.stages * p.slot_bytes, T, t);
    if (p.cluster == 2) cluster_sync_all();     // the other CTA's shared memory is there
    grid_dependency_wait();
    grid_dependents_launch();

    auto fetch = [&](int64_t row, int slot) {
        if (row < row1) {
            uint8_t* s = ring + static_cast<uint32_t>(slot) * p.slot_bytes;
            #pragma unroll
            for (int c = 0; c < C; ++c) {
                const Spot<VEC> sp = spot_of<VEC>(T, t, c, col0);
                fetch8<XT, VEC>(s, T, t, c, static_cast<const XT*>(p.X) + row * p.ldx, sp, N);
                if (has_z)
                    fetch8<ZT, VEC>(s + x_bytes, T, t, c,
                                    static_cast<const ZT*>(p.Z) + row * p.ldz, sp, N);
            }
        }
        cp_async_commit();
    };
    Held<XT, VEC> hx[C];
    Held<ZT, VEC> hz[C];
    auto hold = [&](int64_t row) {
        if (row >= row1) return;
        #pragma unroll
        for (int c = 0; c < C; ++c) {
            const Spot<VEC> sp = spot_of<VEC>(T, t, c, col0);
            hold8<XT, VEC>(hx[c], static_cast<const XT*>(p.X) + row * p.ldx, sp, N);
            if (has_z) hold8<ZT, VEC>(hz[c], static_cast<const ZT*>(p.Z) + row * p.ldz, sp, N);
        }
    };
    const int64_t first = row0 + g.index;
    for (int s = 0; s < p.stages - 1; ++s) fetch(first + static_cast<int64_t>(s) * groups, s);
    if constexpr (!VEC) hold(first);
    fill_vectors<C, VEC>(p, g, par, group, col0);
    int slot = 0;
    for (int64_t row = first; row < row1; row += groups) {
        if constexpr (!VEC) {
            uint8_t* s = ring + static_cast<uint32_t>(slot) * p.slot_bytes;
            #pragma unroll
            for (int c = 0; c < C; ++c) {
                put8<XT, VEC>(s, T, t, c, hx[c]);
                if (has_z) put8<ZT, VEC>(s + x_bytes, T, t, c, hz[c]);
            }
            hold(row + groups);
        }
        {
            int ahead = slot + p.stages - 1;
            if (ahead >= p.stages) ahead -= p.stages;
            fetch(row + static_cast<int64_t>(p.stages - 1) * groups, ahead);
        }
        cp_async_wait(p.stages - 1);
        uint8_t* s = ring + static_cast<uint32_t>(slot) * p.slot_bytes;
        if (++slot == p.stages) slot = 0;

        F8 x[C];
        if (has_z) {
            F8 z[C];
            #pragma unroll
            for (int c = 0; c < C; ++c) take8<ZT>(s + x_bytes, T, t, c, z[c]);
            const F2 r = mk2(norm_stats<C, VEC>(g, p, post, col0, z));
            #pragma unroll
            for (int c = 0; c < C; ++c) {
                const Spot<VEC> sp = spot_of<VEC>(T, t, c, col0);
                if (!sp.some(N)) continue;
                F8 w;
                take8<XT>(s, T, t, c, x[c]);
                take8<float>(par_at<C>(par, p.i_ws, T), T, t, c, w);
                #pragma unroll
                for (int q = 0; q < 4; ++q) z[c][q] = mul2(mul2(z[c][q], r), w[q]);
                if (has_bs) {
                    take8<float>(par_at<C>(par, p.i_bs, T), T, t, c, w);
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) z[c][q] = add2(z[c][q], w[q]);
                }
                if (token_gate) {
                    load_param8<VEC>(gate_row(p, row), p.vec_dtype, p.vec_aligned != 0, sp, N, w);
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) z[c][q] = mul2(z[c][q], mul2(w[q], mk2(p.scale)));
                }
                #pragma unroll
                for (int q = 0; q < 4; ++q) x[c][q] = add2(x[c][q], z[c][q]);
                // the stream as its type holds it: what is stored is what the
                // next norm sees
                store8<XT, VEC, true>(static_cast<XT*>(p.XO) + row * p.ldxo, sp, N, x[c]);
            }
        } else {
            #pragma unroll
            for (int c = 0; c < C; ++c) take8<XT>(s, T, t, c, x[c]);
        }
        if (has_y) {
            const F2 r = mk2(norm_stats<C, VEC>(g, p, pre, col0, x));
            #pragma unroll
            for (int c = 0; c < C; ++c) {
                const Spot<VEC> sp = spot_of<VEC>(T, t, c, col0);
                if (!sp.some(N)) continue;
                F8 w;
                take8<float>(par_at<C>(par, p.i_wpre, T), T, t, c, w);
                #pragma unroll
                for (int q = 0; q < 4; ++q) x[c][q] = mul2(mul2(x[c][q], r), w[q]);
                if (has_bpre) {
                    take8<float>(par_at<C>(par, p.i_bpre, T), T, t, c, w);
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) x[c][q] = add2(x[c][q], w[q]);
                }
                store8<ZT, VEC>(static_cast<ZT*>(p.Y) + row * p.ldy, sp, N, x[c]);
            }
        }
    }
}

// ------------------------------------------------------------------ backward

// One CTA per chunk of rows (or a pair of CTAs, each with half the columns of
// rows wider than one CTA's registers hold), its groups taking the chunk's
// rows in turn.  Per row: the statistics of XO and Z with the sums that the
// pre-norm's Jacobian needs (one exchange; two where a mean comes first), then
// the post-norm's (one more); per column, in registers, the sums over the
// chunk's rows of dY xhat, q zhat, and with BIAS dY and q, where q = dXO' (the
// gate is constant over a chunk and joins in the sum over chunks) or, for
// token gates, q = scale gate dXO'.  The groups' sums meet in shared memory
// (in group order) and go to the chunk's line of partials.
// (The bound of one CTA per SM where registers are not short: N = 5120 bf16,
// RMSNorm on both sides, 96 us without it and 89 with; with the biases' sums
// 2048 columns 90 and 95, rows that are not vectors 29 and 31 at 2000 x 1023.)
template <typename XT, typename ZT, int TT, int C, bool VEC, bool BIAS, int KIND>
__global__ void __launch_bounds__(kBackThreads, VEC && !BIAS ? 1 : 0)
    backward_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(16) uint8_t smem[];
    auto g = make_group<Group<TT, kBackwardSums>>(p, smem);
    const int T = g.T(), t = g.t;
    const int groups = static_cast<int>(blockDim.x) / T;
    uint8_t* par = smem + groups * g.warps() * (8 * kBackwardSums);
    uint8_t* rings = par_at<C>(par, p.n_par, T);
    uint8_t* ring = rings + static_cast<uint32_t>(g.index) * p.stages * p.slot_bytes;
    // a slot: [XO][dXO][Z][dY], the absent ones left out
    const uint32_t xb = static_cast<uint32_t>(C) * 8u * sizeof(XT) * T;
    const uint32_t zb = static_cast<uint32_t>(C) * 8u * sizeof(ZT) * T;
    constexpr bool kAll = KIND != kAnyKind;
    const bool has_z = kAll || p.Z != nullptr, has_dy = kAll || p.dY != nullptr;
    const bool has_dxo = kAll || p.dXO != nullptr, has_dx = kAll || p.dX != nullptr;
    const bool has_dz = kAll || p.dZ != nullptr, token_gate = !kAll && p.token_gate;
    const int pre = kAll ? kind_pre(KIND) : p.pre, post = kAll ? kind_post(KIND) : p.post;
    const uint32_t o_dxo = xb, o_z = o_dxo + (has_dxo ? xb : 0u), o_dy = o_z + (has_z ? zb : 0u);
    const int32_t N = p.N;
    __shared__ float pair[4 * kBackwardSums];
    int32_t col0 = 0;
    int64_t chunk = blockIdx.x;
    if (p.cluster == 2) {
        g.rank = cluster_ctarank();
        g.pair = pair;
        col0 = static_cast<int32_t>(g.rank) * T * C * 8;
        chunk >>= 1;
    }
    int64_t row0, row1, group;
    chunk_span(p, chunk, row0, row1, group);
    zero_ring<VEC>(ring, p.stages * p.slot_bytes, T, t);
    if (p.cluster == 2) cluster_sync_all();     // the other CTA's shared memory is there
    grid_dependency_wait();
    grid_dependents_launch();

    auto fetch = [&](int64_t row, int slot) {
        if (row < row1) {
            uint8_t* s = ring + static_cast<uint32_t>(slot) * p.slot_bytes;
            #pragma unroll
            for (int c = 0; c < C; ++c) {
                const Spot<VEC> sp = spot_of<VEC>(T, t, c, col0);
                fetch8<XT, VEC>(s, T, t, c, static_cast<const XT*>(p.X) + row * p.ldx, sp, N);
                if (has_dxo)
                    fetch8<XT, VEC>(s + o_dxo, T, t, c,
                                    static_cast<const XT*>(p.dXO) + row * p.lddxo, sp, N);
                if (has_z)
                    fetch8<ZT, VEC>(s + o_z, T, t, c,
                                    static_cast<const ZT*>(p.Z) + row * p.ldz, sp, N);
                if (has_dy)
                    fetch8<ZT, VEC>(s + o_dy, T, t, c,
                                    static_cast<const ZT*>(p.dY) + row * p.lddy, sp, N);
            }
        }
        cp_async_commit();
    };
    Held<XT, VEC> hx[C], hd[C];
    Held<ZT, VEC> hz[C], hy[C];
    auto hold = [&](int64_t row) {
        if (row >= row1) return;
        #pragma unroll
        for (int c = 0; c < C; ++c) {
            const Spot<VEC> sp = spot_of<VEC>(T, t, c, col0);
            hold8<XT, VEC>(hx[c], static_cast<const XT*>(p.X) + row * p.ldx, sp, N);
            if (has_dxo) hold8<XT, VEC>(hd[c], static_cast<const XT*>(p.dXO) + row * p.lddxo, sp, N);
            if (has_z) hold8<ZT, VEC>(hz[c], static_cast<const ZT*>(p.Z) + row * p.ldz, sp, N);
            if (has_dy) hold8<ZT, VEC>(hy[c], static_cast<const ZT*>(p.dY) + row * p.lddy, sp, N);
        }
    };

    F8 a_yx[C], a_qz[C], a_y[BIAS ? C : 1], a_q[BIAS ? C : 1];
    #pragma unroll
    for (int c = 0; c < C; ++c) {
        set8(a_yx[c], 0.0f);
        set8(a_qz[c], 0.0f);
        if constexpr (BIAS) {
            set8(a_y[c], 0.0f);
            set8(a_q[c], 0.0f);
        }
    }
    const bool pre_layer = pre == kLayer, post_layer = post == kLayer;

    for (int s = 0; s < p.stages - 1; ++s) fetch(row0 + g.index + static_cast<int64_t>(s) * groups, s);
    if constexpr (!VEC) hold(row0 + g.index);
    fill_vectors<C, VEC>(p, g, par, group, col0);
    int slot = 0;
    for (int64_t row = row0 + g.index; row < row1; row += groups) {
        if constexpr (!VEC) {
            uint8_t* s = ring + static_cast<uint32_t>(slot) * p.slot_bytes;
            #pragma unroll
            for (int c = 0; c < C; ++c) {
                put8<XT, VEC>(s, T, t, c, hx[c]);
                if (has_dxo) put8<XT, VEC>(s + o_dxo, T, t, c, hd[c]);
                if (has_z) put8<ZT, VEC>(s + o_z, T, t, c, hz[c]);
                if (has_dy) put8<ZT, VEC>(s + o_dy, T, t, c, hy[c]);
            }
            hold(row + groups);
        }
        {
            int ahead = slot + p.stages - 1;
            if (ahead >= p.stages) ahead -= p.stages;
            fetch(row + static_cast<int64_t>(p.stages - 1) * groups, ahead);
        }
        cp_async_wait(p.stages - 1);
        uint8_t* s = ring + static_cast<uint32_t>(slot) * p.slot_bytes;
        if (++slot == p.stages) slot = 0;

        // ---- means, where a norm has one: of XO, g = dY wpre, Z
        float mx = 0.0f, mz = 0.0f, gsum = 0.0f;
        if (pre_layer || post_layer) {
            F2 sx = mk2(0.0f), sg = mk2(0.0f), sz = mk2(0.0f);
            #pragma unroll
            for (int c = 0; c < C; ++c) {
                const Spot<VEC> sp = spot_of<VEC>(T, t, c, col0);
                if (!sp.some(N)) continue;
                F8 b;
                if (pre_layer && has_dy) {
                    take8<XT>(s, T, t, c, b);
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) sx = add2(sx, b[q]);
                    take8<ZT>(s + o_dy, T, t, c, b);
                    F8 w;
                    take8<float>(par_at<C>(par, p.i_wpre, T), T, t, c, w);
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) sg = fma2(b[q], w[q], sg);
                }
                if (has_z && post_layer) {
                    take8<ZT>(s + o_z, T, t, c, b);
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) sz = add2(sz, b[q]);
                }
            }
            float v[3] = {sum2(sx), sum2(sg), sum2(sz)};
            group_sum(g, v);
            mx = v[0] * p.inv_n;
            gsum = v[1] * p.inv_n;
            mz = v[2] * p.inv_n;
        }
        // ---- sizes of XO and Z, and the mean of g xhat
        float rx = 1.0f, rz = 1.0f, gx = 0.0f;
        if (pre != kNone || post != kNone) {
            F2 sx = mk2(0.0f), sg = mk2(0.0f), sz = mk2(0.0f);
            #pragma unroll
            for (int c = 0; c < C; ++c) {
                const Spot<VEC> sp = spot_of<VEC>(T, t, c, col0);
                if (!sp.some(N)) continue;
                F8 b, x;
                if (has_dy && pre != kNone) {
                    take8<XT>(s, T, t, c, x);
                    if (pre_layer) center8<VEC>(x, mx, sp, N);
                    take8<ZT>(s + o_dy, T, t, c, b);
                    F8 w;
                    take8<float>(par_at<C>(par, p.i_wpre, T), T, t, c, w);
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        sx = fma2(x[q], x[q], sx);
                        sg = fma2(mul2(b[q], w[q]), x[q], sg);
                    }
                }
                if (has_z && post != kNone) {
                    take8<ZT>(s + o_z, T, t, c, b);
                    if (post_layer) center8<VEC>(b, mz, sp, N);
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) sz = fma2(b[q], b[q], sz);
                }
            }
            float v[3] = {sum2(sx), sum2(sg), sum2(sz)};
            group_sum(g, v);
            if (pre != kNone) {
                rx = inv_size(v[0], p);
                gx = v[1] * rx * p.inv_n;
            }
            if (post != kNone) rz = inv_size(v[2], p);
        }

        // ---- dXO' and the column sums; the post-norm's sums
        F8 d[C];                                     // dXO', then gz = dn wpost
        F2 sgz = mk2(0.0f), sgm = mk2(0.0f);
        #pragma unroll
        for (int c = 0; c < C; ++c) {
            const Spot<VEC> sp = spot_of<VEC>(T, t, c, col0);
            if (!sp.some(N)) continue;
            if (has_dxo) take8<XT>(s + o_dxo, T, t, c, d[c]);
            else set8(d[c], 0.0f);
            if (has_dy) {
                F8 x, b, w;
                take8<XT>(s, T, t, c, x);
                take8<ZT>(s + o_dy, T, t, c, b);
                take8<float>(par_at<C>(par, p.i_wpre, T), T, t, c, w);
                if (pre_layer) center8<VEC>(x, mx, sp, N);
                #pragma unroll
                for (int q = 0; q < 4; ++q) {
                    x[q] = mul2(x[q], mk2(rx));
                    a_yx[c][q] = fma2(b[q], x[q], a_yx[c][q]);
                    if constexpr (BIAS) a_y[c][q] = add2(a_y[c][q], b[q]);
                }
                // rx (g - mean g - xhat mean(g xhat)), g = dY wpre; gx, gsum are 0
                // and rx is 1 where there is no norm
                #pragma unroll
                for (int q = 0; q < 4; ++q) b[q] = fma2(x[q], mk2(-gx), mul2(b[q], w[q]));
                if (pre_layer) center8<VEC>(b, gsum, sp, N);
                #pragma unroll
                for (int q = 0; q < 4; ++q) d[c][q] = fma2(b[q], mk2(rx), d[c][q]);
            }
            if (has_dx)
                store8<XT, VEC>(static_cast<XT*>(p.dX) + row * p.lddx, sp, N, d[c]);
            if (has_z) {
                F8 z, w;
                take8<ZT>(s + o_z, T, t, c, z);
                take8<float>(par_at<C>(par, p.i_ws, T), T, t, c, w);
                if (post_layer) center8<VEC>(z, mz, sp, N);
                #pragma unroll
                for (int q = 0; q < 4; ++q) z[q] = mul2(z[q], mk2(rz));
                if (token_gate) {
                    F8 n, gt;
                    if (p.dgate != nullptr) {
                        // scale * dXO' * n, one row of the gate per row
                        #pragma unroll
                        for (int q = 0; q < 4; ++q) n[q] = mul2(z[q], w[q]);
                        if (p.i_bs >= 0) {
                            F8 b;
                            take8<float>(par_at<C>(par, p.i_bs, T), T, t, c, b);
                            #pragma unroll
                            for (int q = 0; q < 4; ++q) n[q] = add2(n[q], b[q]);
                        }
                        #pragma unroll
                        for (int q = 0; q < 4; ++q) n[q] = mul2(mul2(mk2(p.scale), d[c][q]), n[q]);
                        if (p.grad_dtype == 2)
                            store8<float, VEC>(static_cast<float*>(p.dgate) + row * N, sp, N, n);
                        else if (p.grad_dtype == 1)
                            store8<__nv_bfloat16, VEC>(static_cast<__nv_bfloat16*>(p.dgate) + row * N, sp, N, n);
                        else
                            store8<__half, VEC>(static_cast<__half*>(p.dgate) + row * N, sp, N, n);
                    }
                    load_param8<VEC>(gate_row(p, row), p.vec_dtype, p.vec_aligned != 0, sp, N, gt);
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) d[c][q] = mul2(d[c][q], mul2(gt[q], mk2(p.scale)));
                }
                #pragma unroll
                for (int q = 0; q < 4; ++q) {
                    a_qz[c][q] = fma2(d[c][q], z[q], a_qz[c][q]);
                    if constexpr (BIAS) a_q[c][q] = add2(a_q[c][q], d[c][q]);
                    d[c][q] = mul2(d[c][q], w[q]);
                    sgz = fma2(d[c][q], z[q], sgz);
                    sgm = add2(sgm, d[c][q]);
                }
            }
        }
        if (has_z && has_dz) {
            float gz = 0.0f, gm = 0.0f;
            if (post != kNone) {
                float v[2] = {sum2(sgz), sum2(sgm)};
                group_sum(g, v);
                gz = v[0] * p.inv_n;
                gm = post_layer ? v[1] * p.inv_n : 0.0f;
            }
            #pragma unroll
            for (int c = 0; c < C; ++c) {
                const Spot<VEC> sp = spot_of<VEC>(T, t, c, col0);
                if (!sp.some(N)) continue;
                if (post != kNone) {
                    // rz (gz_j - mean gz - zhat mean(gz zhat)), zhat = (z - mz) rz
                    F8 z;
                    take8<ZT>(s + o_z, T, t, c, z);
                    const F2 k = mk2(-rz * gz), a = mk2(rz * gz * mz - gm);
                    #pragma unroll
                    for (int q = 0; q < 4; ++q)
                        d[c][q] = mul2(add2(fma2(z[q], k, d[c][q]), a), mk2(rz));
                }
                store8<ZT, VEC>(static_cast<ZT*>(p.dZ) + row * p.lddz, sp, N, d[c]);
            }
        }
    }

    // ---- the chunk's column sums: the groups' sums meet in the slots' memory
    if (p.partials == nullptr) return;
    cp_async_wait(0);
    constexpr int kinds = BIAS ? 4 : 2;              // dY xhat, q zhat, dY, q
    F2* line = reinterpret_cast<F2*>(rings);         // one group's sums: T * C * 4 pairs
    auto sums = [&](int k, int c, int q) -> F2& {
        if constexpr (BIAS) {
            if (k == 2) return a_y[c][q];
            if (k == 3) return a_q[c][q];
        }
        return k == 0 ? a_yx[c][q] : a_qz[c][q];
    };
    #pragma unroll
    for (int k = 0; k < kinds; ++k) {
        for (int gi = 1; gi < groups; ++gi) {
            __syncthreads();
            if (g.index == gi) {
                #pragma unroll
                for (int c = 0; c < C; ++c)
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) line[(c * 4 + q) * T + t] = sums(k, c, q);
            }
            __syncthreads();
            if (g.index == 0) {
                #pragma unroll
                for (int c = 0; c < C; ++c)
                    #pragma unroll
                    for (int q = 0; q < 4; ++q)
                        sums(k, c, q) = add2(sums(k, c, q), line[(c * 4 + q) * T + t]);
            }
        }
    }
    if (g.index == 0) {
        float* out = p.partials + chunk * N;
        #pragma unroll
        for (int k = 0; k < kinds; ++k) {
            #pragma unroll
            for (int c = 0; c < C; ++c) {
                const Spot<VEC> sp = spot_of<VEC>(T, t, c, col0);
                #pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float lo, hi;
                    get2(sums(k, c, q), lo, hi);
                    if (sp.in(2 * q, N)) out[k * p.part_stride + sp.at(2 * q)] = lo;
                    if (sp.in(2 * q + 1, N)) out[k * p.part_stride + sp.at(2 * q + 1)] = hi;
                }
            }
        }
    }
}

// ----------------------------------------------------- the sum over the chunks

struct SumParams {
    const float* partials;
    int64_t part_stride;
    int32_t N;
    int32_t chunks;             // lines to add
    int32_t groups, chunks_per_group, token_gate;
    int32_t gated;              // q's sums are weighted by the gate of the chunk's group
    int32_t bias;               // the sums of dY and q were taken
    const void* wpost; const void* bpost; const void* gate;
    int64_t ld_gate;
    int32_t vec_dtype, grad_dtype;
    float scale;
    void* d_pre_weight; void* d_pre_bias; void* d_post_weight; void* d_post_bias; void* d_gate;
    float* lines;               // first of two steps: CTA row y adds its share of the
                                // chunks into line y of [4][kSumSplits][N]
};

__device__ __forceinline__ float param_elem(const void* v, int32_t dtype, int64_t i, float absent) {
    if (v == nullptr) return absent;
    if (dtype == 2) return static_cast<const float*>(v)[i];
    if (dtype == 1) return __bfloat162float(static_cast<const __nv_bfloat16*>(v)[i]);
    return __half2float(static_cast<const __half*>(v)[i]);
}

constexpr int kSumY = 32;
constexpr int kSumSplits = 16;      // lines that many chunks are added to first
// Chunks that one step adds.  (Backward, 8192 x 4096 / 65536 x 512: 4096 chunks
// 497 / 344 us in one step, 462 / 279 in two; 1024 chunks 189 / 138 and 187 / 123.)
constexpr int kSumOneStep = 1024;
// Gate groups that get CTAs of their own; of more, dgate_kernel makes the
// gate's gradient.  (The same: 2 groups 88 / 68 us beside, 93 / 72 by the
// kernel; 32 groups 172 / 121 and 157 / 124; 1024 groups 714 / 186 and 189 / 138.)
constexpr int kSumGroups = 16;

// Sums over the chunks, 32 columns per CTA, kSumY lines of threads that take
// the chunks in turn and are added in line order.  CTAs with blockIdx.y == 0
// make the totals, the gate's row joining chunk by chunk; the others (where
// the gate's gradient is wanted) one group's sums each.  With p.lines, CTA row
// y adds its part of the chunks into line y instead.
static __global__ void __launch_bounds__(32 * kSumY)
    sum_kernel(const __grid_constant__ SumParams p) {
    __shared__ float red[4][kSumY][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int32_t col = static_cast<int32_t>(blockIdx.x) * 32 + tx;
    const bool in = col < p.N;
    grid_dependency_wait();
    grid_dependents_launch();
    int32_t first = 0, last = p.chunks;
    bool gated = p.gated != 0;
    const int32_t y = static_cast<int32_t>(blockIdx.y);
    if (p.lines != nullptr) {
        first = static_cast<int32_t>(static_cast<int64_t>(p.chunks) * y / kSumSplits);
        last = static_cast<int32_t>(static_cast<int64_t>(p.chunks) * (y + 1) / kSumSplits);
    } else if (y > 0) {
        first = (y - 1) * p.chunks_per_group;
        last = y * p.chunks_per_group;
        gated = false;
    }
    float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (in) {
        const float* base = p.partials + col;
        const float one = gated && p.groups == 1 ? param_elem(p.gate, p.vec_dtype, col, 1.0f) : 1.0f;
        #pragma unroll 4
        for (int32_t c = first + ty; c < last; c += kSumY) {
            const float* q = base + static_cast<int64_t>(c) * p.N;
            float gt = one;
            if (gated && p.gate != nullptr && p.groups > 1)
                gt = param_elem(p.gate, p.vec_dtype, (c / p.chunks_per_group) * p.ld_gate + col, 1.0f);
            a[0] += q[0];
            a[1] = fmaf(gt, q[p.part_stride], a[1]);
            if (p.bias) {
                a[2] += q[2 * p.part_stride];
                a[3] = fmaf(gt, q[3 * p.part_stride], a[3]);
            }
        }
    }
    #pragma unroll
    for (int k = 0; k < 4; ++k) red[k][ty][tx] = a[k];
    __syncthreads();
    // line k < 4 adds the k-th sum over the lines
    if (ty < 4) {
        float s = 0.0f;
        #pragma unroll
        for (int i = 0; i < kSumY; ++i) s += red[ty][i][tx];
        red[ty][0][tx] = s;
    }
    __syncthreads();
    if (ty != 0 || !in) return;
    #pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = red[k][0][tx];
    if (p.lines != nullptr) {
        #pragma unroll
        for (int k = 0; k < 4; ++k)
            p.lines[(static_cast<int64_t>(k) * kSumSplits + y) * p.N + col] = a[k];
    } else if (y == 0) {
        const float f = p.token_gate ? 1.0f : p.scale;
        if (p.d_pre_weight) store_elem(p.d_pre_weight, p.grad_dtype, col, a[0]);
        if (p.d_post_weight) store_elem(p.d_post_weight, p.grad_dtype, col, f * a[1]);
        if (p.d_pre_bias) store_elem(p.d_pre_bias, p.grad_dtype, col, a[2]);
        if (p.d_post_bias) store_elem(p.d_post_bias, p.grad_dtype, col, f * a[3]);
    } else {
        float v = a[1] * param_elem(p.wpost, p.vec_dtype, col, 1.0f);
        if (p.bpost != nullptr) v = fmaf(a[3], param_elem(p.bpost, p.vec_dtype, col, 0.0f), v);
        store_elem(p.d_gate, p.grad_dtype, static_cast<int64_t>(y - 1) * p.N + col, p.scale * v);
    }
}

// The gate's gradient where its groups are many (and so of few chunks each):
// a thread per group and column adds the group's chunks.
static __global__ void __launch_bounds__(256)
    dgate_kernel(const __grid_constant__ SumParams p) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int64_t total = static_cast<int64_t>(p.groups) * p.N;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const int32_t gr = static_cast<int32_t>(i / p.N);
        const int32_t col = static_cast<int32_t>(i - static_cast<int64_t>(gr) * p.N);
        const float* q = p.partials + p.part_stride +
                         static_cast<int64_t>(gr) * p.chunks_per_group * p.N + col;
        float s = 0.0f, t = 0.0f;
        for (int32_t c = 0; c < p.chunks_per_group; ++c) {
            s += q[static_cast<int64_t>(c) * p.N];
            if (p.bpost != nullptr) t += q[2 * p.part_stride + static_cast<int64_t>(c) * p.N];
        }
        float v = s * param_elem(p.wpost, p.vec_dtype, col, 1.0f);
        if (p.bpost != nullptr) v = fmaf(t, param_elem(p.bpost, p.vec_dtype, col, 0.0f), v);
        store_elem(p.d_gate, p.grad_dtype, i, p.scale * v);
    }
}

}  // namespace nrm
}  // namespace gemm103
