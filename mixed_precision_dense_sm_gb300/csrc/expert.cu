// expert.cu -- tokens sorted by expert, and the moves of their rows
// (include/expert_sm103.h).
//
// expert_sort_kernel: a stable counting sort in one launch.  The slots are cut
// into contiguous pieces, one per warp; a warp counts its piece in its own line
// of shared memory, 32 slots at a time (the lanes that chose the same expert find
// each other by match), which also gives every slot its rank within the piece.
// Lines become prefixes over the warps of a CTA, CTA totals meet over the cluster
// through distributed shared memory, and a scan over the experts makes the
// offsets; position = expert's offset + lower CTAs + lower warps + rank.  No
// atomics, so the order is that of the slots.  A cluster and not the whole GPU:
// one launch whose phases are joined by hardware barriers beats two launches.
//
// rows_out_kernel (gather, combine_backward) and rows_in_kernel (combine,
// gather_backward): one group of threads per token.  Token-major, because a
// token's row then is read (or written) once for all its k moves and the sums and
// dot products stay in registers; the k rows are at least one 16-byte vector per
// thread each, contiguous over a group.  Bound by HBM.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "device.h"
#include "device_limits.h"
#include "epilogue_ops.cuh"
#include "expert_sm103.h"
#include "f32x2.cuh"
#include "ptx.cuh"

namespace {

using namespace gemm103;

// ------------------------------------------------------------------------ sort

constexpr int kSortThreads = 1024;
constexpr int kSortCluster = 8;              // CTAs at most (the portable cluster size)
constexpr int kHeld = 4;                     // batches of 32 slots a warp holds in registers

struct SortParams {
    const void* ids;
    int64_t ldids;
    int32_t n, k, E;
    int32_t warps;                           // that count: those with slots
    int32_t piece;                           // slots per warp, a multiple of 32
    int32_t ctas;
    int32_t *pos, *offsets, *order;
};

// The expert of a slot; E where it has none.
template <typename ID>
__device__ __forceinline__ int32_t sort_key(const SortParams& p, int32_t slot) {
    if (slot >= p.n) return p.E;
    int64_t at = slot;
    if (p.ldids != p.k) {
        const int32_t t = slot / p.k;
        at = t * p.ldids + (slot - t * p.k);
    }
    const ID e = static_cast<const ID*>(p.ids)[at];
    return e >= 0 && e < p.E ? static_cast<int32_t>(e) : p.E;
}

// Rank of this lane's slot among the warp's slots of its expert so far, which are
// counted in `line`.
__device__ __forceinline__ int32_t sort_rank(int32_t* line, int32_t key, int32_t E, int lane) {
    const uint32_t peers = __match_any_sync(0xffffffffu, key);
    const int32_t before = __popc(peers & ((1u << lane) - 1u));
    const int32_t seen = key < E ? line[key] : 0;
    __syncwarp();
    if (before == 0 && key < E) line[key] = seen + __popc(peers);
    __syncwarp();
    return seen + before;
}

template <typename ID, bool HELD>
__global__ void __launch_bounds__(kSortThreads) expert_sort_kernel(const SortParams p) {
    extern __shared__ int32_t sort_smem[];
    int32_t* hist = sort_smem;                               // [warps][E]
    int32_t* total = hist + p.warps * p.E;                   // [E] this CTA's
    int32_t* base = total + p.E;                             // [E]
    __shared__ int32_t warp_sum[32];
    __shared__ int32_t kept;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t rank = p.ctas > 1 ? static_cast<int32_t>(cluster_ctarank()) : 0;

    for (int32_t i = threadIdx.x; i < p.warps * p.E; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    grid_dependency_wait();
    grid_dependents_launch();

    // count
    const int32_t first = (rank * p.warps + warp) * p.piece;
    int32_t* line = hist + warp * p.E;
    int32_t key[kHeld], at[kHeld];
    if (warp < p.warps) {
        if constexpr (HELD) {
            #pragma unroll
            for (int b = 0; b < kHeld; ++b)
                key[b] = b * 32 < p.piece ? sort_key<ID>(p, first + b * 32 + lane) : p.E;
            #pragma unroll
            for (int b = 0; b < kHeld; ++b)
                if (b * 32 < p.piece) at[b] = sort_rank(line, key[b], p.E, lane);
        } else {
            // ranks wait in pos, each for the thread that wrote it
            int32_t next = sort_key<ID>(p, first + lane);
            for (int32_t b = 0; b < p.piece && first + b < p.n; b += 32) {
                const int32_t cur = next, slot = first + b + lane;
                if (b + 32 < p.piece) next = sort_key<ID>(p, slot + 32);
                const int32_t r = sort_rank(line, cur, p.E, lane);
                if (slot < p.n) p.pos[slot] = r;
            }
        }
    }
    __syncthreads();

    // lines -> prefixes over the warps; the CTA's totals
    const int32_t e = threadIdx.x;                           // blockDim.x >= E
    int32_t mine = 0;
    if (e < p.E) {
        #pragma unroll 8
        for (int32_t w = 0; w < p.warps; ++w) {
            const int32_t c = hist[w * p.E + e];
            hist[w * p.E + e] = mine;
            mine += c;
        }
        total[e] = mine;
    }
    int32_t lower = 0, all = mine;
    if (p.ctas > 1) {
        cluster_sync_all();
        if (e < p.E) {
            all = 0;
            for (int32_t r = 0; r < p.ctas; ++r) {
                int32_t c;
                asm volatile("ld.shared::cluster.s32 %0, [%1];"
                             : "=r"(c)
                             : "r"(map_to_rank(smem_addr(total + e), static_cast<uint32_t>(r)))
                             : "memory");
                if (r < rank) lower += c;
                all += c;
            }
        }
        __syncwarp();
        // (the wait, before the end, keeps every CTA's memory until all have read it)
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    // the experts before e
    int32_t incl = all;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    const int32_t warps = blockDim.x >> 5;
    int32_t below = 0;
    for (int32_t w = 0; w < warps; ++w) below += w < warp ? warp_sum[w] : 0;
    const int32_t offset = below + incl - all;
    if (e < p.E) {
        base[e] = offset + lower;
        if (rank == 0) p.offsets[e] = offset;
        if (e == p.E - 1) {
            kept = offset + all;
            if (rank == 0) p.offsets[p.E] = offset + all;
        }
    }
    __syncthreads();

    // place
    if (warp < p.warps) {
        if constexpr (HELD) {
            #pragma unroll
            for (int b = 0; b < kHeld; ++b) {
                const int32_t slot = first + b * 32 + lane;
                if (b * 32 >= p.piece || slot >= p.n) continue;
                const int32_t i = key[b] < p.E ? base[key[b]] + line[key[b]] + at[b] : -1;
                p.pos[slot] = i;
                if (i >= 0 && p.order != nullptr) p.order[i] = slot;
            }
        } else {
            #pragma unroll 4
            for (int32_t b = 0; b < p.piece; b += 32) {
                const int32_t slot = first + b + lane;
                if (slot >= p.n) break;
                const int32_t c = sort_key<ID>(p, slot);
                const int32_t i = c < p.E ? base[c] + line[c] + p.pos[slot] : -1;
                p.pos[slot] = i;
                if (i >= 0 && p.order != nullptr) p.order[i] = slot;
            }
        }
    }
    if (p.order != nullptr)
        for (int64_t i = static_cast<int64_t>(kept) + rank * blockDim.x + threadIdx.x; i < p.n;
             i += p.ctas * blockDim.x)
            p.order[i] = -1;
    if (p.ctas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename ID, bool HELD>
cudaError_t launch_sort(const SortParams& p, int threads, cudaStream_t stream) {
    auto kern = expert_sort_kernel<ID, HELD>;
    const size_t smem = static_cast<size_t>(p.warps + 2) * p.E * 4;
    static DeviceLimits limit;
    const cudaError_t set = limit.raise(smem, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(smem));
    });
    if (set != cudaSuccess) return set;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.ctas);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.ctas), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = p.ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// ------------------------------------------------------------------------ rows

constexpr int kRowThreads = 256;
constexpr int kTurn = 8;                     // choices handled at a time

struct RowsParams {
    const void* tok_in;                      // X or dY
    int64_t ld_tok_in;
    void* tok_out;                           // Y or dX
    int64_t ld_tok_out;
    const void* rows_in;                     // Ys or dXs
    int64_t ld_rows_in;
    void* rows_out;                          // Xs or dYs
    int64_t ld_rows_out;
    const int32_t* pos;
    const void* weight;
    int64_t ldw;
    void* dweight;
    int64_t lddw;
    int32_t wtype, dwtype;
    int64_t T, k, D, rows;
    int32_t log_group;                       // log2(threads per token)
    int32_t chunks;                          // groups that share a token's columns
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T e[V];
};
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p) {
    return *reinterpret_cast<const Pack<T, V>*>(p);
}

// Positions and weights of choices j0 .. j0 + 7 of a token; -1 where there is none.
__device__ __forceinline__ void load_choices(const RowsParams& p, int64_t t, int64_t j0, int32_t (&at)[kTurn],
                                             float (&w)[kTurn]) {
    #pragma unroll
    for (int j = 0; j < kTurn; ++j) {
        const bool is = j0 + j < p.k;
        const int32_t i = is ? p.pos[t * p.k + j0 + j] : -1;
        at[j] = i >= 0 && i < p.rows ? i : -1;
        w[j] = is && p.weight != nullptr ? load_bias_elem(p.weight, p.wtype, t * p.ldw + j0 + j) : 1.0f;
    }
}

// Sums of v[0..7] over a group of threads (whole warps); the group's thread j has
// the sum of v[j] for j < 8.  By halving: a lane keeps half its values and gives
// the other half away, so 9 shuffles do for 8 sums.
__device__ __forceinline__ float group_sums(float (&v)[kTurn], int log_group, float (*red)[kTurn]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int at = 0;
    #pragma unroll
    for (int n = kTurn / 2, o = 16; n >= 1; n >>= 1, o >>= 1) {
        const bool up = (lane & o) != 0;
        at |= up ? n : 0;
        #pragma unroll
        for (int i = 0; i < n; ++i) {
            const float keep = up ? v[n + i] : v[i], give = up ? v[i] : v[n + i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    float s = v[0];
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    __syncthreads();                         // what was in red has been read
    if ((lane & 3) == 0) red[warp][at] = s;
    __syncthreads();
    const int g = threadIdx.x & ((1 << log_group) - 1), warps = 1 << (log_group - 5);
    float t = 0.0f;
    if (g < kTurn) {
        const int w0 = (threadIdx.x >> log_group) << (log_group - 5);
        for (int w = 0; w < warps; ++w) t += red[w0 + w][g];
    }
    return t;
}

struct Place {
    int64_t t;                               // token
    int32_t g, group;                        // thread of its group, threads of the group
    int32_t v0, v1;                          // vectors of this group
    bool live;
};
__device__ __forceinline__ Place place_of(const RowsParams& p, int32_t nvec) {
    Place a;
    a.group = 1 << p.log_group;
    a.g = static_cast<int32_t>(threadIdx.x) & (a.group - 1);
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kRowThreads >> p.log_group) +
                         (threadIdx.x >> p.log_group);
    int32_t chunk = 0;
    a.t = unit;
    if (p.chunks > 1) {
        a.t = unit / p.chunks;
        chunk = static_cast<int32_t>(unit - a.t * p.chunks);
    }
    const int32_t per = (nvec + p.chunks - 1) / p.chunks;
    a.v0 = chunk * per;
    a.v1 = a.v0 + per < nvec ? a.v0 + per : nvec;
    a.live = a.t < p.T;
    return a;
}

// A token's row, weighted, to its k places; DOT: and the dot products of the row
// with what is at these places in rows_in.
template <typename T, int V, bool DOT>
__global__ void __launch_bounds__(kRowThreads) rows_out_kernel(const RowsParams p) {
    __shared__ float red[DOT ? kRowThreads / 32 : 1][kTurn];
    grid_dependency_wait();
    grid_dependents_launch();
    const int32_t nvec = static_cast<int32_t>(p.D / V), tail = static_cast<int32_t>(p.D - static_cast<int64_t>(nvec) * V);
    const Place a = place_of(p, nvec);
    if (!DOT && !a.live) return;
    const T* x = static_cast<const T*>(p.tok_in) + (a.live ? a.t : 0) * p.ld_tok_in;
    const T* in = static_cast<const T*>(p.rows_in);
    T* out = static_cast<T*>(p.rows_out);
    for (int64_t j0 = 0; j0 < p.k; j0 += kTurn) {
        int32_t at[kTurn];
        float w[kTurn], dot[kTurn];
        #pragma unroll
        for (int j = 0; j < kTurn; ++j) dot[j] = 0.0f, at[j] = -1;
        if (a.live) {
            load_choices(p, a.t, j0, at, w);
            for (int32_t c = a.v0 + a.g; c < a.v1; c += a.group) {
                const int64_t col = static_cast<int64_t>(c) * V;
                const Pack<T, V> xv = load_pack<T, V>(x + col);
                Pack<T, V> o[DOT ? kTurn : 1];
                if constexpr (DOT) {
                    #pragma unroll
                    for (int j = 0; j < kTurn; ++j)
                        if (at[j] >= 0) o[j] = load_pack<T, V>(in + at[j] * p.ld_rows_in + col);
                }
                #pragma unroll
                for (int j = 0; j < kTurn; ++j) {
                    if (at[j] < 0) continue;
                    Pack<T, V> r;
                    #pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float f = to_f<T>(xv.e[i]);
                        if constexpr (DOT) dot[j] = fmaf(f, to_f<T>(o[j].e[i]), dot[j]);
                        r.e[i] = from_f<T>(f * w[j]);
                    }
                    if (!DOT || out != nullptr)
                        *reinterpret_cast<Pack<T, V>*>(out + at[j] * p.ld_rows_out + col) = r;
                }
            }
            // the elements behind the last vector
            if (a.v1 == nvec && a.g < tail) {
                const int64_t col = static_cast<int64_t>(nvec) * V + a.g;
                const float f = to_f<T>(x[col]);
                #pragma unroll
                for (int j = 0; j < kTurn; ++j) {
                    if (at[j] < 0) continue;
                    if constexpr (DOT) dot[j] = fmaf(f, to_f<T>(in[at[j] * p.ld_rows_in + col]), dot[j]);
                    if (!DOT || out != nullptr) out[at[j] * p.ld_rows_out + col] = from_f<T>(f * w[j]);
                }
            }
        }
        if constexpr (DOT) {
            const float s = group_sums(dot, p.log_group, red);
            if (a.live && a.g < kTurn && j0 + a.g < p.k)
                store_elem(p.dweight, p.dwtype, a.t * p.lddw + j0 + a.g, s);
        }
    }
}

// The weighted sum of a token's k rows; DOT: and the rows' dot products with the
// token's row in tok_in.
template <typename T, int V, bool DOT>
__global__ void __launch_bounds__(kRowThreads) rows_in_kernel(const RowsParams p) {
    __shared__ float red[DOT ? kRowThreads / 32 : 1][kTurn];
    grid_dependency_wait();
    grid_dependents_launch();
    const int32_t nvec = static_cast<int32_t>(p.D / V), tail = static_cast<int32_t>(p.D - static_cast<int64_t>(nvec) * V);
    const Place a = place_of(p, nvec);
    if (!DOT && !a.live) return;
    const T* in = static_cast<const T*>(p.rows_in);
    const int64_t tt = a.live ? a.t : 0;
    const T* x = DOT ? static_cast<const T*>(p.tok_in) + tt * p.ld_tok_in : nullptr;
    T* y = p.tok_out != nullptr ? static_cast<T*>(p.tok_out) + tt * p.ld_tok_out : nullptr;
    int32_t at[kTurn];
    float w[kTurn], dot[kTurn];
    #pragma unroll
    for (int j = 0; j < kTurn; ++j) dot[j] = 0.0f, at[j] = -1, w[j] = 0.0f;
    if (a.live) {
        load_choices(p, a.t, 0, at, w);
        for (int32_t c = a.v0 + a.g; c < a.v1; c += a.group) {
            const int64_t col = static_cast<int64_t>(c) * V;
            Pack<T, V> xv;
            if constexpr (DOT) xv = load_pack<T, V>(x + col);
            float acc[V];
            #pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = 0.0f;
            for (int64_t j0 = 0;;) {
                Pack<T, V> r[kTurn];
                #pragma unroll
                for (int j = 0; j < kTurn; ++j)
                    if (at[j] >= 0) r[j] = load_pack<T, V>(in + at[j] * p.ld_rows_in + col);
                #pragma unroll
                for (int j = 0; j < kTurn; ++j) {
                    if (at[j] < 0) continue;
                    #pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float f = to_f<T>(r[j].e[i]);
                        if constexpr (DOT)
                            if (j0 == 0) dot[j] = fmaf(to_f<T>(xv.e[i]), f, dot[j]);
                        acc[i] = fmaf(w[j], f, acc[i]);
                    }
                }
                if (p.k <= kTurn) break;
                j0 = j0 + kTurn < p.k ? j0 + kTurn : 0;
                load_choices(p, a.t, j0, at, w);
                if (j0 == 0) break;
            }
            Pack<T, V> o;
            #pragma unroll
            for (int i = 0; i < V; ++i) o.e[i] = from_f<T>(acc[i]);
            if (!DOT || y != nullptr) *reinterpret_cast<Pack<T, V>*>(y + col) = o;
        }
        // the elements behind the last vector
        if (a.v1 == nvec && a.g < tail) {
            const int64_t col = static_cast<int64_t>(nvec) * V + a.g;
            const float xf = DOT ? to_f<T>(x[col]) : 0.0f;
            float acc = 0.0f;
            for (int64_t j0 = 0;;) {
                #pragma unroll
                for (int j = 0; j < kTurn; ++j) {
                    if (at[j] < 0) continue;
                    const float f = to_f<T>(in[at[j] * p.ld_rows_in + col]);
                    if constexpr (DOT)
                        if (j0 == 0) dot[j] = fmaf(xf, f, dot[j]);
                    acc = fmaf(w[j], f, acc);
                }
                if (p.k <= kTurn) break;
                j0 = j0 + kTurn < p.k ? j0 + kTurn : 0;
                load_choices(p, a.t, j0, at, w);
                if (j0 == 0) break;
            }
            if (!DOT || y != nullptr) y[col] = from_f<T>(acc);
        }
    }
    if constexpr (DOT) {
        // the first eight choices have theirs; further ones read their rows again
        for (int64_t j0 = 0; j0 < p.k; j0 += kTurn) {
            if (j0 > 0) {
                #pragma unroll
                for (int j = 0; j < kTurn; ++j) dot[j] = 0.0f;
                if (a.live) {
                    load_choices(p, a.t, j0, at, w);
                    for (int64_t col = a.g; col < p.D; col += a.group) {
                        const float xf = to_f<T>(x[col]);
                        #pragma unroll
                        for (int j = 0; j < kTurn; ++j)
                            if (at[j] >= 0) dot[j] = fmaf(xf, to_f<T>(in[at[j] * p.ld_rows_in + col]), dot[j]);
                    }
                }
            }
            const float s = group_sums(dot, p.log_group, red);
            if (a.live && a.g < kTurn && j0 + a.g < p.k)
                store_elem(p.dweight, p.dwtype, a.t * p.lddw + j0 + a.g, s);
        }
    }
}

enum RowsKind { kOut, kOutDot, kIn, kInDot };

template <typename T, int V>
cudaError_t launch_rows(RowsKind kind, const RowsParams& p, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    const int64_t per = kRowThreads >> p.log_group;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.T * p.chunks + per - 1) / per), 1, 1);
    cfg.blockDim = dim3(kRowThreads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    switch (kind) {
        case kOut: return cudaLaunchKernelEx(&cfg, rows_out_kernel<T, V, false>, p);
        case kOutDot: return cudaLaunchKernelEx(&cfg, rows_out_kernel<T, V, true>, p);
        case kIn: return cudaLaunchKernelEx(&cfg, rows_in_kernel<T, V, false>, p);
        default: return cudaLaunchKernelEx(&cfg, rows_in_kernel<T, V, true>, p);
    }
}

bool dtype_ok(int32_t t) { return t == GEMM_F16 || t == GEMM_BF16 || t == GEMM_F32; }
int32_t esize(int32_t t) { return t == GEMM_F32 ? 4 : 2; }
bool aligned(const void* p, int32_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

constexpr int64_t kMost = 1ll << 30;         // slots, rows and columns: 32-bit numbers, with room behind

bool sizes_ok(int64_t T, int64_t k) {
    return T >= 0 && k >= 0 && T <= kMost && k <= kMost && (k == 0 || T <= kMost / k);
}

// A matrix argument: `needed` unless it has no elements.
bool matrix_ok(const void* p, int64_t ld, int64_t rows, int64_t cols, int32_t es, bool needed) {
    if (p == nullptr) return !needed || rows == 0 || cols == 0;
    return ld >= (cols > 0 ? cols : 1) && ld <= (1ll << 40) && aligned(p, es);
}


gemm_status_t rows_call(RowsKind kind, RowsParams& p, int32_t dtype, const expert_weights_t* w,
                        cudaStream_t stream) {
    const bool out = kind == kOut || kind == kOutDot;
    if (w != nullptr) {
        if (!matrix_ok(w->weight, w->ldw, p.T, p.k, w->weight ? esize(w->weight_dtype) : 1, false) ||
            (w->weight != nullptr && !dtype_ok(w->weight_dtype)))
            return GEMM_ERR_INVALID_VALUE;
        p.weight = w->weight, p.ldw = w->ldw, p.wtype = w->weight_dtype;
        if (kind == kOutDot || kind == kInDot) {
            if (!matrix_ok(w->dweight, w->lddw, p.T, p.k, w->dweight ? esize(w->dweight_dtype) : 1, false) ||
                (w->dweight != nullptr && !dtype_ok(w->dweight_dtype)))
                return GEMM_ERR_INVALID_VALUE;
            p.dweight = w->dweight, p.lddw = w->lddw, p.dwtype = w->dweight_dtype;
        }
    }
    // without the weights' gradient a backward pass is the other move
    if (p.dweight == nullptr) kind = out ? kOut : kIn;
    const bool dot = kind == kOutDot || kind == kInDot;
    const int32_t es = esize(dtype);
    if (!sizes_ok(p.T, p.k) || p.D < 0 || p.D > kMost || p.rows < 0 || p.rows > kMost || !dtype_ok(dtype))
        return GEMM_ERR_INVALID_VALUE;
    if (p.T > 0 && p.k > 0 && (p.pos == nullptr || !aligned(p.pos, 4))) return GEMM_ERR_INVALID_VALUE;
    if (!matrix_ok(p.tok_in, p.ld_tok_in, p.T, p.D, es, out || dot) ||
        !matrix_ok(p.rows_in, p.ld_rows_in, p.rows, p.D, es, !out || dot) ||
        !matrix_ok(p.tok_out, p.ld_tok_out, p.T, p.D, es, !out && !dot) ||
        !matrix_ok(p.rows_out, p.ld_rows_out, p.rows, p.D, es, out && !dot))
        return GEMM_ERR_INVALID_VALUE;
    const int sms = device_sms();
    if (sms < 0) return GEMM_ERR_LAUNCH;
    if (sms == 0) return GEMM_ERR_NOT_SUPPORTED;
    if (p.T == 0 || (p.D == 0 && !dot)) return GEMM_OK;

    // 16-byte vectors where every row of every matrix starts on one
    const int32_t per = 16 / es;
    auto vector = [&](const void* q, int64_t ld) { return q == nullptr || (aligned(q, 16) && ld % per == 0); };
    const bool vec = vector(p.tok_in, p.ld_tok_in) && vector(p.rows_in, p.ld_rows_in) &&
                     vector(p.tok_out, p.ld_tok_out) && vector(p.rows_out, p.ld_rows_out);
    const int64_t nvec = vec ? p.D / per : p.D;
    // Threads per token: as many as it has vectors, up to a CTA's; whole warps
    // where they add up dot products.
    p.log_group = dot ? 5 : 2;
    while (p.log_group < 8 && (1 << p.log_group) < nvec) ++p.log_group;
    p.chunks = 1;
    if (!dot && p.T < 2 * sms && nvec > 64) {
        // few tokens: their columns over more SMs
        p.log_group = 6;
        p.chunks = static_cast<int32_t>((nvec + 63) / 64);
    }
    cudaError_t e;
    if (dtype == GEMM_F32)
        e = vec ? launch_rows<float, 4>(kind, p, stream) : launch_rows<float, 1>(kind, p, stream);
    else if (dtype == GEMM_BF16)
        e = vec ? launch_rows<__nv_bfloat16, 8>(kind, p, stream) : launch_rows<__nv_bfloat16, 1>(kind, p, stream);
    else
        e = vec ? launch_rows<__half, 8>(kind, p, stream) : launch_rows<__half, 1>(kind, p, stream);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

// A backward pass without outputs: right where they are empty.
gemm_status_t nothing_wanted(int64_t T, int64_t k, int64_t D, int64_t rows) {
    const bool empty = T == 0 || k == 0 || D == 0 || rows == 0;
    return sizes_ok(T, k) && D >= 0 && rows >= 0 && empty ? GEMM_OK : GEMM_ERR_INVALID_VALUE;
}

RowsParams rows_params(int64_t T, int64_t k, int64_t D, int64_t rows, const int32_t* pos) {
    RowsParams p = {};
    p.T = T, p.k = k, p.D = D, p.rows = rows, p.pos = pos;
    return p;
}

}  // namespace

extern "C" {

gemm_status_t expert_sort(int64_t T, int64_t k, int64_t E, const void* ids, int64_t ldids,
                          int32_t id_bytes, int32_t* pos, int32_t* offsets, int32_t* order,
                          gemm_stream_t stream) {
    if (!sizes_ok(T, k) || E < 1 || E > EXPERT_MAX || (id_bytes != 4 && id_bytes != 8))
        return GEMM_ERR_INVALID_VALUE;
    if (!matrix_ok(ids, ldids, T, k, id_bytes, true) || offsets == nullptr || !aligned(offsets, 4) ||
        !aligned(pos, 4) || !aligned(order, 4) || (T > 0 && k > 0 && pos == nullptr))
        return GEMM_ERR_INVALID_VALUE;
    const int sms = device_sms();
    if (sms < 0) return GEMM_ERR_LAUNCH;
    if (sms == 0) return GEMM_ERR_NOT_SUPPORTED;
    SortParams p = {};
    p.ids = ids, p.ldids = T == 1 ? k : ldids;
    p.n = static_cast<int32_t>(T * k), p.k = static_cast<int32_t>(k), p.E = static_cast<int32_t>(E);
    p.pos = pos, p.offsets = offsets, p.order = order;
    // CTAs: one while a warp's piece stays within what it holds
    const int64_t batches = (T * k + 31) / 32;
    p.ctas = 1;
    while (p.ctas < kSortCluster && batches > 32ll * kHeld * p.ctas) p.ctas *= 2;
    int64_t warps = (batches + p.ctas - 1) / p.ctas;
    p.warps = static_cast<int32_t>(warps < 1 ? 1 : warps > 32 ? 32 : warps);
    const int64_t cells = static_cast<int64_t>(p.ctas) * p.warps;
    p.piece = static_cast<int32_t>((batches + cells - 1) / cells * 32);
    int threads = static_cast<int>((E + 31) / 32 * 32);
    if (threads < p.warps * 32) threads = p.warps * 32;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool held = p.piece <= 32 * kHeld;
    const cudaError_t e = id_bytes == 4 ? (held ? launch_sort<int32_t, true>(p, threads, s)
                                                : launch_sort<int32_t, false>(p, threads, s))
                                        : (held ? launch_sort<int64_t, true>(p, threads, s)
                                                : launch_sort<int64_t, false>(p, threads, s));
    if (e != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

gemm_status_t expert_gather(int64_t T, int64_t k, int64_t D, int64_t rows, const void* X,
                            int64_t ldx, const int32_t* pos, void* Xs, int64_t ldxs,
                            int32_t dtype, const expert_weights_t* w, gemm_stream_t stream) {
    RowsParams p = rows_params(T, k, D, rows, pos);
    p.tok_in = X, p.ld_tok_in = ldx, p.rows_out = Xs, p.ld_rows_out = ldxs;
    return rows_call(kOut, p, dtype, w, reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t expert_combine(int64_t T, int64_t k, int64_t D, int64_t rows, const void* Ys,
                             int64_t ldys, const int32_t* pos, void* Y, int64_t ldy,
                             int32_t dtype, const expert_weights_t* w, gemm_stream_t stream) {
    RowsParams p = rows_params(T, k, D, rows, pos);
    p.rows_in = Ys, p.ld_rows_in = ldys, p.tok_out = Y, p.ld_tok_out = ldy;
    return rows_call(kIn, p, dtype, w, reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t expert_gather_backward(int64_t T, int64_t k, int64_t D, int64_t rows,
                                     const void* dXs, int64_t lddxs, const void* X, int64_t ldx,
                                     const int32_t* pos, void* dX, int64_t lddx, int32_t dtype,
                                     const expert_weights_t* w, gemm_stream_t stream) {
    const bool dots = w != nullptr && w->dweight != nullptr;
    if (dX == nullptr && !dots) return nothing_wanted(T, k, D, rows);
    RowsParams p = rows_params(T, k, D, rows, pos);
    p.rows_in = dXs, p.ld_rows_in = lddxs, p.tok_out = dX, p.ld_tok_out = lddx;
    if (dots) p.tok_in = X, p.ld_tok_in = ldx;
    return rows_call(kInDot, p, dtype, w, reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t expert_combine_backward(int64_t T, int64_t k, int64_t D, int64_t rows,
                                      const void* dY, int64_t lddy, const void* Ys, int64_t ldys,
                                      const int32_t* pos, void* dYs, int64_t lddys, int32_t dtype,
                                      const expert_weights_t* w, gemm_stream_t stream) {
    const bool dots = w != nullptr && w->dweight != nullptr;
    if (dYs == nullptr && !dots) return nothing_wanted(T, k, D, rows);
    RowsParams p = rows_params(T, k, D, rows, pos);
    p.tok_in = dY, p.ld_tok_in = lddy, p.rows_out = dYs, p.ld_rows_out = lddys;
    if (dots) p.rows_in = Ys, p.ld_rows_in = ldys;
    return rows_call(kOutDot, p, dtype, w, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
