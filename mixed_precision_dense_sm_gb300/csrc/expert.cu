// expert.cu -- tokens sorted by expert, and the moves of their rows
// (include/expert_sm103.h).
//
// expert_sort_kernel: a stable counting sort in one launch.  The slots are cut
// into contiguous pieces, one per warp; a warp counts its piece in its own line
// of shared memory, 32 slots at a time (the lanes that chose the same expert find
// each other by votes), which also gives every slot its rank within the piece.
// Lines become prefixes over the warps of a CTA, CTA totals meet over the cluster
// through distributed shared memory, and a scan over the experts makes the
// offsets; position = expert's offset + lower CTAs + lower warps + rank.  The order
// is that of the slots.  Up to kOneLaunch slots that is one cluster, whose phases
// are joined by hardware barriers.  More slots go to as many CTAs as they fill, in
// three launches (count, scan, place): a cluster's 16 SMs are then bound by their
// scattered stores.
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
#include "overlap.h"
#include "ptx.cuh"

namespace {

using namespace gemm103;

// ------------------------------------------------------------------------ sort

constexpr int kSortThreads = 1024;
constexpr int kSortCluster = 16;             // CTAs at most
constexpr int kHeld = 8;                     // batches of 32 slots a warp holds in registers
// Slots of the one-launch form: what its 16 CTAs hold (65536 slots: 9.9 us).
// 458752 slots of 999 experts: 44 us by it, in several turns, 18 by three launches.
constexpr int64_t kOneLaunch = 16ll * 32 * 32 * kHeld;
// Slots of a CTA of the three launches; the last CTA has the rest as well, so that
// every CTA's part of pos has room for its counts.
constexpr int32_t kCtaSlots = 4096;
static_assert(kCtaSlots >= EXPERT_MAX && 2 * kCtaSlots <= 32 * 32 * kHeld, "counts fit in pos, slots in registers");

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

// The lanes whose key is this lane's, of `bits` bits: a vote per bit.  (match.any takes
// longer: 65536 slots of 128 experts 10.9 us with it, 9.9 this way.)
__device__ __forceinline__ uint32_t sort_peers(int32_t key, int32_t bits) {
    uint32_t peers = 0xffffffffu;
    for (int32_t b = 0; b < bits; ++b) {
        const bool on = (key >> b) & 1;
        const uint32_t m = __ballot_sync(0xffffffffu, on);
        peers &= on ? m : ~m;
    }
    return peers;
}

// Rank of this lane's slot among the warp's slots of its expert so far, which are
// counted in `line`.
__device__ __forceinline__ int32_t sort_rank(int32_t* line, int32_t key, uint32_t peers, int32_t E, int lane) {
    const int32_t before = __popc(peers & ((1u << lane) - 1u));
    const int32_t seen = key < E ? line[key] : 0;
    __syncwarp();
    if (before == 0 && key < E) line[key] = seen + __popc(peers);
    __syncwarp();
    return seen + before;
}

// The offsets from the experts' totals (thread e: expert e's, `all`): the slots of
// lower experts.
__device__ __forceinline__ int32_t sort_offsets(int32_t all, int32_t* warp_sum) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    return below + incl - all;
}

// Expert e's counts in the CTAs of lower rank of the cluster, and in all of them.
__device__ __forceinline__ void sort_exchange(const int32_t* total, int32_t e, int32_t rank, int32_t ctas,
                                              int32_t& lower, int32_t& all) {
    int32_t c[kSortCluster];
    #pragma unroll
    for (int32_t r = 0; r < kSortCluster; ++r) {
        c[r] = 0;
        if (r < ctas)
            asm volatile("ld.shared::cluster.s32 %0, [%1];"
                         : "=r"(c[r])
                         : "r"(map_to_rank(smem_addr(total + e), static_cast<uint32_t>(r)))
                         : "memory");
    }
    lower = all = 0;
    #pragma unroll
    for (int32_t r = 0; r < kSortCluster; ++r) {
        lower += r < rank ? c[r] : 0;
        all += c[r];
    }
}

// PLACE false: the whole sort, by one cluster.  PLACE true: the last of three
// launches, any number of CTAs, each of which finds the first places of its slots in
// its own part of pos.
template <typename ID, bool PLACE>
__global__ void __launch_bounds__(kSortThreads) expert_sort_kernel(const SortParams p) {
    extern __shared__ int32_t sort_smem[];
    int32_t* hist = sort_smem;                               // [warps][E]
    int32_t* total = hist + p.warps * p.E;                   // [E] this CTA's
    int32_t* base = total + p.E;                             // [E]
    __shared__ int32_t warp_sum[32];
    __shared__ int32_t kept;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t rank = PLACE ? static_cast<int32_t>(blockIdx.x)
                               : p.ctas > 1 ? static_cast<int32_t>(cluster_ctarank()) : 0;

    for (int32_t i = threadIdx.x; i < p.warps * p.E; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    grid_dependency_wait();
    grid_dependents_launch();

    // count
    int32_t piece = p.piece, cta_first = rank * p.warps * p.piece;
    if constexpr (PLACE) {
        cta_first = rank * kCtaSlots;
        if (rank == p.ctas - 1) piece = ((p.n - cta_first + 31) / 32 + p.warps - 1) / p.warps * 32;
    }
    const int32_t first = cta_first + warp * piece;
    int32_t* line = hist + warp * p.E;
    const int32_t bits = 32 - __clz(p.E);                    // keys 0 .. E
    const int32_t e = threadIdx.x;                           // blockDim.x >= E
    if (PLACE && e < p.E) base[e] = p.pos[cta_first + e];
    int32_t key[kHeld], at[kHeld];
    if (warp < p.warps) {
        uint32_t peers[kHeld];
        #pragma unroll
        for (int b = 0; b < kHeld; ++b)
            key[b] = b * 32 < piece ? sort_key<ID>(p, first + b * 32 + lane) : p.E;
        #pragma unroll
        for (int b = 0; b < kHeld; ++b)
            if (b * 32 < piece) peers[b] = sort_peers(key[b], bits);
        #pragma unroll
        for (int b = 0; b < kHeld; ++b)
            if (b * 32 < piece) at[b] = sort_rank(line, key[b], peers[b], p.E, lane);
    }
    __syncthreads();

    // lines -> prefixes over the warps; the CTA's totals
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
    if constexpr (PLACE) {
        if (threadIdx.x == 0) kept = p.offsets[p.E];
    } else {
        int32_t lower = 0, all = mine;
        if (p.ctas > 1) {
            cluster_sync_all();
            if (e < p.E) sort_exchange(total, e, rank, p.ctas, lower, all);
            __syncwarp();
            // (the wait, before the end, keeps every CTA's memory until all have read it)
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        }
        const int32_t offset = sort_offsets(all, warp_sum);
        if (e < p.E) {
            base[e] = offset + lower;
            if (rank == 0) p.offsets[e] = offset;
            if (e == p.E - 1) {
                kept = offset + all;
                if (rank == 0) p.offsets[p.E] = offset + all;
            }
        }
    }
    __syncthreads();

    // place
    if (warp < p.warps) {
        #pragma unroll
        for (int b = 0; b < kHeld; ++b) {
            const int32_t slot = first + b * 32 + lane;
            if (b * 32 >= piece || slot >= p.n) continue;
            const int32_t i = key[b] < p.E ? base[key[b]] + line[key[b]] + at[b] : -1;
            p.pos[slot] = i;
            if (i >= 0 && p.order != nullptr) p.order[i] = slot;
        }
    }
    if (p.order != nullptr)
        for (int64_t i = static_cast<int64_t>(kept) + static_cast<int64_t>(rank) * blockDim.x + threadIdx.x; i < p.n;
             i += static_cast<int64_t>(p.ctas) * blockDim.x)
            p.order[i] = -1;
    if (!PLACE && p.ctas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The first of three launches: a CTA's counts, into its own part of pos.  (The order
// of the atomics does not matter to sums of integers.)
template <typename ID>
__global__ void __launch_bounds__(kSortThreads) expert_count_kernel(const SortParams p) {
    __shared__ int32_t count[EXPERT_MAX];
    for (int32_t i = threadIdx.x; i < p.E; i += blockDim.x) count[i] = 0;
    __syncthreads();
    grid_dependency_wait();
    grid_dependents_launch();
    const int32_t first = static_cast<int32_t>(blockIdx.x) * kCtaSlots;
    const int32_t behind = blockIdx.x + 1 == gridDim.x ? p.n : first + kCtaSlots;
    #pragma unroll 4
    for (int32_t i = first + static_cast<int32_t>(threadIdx.x); i < behind; i += kSortThreads) {
        const int32_t key = sort_key<ID>(p, i);
        if (key < p.E) atomicAdd(&count[key], 1);
    }
    __syncthreads();
    for (int32_t i = threadIdx.x; i < p.E; i += blockDim.x) p.pos[first + i] = count[i];
}

// The second: one cluster turns the counts into first places, and writes the offsets.
__global__ void __launch_bounds__(kSortThreads) expert_scan_kernel(const SortParams p, int32_t counted) {
    __shared__ int32_t total[EXPERT_MAX];
    __shared__ int32_t warp_sum[32];
    grid_dependency_wait();
    grid_dependents_launch();
    const int32_t rank = static_cast<int32_t>(cluster_ctarank()), ctas = p.ctas;
    const int32_t r0 = static_cast<int32_t>(static_cast<int64_t>(counted) * rank / ctas);
    const int32_t r1 = static_cast<int32_t>(static_cast<int64_t>(counted) * (rank + 1) / ctas);
    const int32_t e = threadIdx.x;
    int32_t mine = 0;
    if (e < p.E) {
        #pragma unroll 8
        for (int32_t r = r0; r < r1; ++r) mine += p.pos[r * kCtaSlots + e];
        total[e] = mine;
    }
    cluster_sync_all();
    int32_t lower = 0, all = 0;
    if (e < p.E) sort_exchange(total, e, rank, ctas, lower, all);
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    const int32_t offset = sort_offsets(all, warp_sum);
    if (e < p.E) {
        int32_t at = offset + lower;
        #pragma unroll 8
        for (int32_t r = r0; r < r1; ++r) {
            const int32_t c = p.pos[r * kCtaSlots + e];
            p.pos[r * kCtaSlots + e] = at;
            at += c;
        }
        if (rank == 0) {
            p.offsets[e] = offset;
            if (e == p.E - 1) p.offsets[p.E] = offset + all;
        }
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

cudaLaunchConfig_t sort_config(int grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                               cudaLaunchAttribute* attr) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cfg;
}

template <typename ID, bool PLACE>
cudaError_t launch_sort(const SortParams& p, cudaStream_t stream) {
    auto kern = expert_sort_kernel<ID, PLACE>;
    const size_t smem = static_cast<size_t>(p.warps + 2) * p.E * 4;
    static DeviceLimits limit;
    const cudaError_t set = limit.raise(smem, [&] {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        return e != cudaSuccess ? e
                                : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       static_cast<int>(smem));
    });
    if (set != cudaSuccess) return set;
    int threads = (p.E + 31) / 32 * 32;
    if (threads < p.warps * 32) threads = p.warps * 32;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = sort_config(p.ctas, threads, smem, PLACE ? 1 : p.ctas, stream, attr);
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename ID>
cudaError_t run_sort(SortParams p, cudaStream_t stream) {
    const int64_t batches = (static_cast<int64_t>(p.n) + 31) / 32;
    if (p.n <= kOneLaunch) {
        // CTAs: one while a warp has no more than two batches
        p.ctas = 1;
        while (p.ctas < kSortCluster && batches > 32ll * 2 * p.ctas) p.ctas *= 2;
        const int64_t warps = (batches + p.ctas - 1) / p.ctas;
        p.warps = static_cast<int32_t>(warps < 1 ? 1 : warps > 32 ? 32 : warps);
        const int64_t cells = static_cast<int64_t>(p.ctas) * p.warps;
        p.piece = static_cast<int32_t>((batches + cells - 1) / cells * 32);
        return launch_sort<ID, false>(p, stream);
    }
    cudaLaunchAttribute attr[2];
    const int ctas = p.n / kCtaSlots;
    cudaLaunchConfig_t cfg = sort_config(ctas, kSortThreads, 0, 1, stream, attr);
    cudaError_t e = cudaLaunchKernelEx(&cfg, expert_count_kernel<ID>, p);
    if (e != cudaSuccess) return e;
    p.ctas = 8;
    cfg = sort_config(8, kSortThreads, 0, 8, stream, attr);
    e = cudaLaunchKernelEx(&cfg, expert_scan_kernel, p, ctas);
    if (e != cudaSuccess) return e;
    p.ctas = ctas;
    p.warps = 32;
    p.piece = kCtaSlots / 32;
    return launch_sort<ID, true>(p, stream);
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

// V elements of a row for one thread of a group: a 16-byte vector, or, A false (rows
// that do not all start on 16 bytes), V single elements a group's width apart, which
// keeps both the accesses of a warp contiguous and as many in flight.
template <typename T, int V, bool A>
struct alignas(A ? sizeof(T) * V : sizeof(T)) Pack {
    T e[V];
};
template <typename T, int V, bool A>
__device__ __forceinline__ Pack<T, V, A> load_pack(const T* p, int32_t step, int32_t left) {
    Pack<T, V, A> r;
    if constexpr (A) {
        r = *reinterpret_cast<const Pack<T, V, A>*>(p);
    } else {
        #pragma unroll
        for (int i = 0; i < V; ++i) r.e[i] = i * step < left ? p[i * step] : from_f<T>(0.0f);
    }
    return r;
}
template <typename T, int V, bool A>
__device__ __forceinline__ void store_pack(T* p, int32_t step, int32_t left, const Pack<T, V, A>& r) {
    if constexpr (A) {
        *reinterpret_cast<Pack<T, V, A>*>(p) = r;
    } else {
        #pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * step < left) p[i * step] = r.e[i];
    }
}

// Sums of v[0..7] over a group of threads (whole warps); the group's thread j has
// the sum of v[j] for j < 8.  By halving: a lane keeps half its values and gives
// the other half away, so 9 shuffles do for 8 sums.  `red` is read again two calls
// later at the earliest (callers take two in turn): one barrier, the group's own, per
// call.
__device__ __forceinline__ float group_sums(float (&v)[kTurn], int log_group, float (*red)[kTurn], int lane, int warp) {
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
    if ((lane & 3) == 0) red[warp][at] = s;
    const int group = 1 << log_group, mine = static_cast<int>(threadIdx.x) >> log_group;
    if (group > 32) asm volatile("bar.sync %0, %1;" ::"r"(1 + mine), "r"(group) : "memory");
    else __syncwarp();
    const int g = static_cast<int>(threadIdx.x) & (group - 1), warps = group >> 5;
    float t = 0.0f;
    if (g < kTurn)
        for (int w = 0; w < warps; ++w) t += red[mine * warps + w][g];
    return t;
}

// A group's share of the work: token t, and columns c0, c0 + step, ... below c1 (each
// the first of V).
struct Place {
    int64_t t;
    int32_t g, group;                        // thread of its group, threads of the group
    int32_t c0, c1, step;
    bool live;
};
template <int V, bool A>
__device__ __forceinline__ Place place_of(const RowsParams& p, int64_t unit) {
    Place a;
    a.group = 1 << p.log_group;
    a.g = static_cast<int32_t>(threadIdx.x) & (a.group - 1);
    int32_t chunk = 0;
    a.t = unit;
    if (p.chunks > 1) {
        a.t = unit / p.chunks;
        chunk = static_cast<int32_t>(unit - a.t * p.chunks);
    }
    a.live = a.t < p.T;
    a.step = a.group * V;
    const int32_t D = static_cast<int32_t>(p.D), whole = A ? D / V * V : D;
    const int32_t per = ((whole + p.chunks - 1) / p.chunks + a.step - 1) / a.step * a.step;
    const int32_t first = chunk * per;
    a.c0 = first + a.g * (A ? V : 1);
    a.c1 = p.chunks > 1 && first + per < whole ? first + per : whole;
    return a;
}

// Positions and weights of choices j0 .. j0 + 7 of a token; -1 where there is none.
__device__ __forceinline__ void load_choices(const RowsParams& p, const Place& a, int64_t j0, int32_t (&at)[kTurn],
                                             float (&w)[kTurn]) {
    #pragma unroll
    for (int j = 0; j < kTurn; ++j) {
        const bool is = a.live && j0 + j < p.k;
        const int32_t i = is ? p.pos[a.t * p.k + j0 + j] : -1;
        at[j] = i >= 0 && i < p.rows ? i : -1;
        w[j] = is && p.weight != nullptr ? load_bias_elem(p.weight, p.wtype, a.t * p.ldw + j0 + j) : 1.0f;
    }
}

// A token's row, weighted, to its k places; DOT: and the dot products of the row
// with what is at these places in rows_in.
template <typename T, int V, bool A, bool DOT>
__global__ void __launch_bounds__(kRowThreads, DOT ? 2 : 4) rows_out_kernel(const RowsParams p) {
    __shared__ float red[2][DOT ? kRowThreads / 32 : 1][kTurn];
    grid_dependency_wait();
    grid_dependents_launch();
    const int32_t D = static_cast<int32_t>(p.D), tail = A ? D % V : 0;
    const T* in = static_cast<const T*>(p.rows_in);
    T* out = static_cast<T*>(p.rows_out);
    const Place a = place_of<V, A>(p, static_cast<int64_t>(blockIdx.x) * (kRowThreads >> p.log_group) +
                                          (threadIdx.x >> p.log_group));
    if (!DOT && !a.live) return;
    int32_t at[kTurn];
    float w[kTurn];
    load_choices(p, a, 0, at, w);
    const T* x = static_cast<const T*>(p.tok_in) + (a.live ? a.t : 0) * p.ld_tok_in;
    for (int64_t j0 = 0; j0 < p.k; j0 += kTurn) {
        float dot[kTurn];
        #pragma unroll
        for (int j = 0; j < kTurn; ++j) dot[j] = 0.0f;
        if (j0 > 0) load_choices(p, a, j0, at, w);
        if (a.live) {
            for (int32_t col = a.c0; col < a.c1; col += a.step) {
                const int32_t left = a.c1 - col;
                const Pack<T, V, A> xv = load_pack<T, V, A>(x + col, a.group, left);
                Pack<T, V, A> o[DOT ? kTurn : 1];
                if constexpr (DOT) {
                    #pragma unroll
                    for (int j = 0; j < kTurn; ++j)
                        if (at[j] >= 0) o[j] = load_pack<T, V, A>(in + at[j] * p.ld_rows_in + col, a.group, left);
                }
                #pragma unroll
                for (int j = 0; j < kTurn; ++j) {
                    if (at[j] < 0) continue;
                    Pack<T, V, A> r;
                    #pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float f = to_f<T>(xv.e[i]);
                        if constexpr (DOT) {
                            if (A || i * a.group < left) dot[j] = fmaf(f, to_f<T>(o[j].e[i]), dot[j]);
                        }
                        r.e[i] = from_f<T>(f * w[j]);
                    }
                    if (!DOT || out != nullptr)
                        store_pack<T, V, A>(out + at[j] * p.ld_rows_out + col, a.group, left, r);
                }
            }
            // the elements behind the last vector, which may be more than the group's threads
            for (int32_t col = a.c1 + a.g; a.c1 + tail == D && col < D; col += a.group) {
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
            const float s = group_sums(dot, p.log_group, red[(j0 / kTurn) & 1], threadIdx.x & 31, threadIdx.x >> 5);
            if (a.live && a.g < kTurn && j0 + a.g < p.k)
                store_elem(p.dweight, p.dwtype, a.t * p.lddw + j0 + a.g, s);
        }
    }
}

// The weighted sum of a token's k rows; DOT: and the rows' dot products with the
// token's row in tok_in.
template <typename T, int V, bool A, bool DOT>
__global__ void __launch_bounds__(kRowThreads, DOT ? 2 : 3) rows_in_kernel(const RowsParams p) {
    __shared__ float red[2][DOT ? kRowThreads / 32 : 1][kTurn];
    grid_dependency_wait();
    grid_dependents_launch();
    const int32_t D = static_cast<int32_t>(p.D), tail = A ? D % V : 0;
    const T* in = static_cast<const T*>(p.rows_in);
    const Place a = place_of<V, A>(p, static_cast<int64_t>(blockIdx.x) * (kRowThreads >> p.log_group) +
                                          (threadIdx.x >> p.log_group));
    if (!DOT && !a.live) return;
    int32_t at[kTurn];
    float w[kTurn];
    load_choices(p, a, 0, at, w);
    const int64_t tt = a.live ? a.t : 0;
    const T* x = DOT ? static_cast<const T*>(p.tok_in) + tt * p.ld_tok_in : nullptr;
    T* y = p.tok_out != nullptr ? static_cast<T*>(p.tok_out) + tt * p.ld_tok_out : nullptr;
    float dot[kTurn];
    #pragma unroll
    for (int j = 0; j < kTurn; ++j) dot[j] = 0.0f;
    if (a.live) {
        for (int32_t col = a.c0; col < a.c1; col += a.step) {
            const int32_t left = a.c1 - col;
            Pack<T, V, A> xv;
            if constexpr (DOT) xv = load_pack<T, V, A>(x + col, a.group, left);
            float acc[V];
            #pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = 0.0f;
            for (int64_t j0 = 0;;) {
                Pack<T, V, A> r[kTurn];
                #pragma unroll
                for (int j = 0; j < kTurn; ++j)
                    if (at[j] >= 0) r[j] = load_pack<T, V, A>(in + at[j] * p.ld_rows_in + col, a.group, left);
                #pragma unroll
                for (int j = 0; j < kTurn; ++j) {
                    if (at[j] < 0) continue;
                    #pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float f = to_f<T>(r[j].e[i]);
                        if constexpr (DOT) {
                            if (j0 == 0 && (A || i * a.group < left)) dot[j] = fmaf(to_f<T>(xv.e[i]), f, dot[j]);
                        }
                        acc[i] = fmaf(w[j], f, acc[i]);
                    }
                }
                if (p.k <= kTurn) break;
                j0 = j0 + kTurn < p.k ? j0 + kTurn : 0;
                load_choices(p, a, j0, at, w);
                if (j0 == 0) break;
            }
            Pack<T, V, A> o;
            #pragma unroll
            for (int i = 0; i < V; ++i) o.e[i] = from_f<T>(acc[i]);
            if (!DOT || y != nullptr) store_pack<T, V, A>(y + col, a.group, left, o);
        }
        // the elements behind the last vector, which may be more than the group's threads
        for (int32_t col = a.c1 + a.g; a.c1 + tail == D && col < D; col += a.group) {
            const float xf = DOT ? to_f<T>(x[col]) : 0.0f;
            float acc = 0.0f;
            for (int64_t j0 = 0;;) {
                #pragma unroll
                for (int j = 0; j < kTurn; ++j) {
                    if (at[j] < 0) continue;
                    const float f = to_f<T>(in[at[j] * p.ld_rows_in + col]);
                    if constexpr (DOT) {
                        if (j0 == 0) dot[j] = fmaf(xf, f, dot[j]);
                    }
                    acc = fmaf(w[j], f, acc);
                }
                if (p.k <= kTurn) break;
                j0 = j0 + kTurn < p.k ? j0 + kTurn : 0;
                load_choices(p, a, j0, at, w);
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
                load_choices(p, a, j0, at, w);
                if (a.live) {
                    for (int32_t col = a.g; col < D; col += a.group) {
                        const float xf = to_f<T>(x[col]);
                        #pragma unroll
                        for (int j = 0; j < kTurn; ++j)
                            if (at[j] >= 0) dot[j] = fmaf(xf, to_f<T>(in[at[j] * p.ld_rows_in + col]), dot[j]);
                    }
                }
            }
            const float s = group_sums(dot, p.log_group, red[(j0 / kTurn) & 1], threadIdx.x & 31, threadIdx.x >> 5);
            if (a.live && a.g < kTurn && j0 + a.g < p.k)
                store_elem(p.dweight, p.dwtype, a.t * p.lddw + j0 + a.g, s);
        }
    }
}

// ------------------------------------------------------------- rows in a ring

// rows_in, without or with dot products, for many tokens of at most kTurn choices on
// rows of vectors: what is read (the k rows, and for dot products the token's own)
// passes through a ring of `cp.async` slots in
// shared memory, which only the copying thread reads, so that one CTA per SM keeps
// its 180 KB of loads in flight without registers for them and without a barrier.
// A stage is one vector of every row per thread; a token takes `passes` of them.  A
// group has consecutive tokens, and their positions and weights come in batches, one
// batch ahead: a load waits behind all that is in flight, so positions that are
// fetched a token ahead come too late.  (8192 tokens x 8 of 4096 bf16, whose bytes
// take 89 us: 98; by direct loads, three CTAs of 80 registers, 137; by this ring with
// positions a token ahead 130.  rows_out with dot products, which writes as much as it
// reads, gains nothing: 203, directly 187.)

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// K: choices at most (4 or 8).
template <bool DOT, int K>
struct Ring {
    static constexpr int kRows = K + (DOT ? 1 : 0);
    static constexpr int kStageBytes = kRows * kRowThreads * 16;
    static constexpr int kTableBytes = 2 * 2 * kRowThreads * 8;      // two batches of two entries per thread
    static constexpr int kStages = (230400 - kTableBytes) / kStageBytes;
    // A batch (2 group / K tokens, a group at least 32 threads) is no shorter than the
    // ring, so that what is read is in the batch before that of the loads at most.
    static_assert(2 * 32 / K >= kStages - 1, "two batches are enough");
};

template <typename T, bool DOT, int K>
__global__ void __launch_bounds__(kRowThreads, 1) rows_ring_kernel(const RowsParams p) {
    using R = Ring<DOT, K>;
    constexpr int V = 16 / sizeof(T);
    extern __shared__ uint4 ring_smem[];
    __shared__ float red[2][kRowThreads / 32][kTurn];
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t group = 1 << p.log_group, g = static_cast<int32_t>(threadIdx.x) & (group - 1);
    const int32_t which = static_cast<int32_t>(threadIdx.x) >> p.log_group, per_cta = kRowThreads >> p.log_group;
    const int32_t nvec = static_cast<int32_t>(p.D / V), passes = (nvec + group - 1) >> p.log_group;
    const int32_t batch = 2 * group / K;                                // tokens
    const int64_t groups = static_cast<int64_t>(gridDim.x) * per_cta;
    const int64_t share = (p.T + groups - 1) / groups;
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * per_cta + which) * share;
    const int64_t t1 = t0 + share < p.T ? t0 + share : p.T;
    const T* in = static_cast<const T*>(p.rows_in);
    const T* tok = static_cast<const T*>(p.tok_in);
    // tables of this group: [two batches][tokens][K]
    int32_t* at_table = reinterpret_cast<int32_t*>(ring_smem + R::kStages * (R::kRows * kRowThreads)) + which * 4 * group;
    float* w_table = reinterpret_cast<float*>(ring_smem + R::kStages * (R::kRows * kRowThreads)) +
                     4 * kRowThreads + which * 4 * group;
    auto group_sync = [&] {
        if (group > 32) asm volatile("bar.sync %0, %1;" ::"r"(1 + which), "r"(group) : "memory");
        else __syncwarp();
    };

    // two entries of the batch that begins at token t, for this thread
    int32_t at_fetched[2];
    float w_fetched[2];
    auto fetch = [&](int64_t t) {
        #pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int32_t e = q * group + g, j = e % K;
            const int64_t n = t + e / K;
            const bool is = n < t1 && j < p.k;
            const int32_t i = is ? p.pos[n * p.k + j] : -1;
            at_fetched[q] = i >= 0 && i < p.rows ? i : -1;
            w_fetched[q] = is && p.weight != nullptr ? load_bias_elem(p.weight, p.wtype, n * p.ldw + j) : 1.0f;
        }
    };

    // The loads: next token, its pass, place in its batch, the batch's half of the
    // table, and the stage.
    int64_t t_load = t0;
    int32_t pass_load = 0, in_batch = 0, half_load = 1, stage_load = 0;
    fetch(t0);
    auto load = [&] {
        if (t_load < t1) {
            if (pass_load == 0 && in_batch == 0) {
                // Its batch to the table, over the batch before last: the group's
                // threads are all here, so none is further back than the last.
                half_load ^= 1;
                group_sync();
                #pragma unroll
                for (int q = 0; q < 2; ++q) {
                    at_table[half_load * 2 * group + q * group + g] = at_fetched[q];
                    w_table[half_load * 2 * group + q * group + g] = w_fetched[q];
                }
                group_sync();
                fetch(t_load + batch);
            }
            const int32_t v = (pass_load << p.log_group) + g;
            const uint32_t to = smem_addr(ring_smem + stage_load * (R::kRows * kRowThreads) + threadIdx.x);
            if (v < nvec) {
                int32_t at[K];
                #pragma unroll
                for (int j = 0; j < K; j += 4)
                    *reinterpret_cast<int4*>(at + j) =
                        *reinterpret_cast<const int4*>(at_table + half_load * 2 * group + in_batch * K + j);
                #pragma unroll
                for (int j = 0; j < K; ++j)
                    if (at[j] >= 0) cp_async16(to + j * (kRowThreads * 16), in + at[j] * p.ld_rows_in + v * V);
                if (DOT) cp_async16(to + K * (kRowThreads * 16), tok + t_load * p.ld_tok_in + v * V);
            }
            stage_load = stage_load + 1 == R::kStages ? 0 : stage_load + 1;
            if (++pass_load == passes) {
                pass_load = 0;
                ++t_load;
                in_batch = in_batch + 1 == batch ? 0 : in_batch + 1;
            }
        }
        cp_async_commit();
    };
    #pragma unroll 1
    for (int s = 0; s < R::kStages - 1; ++s) load();

    int32_t stage = 0, odd = 0, here = 0, half = 0;
    for (int64_t t = t0; t < t1; ++t, odd ^= 1) {
        alignas(16) int32_t at[K];
        alignas(16) float w[K];
        float dot[kTurn];
        #pragma unroll
        for (int j = 0; j < K; j += 4) {
            *reinterpret_cast<int4*>(at + j) = *reinterpret_cast<const int4*>(at_table + half * 2 * group + here * K + j);
            *reinterpret_cast<float4*>(w + j) = *reinterpret_cast<const float4*>(w_table + half * 2 * group + here * K + j);
        }
        if (++here == batch) here = 0, half ^= 1;
        #pragma unroll
        for (int j = 0; j < kTurn; ++j) dot[j] = 0.0f;
        #pragma unroll 1
        for (int32_t c = 0; c < passes; ++c) {
            load();                                      // into the stage read in the turn before
            cp_async_wait<R::kStages - 1>();
            const int32_t v = (c << p.log_group) + g;
            if (v < nvec) {
                const uint4* from = ring_smem + stage * (R::kRows * kRowThreads) + threadIdx.x;
                float x[V], acc[V];
                if constexpr (DOT) {
                    const uint4 u = from[K * kRowThreads];
                    const T* e = reinterpret_cast<const T*>(&u);
                    #pragma unroll
                    for (int i = 0; i < V; ++i) x[i] = to_f<T>(e[i]);
                }
                #pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = 0.0f;
                #pragma unroll
                for (int j = 0; j < K; ++j) {
                    if (at[j] < 0) continue;
                    const uint4 u = from[j * kRowThreads];
                    const T* e = reinterpret_cast<const T*>(&u);
                    #pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float f = to_f<T>(e[i]);
                        if constexpr (DOT) dot[j] = fmaf(x[i], f, dot[j]);
                        acc[i] = fmaf(w[j], f, acc[i]);
                    }
                }
                if (p.tok_out != nullptr) {
                    Pack<T, V, true> r;
                    #pragma unroll
                    for (int i = 0; i < V; ++i) r.e[i] = from_f<T>(acc[i]);
                    *reinterpret_cast<Pack<T, V, true>*>(static_cast<T*>(p.tok_out) + t * p.ld_tok_out + v * V) = r;
                }
            }
            stage = stage + 1 == R::kStages ? 0 : stage + 1;
        }
        if constexpr (DOT) {
            const float s = group_sums(dot, p.log_group, red[odd], lane, warp);
            if (g < p.k && g < kTurn) store_elem(p.dweight, p.dwtype, t * p.lddw + g, s);
        }
    }
}

enum RowsKind { kOut, kOutDot, kIn, kInDot };

template <typename T, int V, bool A>
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
        case kOut: return cudaLaunchKernelEx(&cfg, rows_out_kernel<T, V, A, false>, p);
        case kOutDot: return cudaLaunchKernelEx(&cfg, rows_out_kernel<T, V, A, true>, p);
        case kIn: return cudaLaunchKernelEx(&cfg, rows_in_kernel<T, V, A, false>, p);
        default: return cudaLaunchKernelEx(&cfg, rows_in_kernel<T, V, A, true>, p);
    }
}

template <typename T, bool DOT, int K>
cudaError_t launch_ring(const RowsParams& p, int sms, cudaStream_t stream) {
    using R = Ring<DOT, K>;
    auto kern = rows_ring_kernel<T, DOT, K>;
    constexpr int kSmem = R::kStages * R::kStageBytes + R::kTableBytes;
    static DeviceLimits limit;
    const cudaError_t set = limit.raise(kSmem, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    });
    if (set != cudaSuccess) return set;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    const int64_t per = kRowThreads >> p.log_group, ctas = (p.T + per - 1) / per;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas < sms ? ctas : sms), 1, 1);
    cfg.blockDim = dim3(kRowThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}
template <typename T>
cudaError_t launch_ring(RowsKind kind, const RowsParams& p, int sms, cudaStream_t stream) {
    if (kind == kInDot)
        return p.k <= 4 ? launch_ring<T, true, 4>(p, sms, stream) : launch_ring<T, true, 8>(p, sms, stream);
    return p.k <= 4 ? launch_ring<T, false, 4>(p, sms, stream) : launch_ring<T, false, 8>(p, sms, stream);
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

// CTAs write outputs while others still read inputs: each output has to be apart from
// every input, and from the others.
template <int INS, int OUTS>
bool outputs_apart(const Region (&in)[INS], const Region (&out)[OUTS]) {
    for (int o = 0; o < OUTS; ++o) {
        for (int i = 0; i < INS; ++i)
            if (overlap(out[o], in[i])) return false;
        for (int i = 0; i < o; ++i)
            if (overlap(out[o], out[i])) return false;
    }
    return true;
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
    auto matrix = [](const void* q, int64_t rows, int64_t ld, int64_t cols, int64_t bytes) {
        return Region{q, rows, ld * bytes, cols * bytes};
    };
    // (dYs may be Ys: a row's elements are read before they are written, by the same thread)
    const bool in_place = p.rows_in == p.rows_out && (p.ld_rows_in == p.ld_rows_out || p.rows <= 1);
    const Region in[] = {matrix(p.tok_in, p.T, p.ld_tok_in, p.D, es),
                         matrix(in_place ? nullptr : p.rows_in, p.rows, p.ld_rows_in, p.D, es),
                         matrix(p.pos, p.T, p.k, p.k, 4), matrix(p.weight, p.T, p.ldw, p.k, esize(p.wtype))};
    const Region out_of[] = {matrix(p.tok_out, p.T, p.ld_tok_out, p.D, es),
                             matrix(p.rows_out, p.rows, p.ld_rows_out, p.D, es),
                             matrix(p.dweight, p.T, p.lddw, p.k, esize(p.dwtype))};
    if (!outputs_apart(in, out_of)) return GEMM_ERR_INVALID_VALUE;

    // 16-byte vectors where every row of every matrix starts on one
    const int32_t per = 16 / es;
    auto vector = [&](const void* q, int64_t ld) { return q == nullptr || (aligned(q, 16) && ld % per == 0); };
    const bool vec = vector(p.tok_in, p.ld_tok_in) && vector(p.rows_in, p.ld_rows_in) &&
                     vector(p.tok_out, p.ld_tok_out) && vector(p.rows_out, p.ld_rows_out);
    const int64_t nvec = vec ? p.D / per : (p.D + 3) / 4;
    // Threads per token: as many as it has vectors, up to a CTA's; whole warps
    // where they add up dot products.
    p.log_group = dot ? 5 : 2;
    while (p.log_group < 8 && (1 << p.log_group) < nvec) ++p.log_group;
    p.chunks = 1;
    cudaError_t e;
    const int64_t waves = p.T >> (8 - (p.log_group < 5 ? 5 : p.log_group));
    if (vec && p.D % per == 0 && (kind == kIn || kind == kInDot) && p.k <= kTurn && nvec >= 32 && waves >= 8 * sms) {
        // tokens enough to fill the ring several times
        if (p.log_group < 5) p.log_group = 5;
        e = dtype == GEMM_F32    ? launch_ring<float>(kind, p, sms, stream)
            : dtype == GEMM_BF16 ? launch_ring<__nv_bfloat16>(kind, p, sms, stream)
                                 : launch_ring<__half>(kind, p, sms, stream);
        if (e == cudaSuccess) return GEMM_OK;
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    if (!dot && p.T < 2 * sms && nvec > 64) {
        // few tokens: their columns over more SMs
        p.log_group = 6;
        p.chunks = static_cast<int32_t>((nvec + 63) / 64);
    }
    if (dtype == GEMM_F32)
        e = vec ? launch_rows<float, 4, true>(kind, p, stream) : launch_rows<float, 4, false>(kind, p, stream);
    else if (dtype == GEMM_BF16)
        e = vec ? launch_rows<__nv_bfloat16, 8, true>(kind, p, stream)
                : launch_rows<__nv_bfloat16, 4, false>(kind, p, stream);
    else
        e = vec ? launch_rows<__half, 8, true>(kind, p, stream)
                : launch_rows<__half, 4, false>(kind, p, stream);
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
    const Region in[] = {{ids, T, ldids * id_bytes, k * id_bytes}};
    const Region out[] = {{pos, 1, T * k * 4, T * k * 4}, {offsets, 1, (E + 1) * 4, (E + 1) * 4}, {order, 1, T * k * 4, T * k * 4}};
    if (!outputs_apart(in, out)) return GEMM_ERR_INVALID_VALUE;
    SortParams p = {};
    p.ids = ids, p.ldids = T == 1 ? k : ldids;
    p.n = static_cast<int32_t>(T * k), p.k = static_cast<int32_t>(k), p.E = static_cast<int32_t>(E);
    p.pos = pos, p.offsets = offsets, p.order = order;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = id_bytes == 4 ? run_sort<int32_t>(p, s) : run_sort<int64_t>(p, s);
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
