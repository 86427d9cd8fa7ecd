// norm.cu -- host side of the norms around a block (include/norm_sm103.h):
// argument checks, the work split and the launches.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "device.h"
#include "norm_launch.h"
#include "norm_sm103.h"

namespace {

using namespace gemm103;
using namespace gemm103::nrm;

constexpr int64_t kSmemPerCta = 227 * 1024 - 256;
constexpr int64_t kSmemPerSm = 228 * 1024;
constexpr int64_t kMaxColumnsPerCta = 8192;

bool dtype_ok(int32_t t) { return t == GEMM_F16 || t == GEMM_BF16 || t == GEMM_F32; }
int64_t esize(int32_t t) { return t == GEMM_F32 ? 4 : 2; }
bool kind_ok(int32_t k) { return k == NORM_NONE || k == NORM_RMS || k == NORM_LAYER; }
bool aligned(const void* p, int64_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

bool pair_ok(int32_t x, int32_t z) { return x == z || x == GEMM_F32; }

// A matrix the call uses: NULL is refused where it is needed.
bool matrix_ok(const void* p, int64_t ld, int64_t N, int32_t dtype) {
    return p != nullptr && ld >= N && aligned(p, esize(dtype));
}

bool vector16(const void* p, int64_t ld, int32_t dtype) {
    return p == nullptr || (aligned(p, 16) && ld * esize(dtype) % 16 == 0);
}

gemm_status_t check_block(int64_t M, int64_t N, int32_t x_dtype, int32_t z_dtype,
                          const norm_block_t* b) {
    if (b == nullptr || M < 0 || N < 0 || M > INT32_MAX || N > INT32_MAX)
        return GEMM_ERR_INVALID_VALUE;
    if (!dtype_ok(x_dtype) || !dtype_ok(z_dtype) || !kind_ok(b->pre) || !kind_ok(b->post))
        return GEMM_ERR_INVALID_VALUE;
    if (!(b->eps > 0.0f) || std::isinf(b->eps) || !std::isfinite(b->scale))
        return GEMM_ERR_INVALID_VALUE;
    const void* vecs[] = {b->pre_weight, b->pre_bias, b->post_weight, b->post_bias, b->gate};
    for (const void* v : vecs) {
        if (v == nullptr) continue;
        if (!dtype_ok(b->vec_dtype) || !aligned(v, esize(b->vec_dtype))) return GEMM_ERR_INVALID_VALUE;
    }
    if (b->gate != nullptr && (b->gate_rows < 1 || b->ld_gate < N)) return GEMM_ERR_INVALID_VALUE;
    if (!pair_ok(x_dtype, z_dtype)) return GEMM_ERR_NOT_SUPPORTED;
    if (N > NORM_MAX_N) return GEMM_ERR_NOT_SUPPORTED;
    return GEMM_OK;
}

void fill_block(Params& p, int64_t M, int64_t N, const norm_block_t* b) {
    p.M = M;
    p.N = static_cast<int32_t>(N);
    p.wpre = b->pre_weight;
    p.bpre = b->pre_bias;
    p.wpost = b->post_weight;
    p.bpost = b->post_bias;
    p.gate = b->gate;
    p.ld_gate = b->gate ? b->ld_gate : 0;
    p.vec_dtype = b->vec_dtype;
    bool wide = true;
    const void* vecs[] = {b->pre_weight, b->pre_bias, b->post_weight, b->post_bias};
    for (const void* v : vecs) wide = wide && aligned(v, 16);
    if (b->gate) wide = wide && vector16(b->gate, b->ld_gate, b->vec_dtype);
    p.vec_aligned = wide ? 1 : 0;
    p.pre = b->pre;
    p.post = b->post;
    p.scale = b->scale;
    p.eps = b->eps;
    p.inv_n = 1.0f / static_cast<float>(N);
}

// Threads per row: the fewest of 32, 64, ... (and 384) whose `chunks8` chunks
// of 8 hold N.
int threads_for(int64_t N, int chunks8) {
    int t = 32;
    while (static_cast<int64_t>(t) * 8 * chunks8 < N) t *= 2;
    return t == 512 && N <= static_cast<int64_t>(384) * 8 * chunks8 ? 384 : t;
}

constexpr double kChunkCost = 32768.0;

struct Chunks {
    int64_t group_rows, groups, per_group, rows;
};

// Rows cut into chunks, each inside one group of the gate, for `resident` CTAs
// that work at a time on one each.  The size is the one whose waves take the
// shortest: a chunk costs its rows and, to fill its vectors and write its
// sums, about kChunkCost elements more.  (8192 x 4096, backward, 16 groups of
// the gate: 157 us in 160 chunks, two waves, 100 in 144.  512 groups: 148 in
// chunks of half a group and 179 of a whole one, which a cost of 8192 takes.)
Chunks chunks_for(int64_t M, int64_t N, int64_t gate_rows, int64_t resident) {
    Chunks c;
    c.group_rows = (gate_rows > 1 && gate_rows < M) ? gate_rows : (M > 0 ? M : 1);
    c.groups = ceil_div(M > 0 ? M : 1, c.group_rows);
    const int64_t per = ceil_div(resident, c.groups);
    double best = INFINITY;
    int64_t most = c.groups > 1 && per < 4 ? 4 : per;
    if (most > c.group_rows) most = c.group_rows;
    c.rows = ceil_div(c.group_rows, most);
    for (int64_t i = c.groups > 1 ? (most > 64 ? most - 64 : 1) : most; i <= most; ++i) {
        const int64_t rows = ceil_div(c.group_rows, i);
        const int64_t waves = ceil_div(c.groups * ceil_div(c.group_rows, rows), resident);
        const double cost = static_cast<double>(waves) * (static_cast<double>(rows) * static_cast<double>(N) + kChunkCost);
        if (cost < best) {
            best = cost;
            c.rows = rows;
        }
    }
    c.per_group = ceil_div(c.group_rows, c.rows);
    return c;
}

// Of the backward pass: a CTA, or a pair of them, per SM.
Chunks back_chunks(int64_t M, int64_t N, int64_t gate_rows, int sms) {
    const int64_t resident = N > kMaxColumnsPerCta ? sms / 2 : sms;
    return chunks_for(M, N, gate_rows, resident > 0 ? resident : 1);
}

void set_chunks(Params& p, const Chunks& c) {
    p.chunk_group_rows = c.group_rows;
    p.chunks_per_group = static_cast<int32_t>(c.per_group);
    p.chunk_rows = c.rows;
}

// Shared memory of a CTA of `groups` groups: exchange buffers for `sums` values,
// the n_par vectors, the groups' rings.
int64_t smem_for(const Params& p, int sums, int chunks8, int groups, int stages) {
    return groups * static_cast<int64_t>(p.T / 32 * 8 * sums) + static_cast<int64_t>(p.n_par) * chunks8 * 32 * p.T +
           static_cast<int64_t>(groups) * stages * p.slot_bytes;
}

// Groups per CTA and slots per group: the most rows worked on per SM among
// CTAs of up to `most` threads, all resident within `resident` threads, that
// have a second slot per group; of those the deepest rings, then the largest
// CTA (many small ones leave the default split of an SM's memory with
// room for few: 5 of 32 one-warp CTAs).  One slot only where two fit nowhere.  Returns CTAs per SM (at most
// `per_sm`), 0 where nothing fits.
int choose_cta(Params& p, int sums, int chunks8, int most, int resident, int per_sm, int& groups) {
    int64_t best = 0;
    int ctas = 0;
    for (int stages = kMaxStages; stages >= 1; --stages) {
        if (stages == 1 && best > 0) break;
        // (named barriers number the groups of more than a warp: 15 at most)
        // (a pair of CTAs has one exchange buffer and one barrier: one group)
        for (int g = 1; g * p.T <= most && (g <= 15 || p.T == 32) && (g == 1 || p.cluster == 1); g *= 2) {
            const int64_t bytes = smem_for(p, sums, chunks8, g, stages);
            if (bytes > kSmemPerCta) continue;
            int64_t n = kSmemPerSm / (bytes + 1024);
            if (n > resident / (g * p.T)) n = resident / (g * p.T);
            if (n > per_sm) n = per_sm;
            if (n * g > best || (n * g == best && stages == p.stages)) {
                best = n * g;
                ctas = static_cast<int>(n);
                groups = g;
                p.stages = stages;
            }
        }
    }
    return ctas;
}

gemm_status_t status_of(cudaError_t e) {
    if (e == cudaSuccess) return GEMM_OK;
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
}

cudaError_t run_forward(int32_t x, int32_t z, const Launch& l) {
    if (x == GEMM_F16) return forward_f16_f16(l);
    if (x == GEMM_BF16) return forward_bf16_bf16(l);
    if (z == GEMM_F16) return forward_f32_f16(l);
    if (z == GEMM_BF16) return forward_f32_bf16(l);
    return forward_f32_f32(l);
}

cudaError_t run_backward(int32_t x, int32_t z, const Launch& l) {
    if (x == GEMM_F16) return backward_f16_f16(l);
    if (x == GEMM_BF16) return backward_bf16_bf16(l);
    if (z == GEMM_F16) return backward_f32_f16(l);
    if (z == GEMM_BF16) return backward_f32_bf16(l);
    return backward_f32_f32(l);
}

template <typename K>
cudaError_t launch_sum(K kern, dim3 grid, int threads, const SumParams& s, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, s);
}

// The sums over the chunks: one step, or two where there are many chunks
// (`lines`, kSumSplits of them, hold the first step's); the gate's gradient
// beside it, or by its own kernel where it has many groups.
cudaError_t run_sum(SumParams s, float* lines, int sms, cudaStream_t stream) {
    const unsigned cols = static_cast<unsigned>(ceil_div(s.N, 32));
    const bool two = s.chunks > kSumOneStep;
    const bool own = s.d_gate != nullptr && (two || s.groups > kSumGroups);
    cudaError_t e = cudaSuccess;
    if (own) {
        const int64_t want = ceil_div(static_cast<int64_t>(s.groups) * s.N, 256);
        const int64_t most = static_cast<int64_t>(sms) * 8;
        e = launch_sum(dgate_kernel, dim3(static_cast<unsigned>(want < most ? want : most), 1, 1), 256, s,
                       stream);
        if (e != cudaSuccess) return e;
    }
    const bool totals = s.d_pre_weight || s.d_pre_bias || s.d_post_weight || s.d_post_bias;
    if (own && !totals) return e;
    if (two) {
        SumParams f = s;
        f.lines = lines;
        e = launch_sum(sum_kernel, dim3(cols, kSumSplits, 1), 32 * kSumY, f, stream);
        if (e != cudaSuccess) return e;
        s.partials = lines;
        s.part_stride = static_cast<int64_t>(kSumSplits) * s.N;
        s.chunks = kSumSplits;
        s.gated = 0;
        s.d_gate = nullptr;
    }
    const unsigned groups = s.d_gate && !own ? static_cast<unsigned>(s.groups) : 0u;
    return launch_sum(sum_kernel, dim3(cols, 1 + groups, 1), 32 * kSumY, s, stream);
}

}  // namespace

extern "C" {

gemm_status_t norm_block_forward(int64_t M, int64_t N, const void* X, int64_t ldx,
                                 const void* Z, int64_t ldz, void* XO, int64_t ldxo,
                                 void* Y, int64_t ldy, int32_t x_dtype, int32_t z_dtype,
                                 const norm_block_t* block, gemm_stream_t stream) {
    gemm_status_t st = check_block(M, N, x_dtype, z_dtype, block);
    if (st == GEMM_ERR_INVALID_VALUE) return st;
    const bool some = M > 0 && N > 0;         // of nothing, the pointers are not looked at
    if (some && ((Z == nullptr) != (XO == nullptr) || (Z == nullptr && Y == nullptr)))
        return GEMM_ERR_INVALID_VALUE;
    if (some &&
        (!matrix_ok(X, ldx, N, x_dtype) || (Z && !matrix_ok(Z, ldz, N, z_dtype)) ||
         (XO && !matrix_ok(XO, ldxo, N, x_dtype)) || (Y && !matrix_ok(Y, ldy, N, z_dtype))))
        return GEMM_ERR_INVALID_VALUE;
    if (st != GEMM_OK) return st;
    if (M == 0 || N == 0) return GEMM_OK;
    const int sms = device_sms();
    if (sms < 0) return GEMM_ERR_LAUNCH;
    if (sms == 0) return GEMM_ERR_NOT_SUPPORTED;

    Launch l;
    std::memset(&l, 0, sizeof l);
    Params& p = l.p;
    fill_block(p, M, N, block);
    p.X = X;
    p.ldx = ldx;
    p.Z = Z;
    p.ldz = ldz;
    p.XO = XO;
    p.ldxo = ldxo;
    p.Y = Y;
    p.ldy = ldy;
    p.vec = N % 8 == 0 && vector16(X, ldx, x_dtype) && vector16(Z, ldz, z_dtype) &&
            vector16(XO, ldxo, x_dtype) && vector16(Y, ldy, z_dtype);
    p.token_gate = Z && block->gate && block->gate_rows == 1 ? 1 : 0;
    p.i_ws = p.i_bs = p.i_wpre = p.i_bpre = -1;
    if (Z) p.i_ws = p.n_par++;
    if (Z && block->post_bias) p.i_bs = p.n_par++;
    if (Y) p.i_wpre = p.n_par++;
    if (Y && block->pre_bias) p.i_bpre = p.n_par++;
    // 16 elements per thread, which halves what a row costs beside its
    // elements; 8 where rows are few (one row's latency counts) or narrow, and
    // for rows that are not vectors, whose addresses take registers: FP32 ones
    // (32800 x 1023, RMSNorm on both sides, 117 us by 16, 93 by 8) and 16-bit
    // ones but where the post-norm has a mean to take first or rows are long
    // (8194 x 4095 bf16 100 and 86, LayerNorm on both sides 124 and 140; 4096 x
    // 8191 108 and 117)
    const bool loose8 = !p.vec && (x_dtype == GEMM_F32 || (N <= 4096 && !(Z && block->post == kLayer)));
    l.chunks8 = N > kMaxColumnsPerCta ? 2 : (M <= sms || N <= 256 || loose8) ? 1 : 2;
    p.cluster = N > kMaxColumnsPerCta ? 2 : 1;
    p.T = threads_for(ceil_div(round_up(N, 16 * p.cluster), p.cluster), l.chunks8);
    p.slot_bytes = static_cast<uint32_t>(l.chunks8 * 8 * p.T * (esize(x_dtype) + (Z ? esize(z_dtype) : 0)));
    int groups = 1;
    // 64 registers per thread
    const int ctas = choose_cta(p, kForwardSums, l.chunks8, 1024, 1024, 32, groups);
    if (ctas == 0) return GEMM_ERR_NOT_SUPPORTED;
    const Chunks ch = chunks_for(M, N, Z && block->gate ? block->gate_rows : 1,
                                 static_cast<int64_t>(sms) * ctas / p.cluster);
    set_chunks(p, ch);
    // no more groups than a chunk has rows
    while (groups > 1 && groups / 2 >= ch.rows) groups /= 2;
    l.threads = groups * p.T;
    l.grid = static_cast<int>(ch.groups * ch.per_group * p.cluster);
    l.smem = static_cast<size_t>(smem_for(p, kForwardSums, l.chunks8, groups, p.stages));
    l.stream = reinterpret_cast<cudaStream_t>(stream);
    return status_of(run_forward(x_dtype, z_dtype, l));
}

int64_t norm_block_backward_workspace(int64_t M, int64_t N, int64_t gate_rows, int32_t num_sms) {
    if (M < 0 || N < 0 || M > INT32_MAX || N > INT32_MAX || gate_rows < 1 || num_sms < 0) return -1;
    if (num_sms == 0) {
        num_sms = device_sms();
        if (num_sms <= 0) return -1;
    }
    const Chunks c = back_chunks(M, N, gate_rows, num_sms);
    return 4 * (c.groups * c.per_group + kSumSplits) * N * 4;
}

gemm_status_t norm_block_backward(int64_t M, int64_t N, const void* XO, int64_t ldxo,
                                  const void* Z, int64_t ldz, const void* dY, int64_t lddy,
                                  const void* dXO, int64_t lddxo, void* dX, int64_t lddx,
                                  void* dZ, int64_t lddz, int32_t x_dtype, int32_t z_dtype,
                                  const norm_block_t* block, const norm_block_grads_t* grads,
                                  void* workspace, int64_t workspace_bytes,
                                  gemm_stream_t stream) {
    gemm_status_t st = check_block(M, N, x_dtype, z_dtype, block);
    if (st == GEMM_ERR_INVALID_VALUE) return st;
    norm_block_grads_t none;
    std::memset(&none, 0, sizeof none);
    const norm_block_grads_t& gr = grads ? *grads : none;
    void* const outs[] = {gr.d_pre_weight, gr.d_pre_bias, gr.d_post_weight, gr.d_post_bias, gr.d_gate};
    bool sums = false;
    for (void* o : outs) {
        if (o == nullptr) continue;
        sums = true;
        if (!dtype_ok(gr.grad_dtype) || !aligned(o, esize(gr.grad_dtype))) return GEMM_ERR_INVALID_VALUE;
    }
    const bool some = M > 0 && N > 0;         // of nothing, the pointers are not looked at
    if (some && Z == nullptr && (dZ || gr.d_post_weight || gr.d_post_bias || gr.d_gate))
        return GEMM_ERR_INVALID_VALUE;
    if (some && gr.d_gate && block->gate == nullptr) return GEMM_ERR_INVALID_VALUE;
    if (some) {
        if (!matrix_ok(XO, ldxo, N, x_dtype) || (Z && !matrix_ok(Z, ldz, N, z_dtype)) ||
            (dY && !matrix_ok(dY, lddy, N, z_dtype)) || (dXO && !matrix_ok(dXO, lddxo, N, x_dtype)) ||
            (dX && !matrix_ok(dX, lddx, N, x_dtype)) || (dZ && !matrix_ok(dZ, lddz, N, z_dtype)))
            return GEMM_ERR_INVALID_VALUE;
        if (sums && (workspace == nullptr || !aligned(workspace, 16))) return GEMM_ERR_INVALID_VALUE;
    }
    if (st != GEMM_OK) return st;
    if (N == 0) return GEMM_OK;
    const int sms = device_sms();
    if (sms < 0) return GEMM_ERR_LAUNCH;
    if (sms == 0) return GEMM_ERR_NOT_SUPPORTED;
    const bool token = block->gate != nullptr && block->gate_rows == 1;
    const Chunks ch = back_chunks(M, N, block->gate ? block->gate_rows : 1, sms);
    const int64_t chunks = M > 0 ? ch.groups * ch.per_group : 0;
    if (M > 0 && sums && workspace_bytes < 4 * (chunks + kSumSplits) * N * 4) return GEMM_ERR_INVALID_VALUE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

    Launch l;
    std::memset(&l, 0, sizeof l);
    Params& p = l.p;
    fill_block(p, M, N, block);
    p.X = XO;
    p.ldx = ldxo;
    p.Z = Z;
    p.ldz = ldz;
    p.dY = dY;
    p.lddy = lddy;
    p.dXO = dXO;
    p.lddxo = lddxo;
    p.dX = dX;
    p.lddx = lddx;
    p.dZ = dZ;
    p.lddz = lddz;
    p.vec = N % 8 == 0 && vector16(XO, ldxo, x_dtype) && vector16(Z, ldz, z_dtype) &&
            vector16(dY, lddy, z_dtype) && vector16(dXO, lddxo, x_dtype) &&
            vector16(dX, lddx, x_dtype) && vector16(dZ, lddz, z_dtype) &&
            (!token || vector16(gr.d_gate, N, gr.grad_dtype));
    p.token_gate = token ? 1 : 0;
    set_chunks(p, ch);
    p.i_ws = p.i_bs = p.i_wpre = p.i_bpre = -1;
    if (Z) p.i_ws = p.n_par++;
    if (dY) p.i_wpre = p.n_par++;
    if (token && gr.d_gate && block->post_bias) p.i_bs = p.n_par++;
    p.partials = sums ? static_cast<float*>(workspace) : nullptr;
    p.part_stride = chunks * N;
    p.dgate = token ? gr.d_gate : nullptr;
    p.grad_dtype = gr.grad_dtype;
    l.bias = gr.d_pre_bias || gr.d_post_bias || (!token && gr.d_gate && block->post_bias);
    if (M > 0) {
        // 8192 columns fill a CTA's registers: wider rows take a pair of CTAs
        // (rows that are not vectors: 16 per thread spill, 32800 x 1023 FP32 231 us against 171)
        l.chunks8 = N > (p.vec ? 256 : 4096) ? 2 : 1;
        p.cluster = N > kMaxColumnsPerCta ? 2 : 1;
        p.T = threads_for(ceil_div(round_up(N, 16 * p.cluster), p.cluster), l.chunks8);
        p.slot_bytes = static_cast<uint32_t>(
            l.chunks8 * 8 * p.T *
            (esize(x_dtype) * (dXO ? 2 : 1) + (Z ? esize(z_dtype) : 0) + (dY ? esize(z_dtype) : 0)));
        int groups = 1;
        if (choose_cta(p, kBackwardSums, l.chunks8, kBackThreads, kBackThreads, 1, groups) == 0) return GEMM_ERR_NOT_SUPPORTED;
        while (groups > 1 && groups / 2 >= ch.rows) groups /= 2;
        l.threads = groups * p.T;
        l.smem = static_cast<size_t>(smem_for(p, kBackwardSums, l.chunks8, groups, p.stages));
        // the groups' column sums pass through the ring's memory
        const size_t line = static_cast<size_t>(smem_for(p, kBackwardSums, l.chunks8, groups, 0)) +
                            static_cast<size_t>(p.T) * l.chunks8 * 32;
        if (l.smem < line) l.smem = line;
        if (l.smem > static_cast<size_t>(kSmemPerCta)) return GEMM_ERR_NOT_SUPPORTED;
        l.grid = static_cast<int>(chunks * p.cluster);
        l.stream = s;
        st = status_of(run_backward(x_dtype, z_dtype, l));
        if (st != GEMM_OK) return st;
    }
    if (!sums) return GEMM_OK;
    if (gr.d_gate && token && !(gr.d_pre_weight || gr.d_pre_bias || gr.d_post_weight || gr.d_post_bias))
        return GEMM_OK;                                   // written row by row
    SumParams sp;
    std::memset(&sp, 0, sizeof sp);
    sp.partials = p.partials;
    sp.part_stride = p.part_stride;
    sp.N = static_cast<int32_t>(N);
    sp.groups = static_cast<int32_t>(M > 0 ? ch.groups : 1);
    sp.chunks_per_group = M > 0 ? p.chunks_per_group : 0;
    sp.chunks = sp.groups * sp.chunks_per_group;
    sp.gated = token || M == 0 ? 0 : 1;    // (no rows: the gate has none either)
    sp.token_gate = p.token_gate;
    sp.bias = l.bias ? 1 : 0;
    sp.wpost = p.wpost;
    sp.bpost = p.bpost;
    sp.gate = M > 0 ? p.gate : nullptr;
    sp.ld_gate = p.ld_gate;
    sp.vec_dtype = p.vec_dtype;
    sp.grad_dtype = gr.grad_dtype;
    sp.scale = p.scale;
    sp.d_pre_weight = gr.d_pre_weight;
    sp.d_pre_bias = gr.d_pre_bias;
    sp.d_post_weight = gr.d_post_weight;
    sp.d_post_bias = gr.d_post_bias;
    sp.d_gate = (token || M == 0) ? nullptr : gr.d_gate;
    return status_of(run_sum(sp, p.partials ? p.partials + 4 * p.part_stride : nullptr, sms, s));
}

}  // extern "C"
