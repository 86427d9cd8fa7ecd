// ortho.cu -- the orthogonalised update (include/ortho_sm103.h): the norm, the
// scaled copy, and the schedule of the products (ortho_kern.cuh).
#include <cmath>
#include <cstring>
#include <mutex>

#include "device_limits.h"
#include "f32x2.cuh"
#include "ortho_kern.cuh"
#include "ortho_launch.h"

namespace gemm103 {
namespace {

constexpr int kPrepThreads = 256;
constexpr int kMostParts = 512;              // partial sums of a matrix, at most

struct PrepParams {
    const void* G;
    int64_t ldg, stride_g;
    int32_t rows, cols, parts;               // as stored; CTAs that sum each matrix
    int32_t vec;                             // G's rows are 16-byte vectors
    int32_t xr, xc;                          // padded sides
    double* sums;                            // [batch][parts]
    int32_t* done;                           // [products][batch], zeroed for the products' kernel
    int32_t products;
    float eps;
    __half *hi, *down;                       // down: lo's second bytes, 8 in the place of 8 halves, or NULL
    uint8_t* lo;
};

// Eight elements of a row as FP32, zeros behind its end.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int32_t col, int32_t cols, bool vec, float (&f)[8]) {
    constexpr int kPer = 16 / sizeof(T);
    if (vec && col + 8 <= cols) {
        #pragma unroll
        for (int q = 0; q < 8 / kPer; ++q) {
            const uint4 u = *reinterpret_cast<const uint4*>(row + col + q * kPer);
            const T* e = reinterpret_cast<const T*>(&u);
            #pragma unroll
            for (int i = 0; i < kPer; ++i) f[q * kPer + i] = to_f<T>(e[i]);
        }
    } else {
        #pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = col + i < cols ? to_f<T>(row[col + i]) : 0.0f;
    }
}

// Sum over the CTA in a fixed order; every thread gets it.
__device__ __forceinline__ double cta_sum(double v, double* red) {
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
    #pragma unroll
    for (int w = 0; w < kPrepThreads / 32; ++w) t += red[w];
    return t;
}

constexpr int kPieces = 4;                   // of 8 elements, in flight per thread

// Partial sums of squares.  32 elements in FP32, kept where the sum lies in
// [2^-90, 2^127) (32 squares below 2^-126 are under 2^-31 of it), else again in
// FP64; FP64 from there on.  (One FP64 addition for 8 elements bound the pass: 59M
// elements 40 us.)
template <typename T>
__global__ void __launch_bounds__(kPrepThreads) ortho_norm_kernel(const PrepParams p) {
    __shared__ double red[kPrepThreads / 32];
    grid_dependency_wait();
    grid_dependents_launch();
    if (blockIdx.x == 0)
        for (int32_t i = threadIdx.x; i < p.products; i += kPrepThreads)
            p.done[static_cast<int64_t>(i) * gridDim.y + blockIdx.y] = 0;
    const T* g = static_cast<const T*>(p.G) + blockIdx.y * p.stride_g;
    const int32_t per_row = (p.cols + 7) >> 3;
    const int64_t total = static_cast<int64_t>(p.rows) * per_row;
    double acc = 0.0;
    const int64_t stride = static_cast<int64_t>(p.parts) * kPrepThreads;
    for (int64_t q0 = static_cast<int64_t>(blockIdx.x) * kPrepThreads + threadIdx.x; q0 < total; q0 += kPieces * stride) {
        float f[kPieces][8];
        #pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const int64_t q = q0 + k * stride;
            #pragma unroll
            for (int i = 0; i < 8; ++i) f[k][i] = 0.0f;
            if (q < total) {
                const uint32_t r = static_cast<uint32_t>(q) / static_cast<uint32_t>(per_row);
                const int32_t col = static_cast<int32_t>(static_cast<uint32_t>(q) - r * per_row) * 8;
                load8<T>(g + r * p.ldg, col, p.cols, p.vec, f[k]);
            }
        }
        float s = 0.0f, t = 0.0f;
        bool any = false;
        #pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            #pragma unroll
            for (int i = 0; i < 8; i += 2) s = fmaf(f[k][i], f[k][i], s), t = fmaf(f[k][i + 1], f[k][i + 1], t);
        }
        s += t;
        if (s >= 0x1p-90f && s < 0x1p127f) {
            acc += static_cast<double>(s);
            continue;
        }
        #pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            #pragma unroll
            for (int i = 0; i < 8; ++i) any = any || f[k][i] != 0.0f;            // (NaN is not 0)
        }
        if (!any) continue;
        #pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
                const double d = static_cast<double>(f[k][i]);
                acc = fma(d, d, acc);
            }
        }
    }
    const double s = cta_sum(acc, red);
    if (threadIdx.x == 0) p.sums[static_cast<int64_t>(blockIdx.y) * p.parts + blockIdx.x] = s;
}

// kScale / (norm + eps).
__device__ __forceinline__ double ortho_factor(const PrepParams& p, double* red) {
    double s = 0.0;
    for (int32_t i = threadIdx.x; i < p.parts; i += kPrepThreads)
        s += p.sums[static_cast<int64_t>(blockIdx.y) * p.parts + i];
    return static_cast<double>(kOrthoScale) / (sqrt(cta_sum(s, red)) + static_cast<double>(p.eps));
}

// x times the factor as x f g: the factor in FP32, or where that does not hold it
// the two halves of its exponent range.  (A product in FP64 for every element, even
// one that is not taken, made this pass 353 us for 59M elements, of 75.)
struct Factor {
    float f, g;
};
__device__ __forceinline__ Factor split_factor(double f) {
    Factor r;
    const bool fits = !(f >= 0x1p120) && !(f < 0x1p-120);       // (NaN and 0 go on as they are)
    if (fits || f == 0.0) {
        r.f = static_cast<float>(f), r.g = 1.0f;
    } else {
        const double h = f >= 1.0 ? 0x1p100 : 0x1p-100;
        r.f = static_cast<float>(f / h), r.g = static_cast<float>(h);
    }
    return r;
}
__device__ __forceinline__ float scaled(float x, const Factor& f) { return x * f.f * f.g; }

__device__ __forceinline__ void store_pair8(const PrepParams& p, int64_t at, const float (&x)[8]) {
    F2 v[4], y[4];
    #pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mk2(x[2 * i], x[2 * i + 1]);
    const uint4 h = pack8(v);
    half8(h, y);
    #pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fma2(y[i], mk2(-1.0f), v[i]);
    uint2 up, down;
    pack_low8(y, v, up, down);
    *reinterpret_cast<uint4*>(p.hi + at) = h;
    *reinterpret_cast<uint2*>(p.lo + at) = up;
    if (p.down != nullptr) *reinterpret_cast<uint2*>(p.down + at) = down;
}

// X = G times the factor, as hi + lo, padded with zeros.
template <typename T>
__global__ void __launch_bounds__(kPrepThreads) ortho_scale_kernel(const PrepParams p) {
    __shared__ double red[kPrepThreads / 32];
    grid_dependency_wait();
    grid_dependents_launch();
    const Factor f = split_factor(ortho_factor(p, red));
    const T* g = static_cast<const T*>(p.G) + blockIdx.y * p.stride_g;
    const int64_t base = static_cast<int64_t>(blockIdx.y) * p.xr * p.xc;
    const uint32_t per_row = static_cast<uint32_t>(p.xc) >> 3;
    const int64_t total = static_cast<int64_t>(p.xr) * per_row;
    for (int64_t q = static_cast<int64_t>(blockIdx.x) * kPrepThreads + threadIdx.x; q < total;
         q += static_cast<int64_t>(gridDim.x) * kPrepThreads) {
        const int32_t r = static_cast<int32_t>(static_cast<uint32_t>(q) / per_row);
        const int32_t col = static_cast<int32_t>(static_cast<uint32_t>(q) - r * per_row) * 8;
        float x[8];
        #pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.0f;
        if (r < p.rows && col < p.cols) {
            load8<T>(g + r * p.ldg, col, p.cols, p.vec, x);
            #pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = scaled(x[i], f);
            // behind the row's end a factor that is not finite must not reach the padding
            #pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + i >= p.cols) x[i] = 0.0f;
        }
        store_pair8(p, base + q * 8, x);
    }
}

int64_t pad64(int64_t v) { return (v + 63) & ~static_cast<int64_t>(63); }
int64_t up256(int64_t v) { return (v + 255) & ~static_cast<int64_t>(255); }

// Where things lie in the workspace, in bytes.
struct Layout {
    int64_t np, xr, xc;
    int64_t hi[2], lo, a, b, diag_a, diag, sums, done, bytes;
};
Layout layout(int64_t batch, int64_t rows, int64_t cols) {
    Layout l;
    l.xr = pad64(rows);
    l.xc = pad64(cols);
    l.np = rows < cols ? l.xr : l.xc;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += up256(bytes);
        return here;
    };
    const int64_t x = batch * l.xr * l.xc * 2, s = batch * l.np * l.np * 2;
    l.hi[0] = take(x);
    l.hi[1] = take(x);
    l.lo = take(x / 2);
    l.a = take(s);
    l.b = take(s);
    l.diag_a = take(batch * l.np * 4);
    l.diag = take(batch * l.np * 4);
    l.sums = take(batch * kMostParts * 8);
    l.done = take(batch * 3 * ORTHO_MAX_STEPS * 4);
    l.bytes = at;
    return l;
}

// batch matrices of `rows` x `cols` halves, cols a multiple of 64, one behind the
// other: (64 elements, row, chunk, matrix), boxes of box_rows rows by box_chunks chunks.
bool encode_map(const OrthoCall& c, CUtensorMap* map, const void* ptr, int64_t rows, int64_t cols,
                uint32_t box_rows = 128, uint32_t box_chunks = 2) {
    const cuuint64_t dims[4] = {64u, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(cols / 64),
                                static_cast<cuuint64_t>(c.batch)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(cols * 2), 128u, static_cast<cuuint64_t>(rows * cols * 2)};
    const cuuint32_t box[4] = {64u, box_rows, box_chunks, 1u};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return c.encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaLaunchConfig_t config(dim3 grid, int threads, size_t smem, cudaStream_t stream, cudaLaunchAttribute* attr,
                          int cluster) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cfg;
}

struct Maps {
    CUtensorMap x[2], a, b;              // boxes of 128 rows by two chunks
    CUtensorMap x_few[2], a_few, b_few;  // narrow tiles' K-major B: of as many rows as columns
    CUtensorMap x_narrow[2];             // narrow tiles' MN-major B: of one chunk
};

// Products [p.first, p.last) on CTA pairs.  More than one: a cooperative launch.
template <bool FINE>
cudaError_t launch_pair(const OrthoCall& c, const Maps& m, const OrthoParams& p) {
    auto kern = ortho_pair_kernel<FINE>;
    static DeviceLimits limit;
    cudaError_t e = limit.raise(kOrthoPairSmem, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kOrthoPairSmem));
    });
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    const bool chain = p.last - p.first > 1;
    int64_t pairs = static_cast<int64_t>(p.batch) * (p.tiles_step > p.tiles_sym ? p.tiles_step : p.tiles_sym);
    if (pairs > c.sms / 2) pairs = c.sms / 2;
    cudaLaunchConfig_t cfg = config(dim3(static_cast<unsigned>(2 * pairs), 1, 1), kOrthoPairThreads, kOrthoPairSmem,
                                    c.stream, attr, 2);
    // no more pairs than can be resident at once: they take the tiles in turns
    static std::mutex mu;
    static PerDevice<int> known;
    int most = 0;
    {
        std::lock_guard<std::mutex> g(mu);
        int* k = known.current();
        if (k != nullptr) most = *k;
        if (most == 0) {
            cudaLaunchConfig_t q = cfg;
            q.gridDim = dim3(static_cast<unsigned>(c.sms / 2 * 2), 1, 1);
            q.attrs = &attr[1];
            q.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&most, kern, &q);
            if (e != cudaSuccess) return e;
            if (most < 1) return cudaErrorInvalidConfiguration;
            if (k != nullptr) *k = most;
        }
    }
    if (pairs > most) cfg.gridDim = dim3(static_cast<unsigned>(2 * most), 1, 1);
    if (chain) {
        attr[0].id = cudaLaunchAttributeCooperative;
        attr[0].val.cooperative = 1;
    }
    return cudaLaunchKernelEx(&cfg, kern, m.x[0], m.x[1], m.a, m.b, p);
}

template <int MODE, int NB>
cudaError_t launch_tile(const OrthoCall& c, const CUtensorMap& a, const CUtensorMap& b, const OrthoParams& p) {
    auto kern = ortho_tile_kernel<MODE, NB>;
    static DeviceLimits limit;
    const cudaError_t e = limit.raise(kOrthoTileSmem, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kOrthoTileSmem));
    });
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config(dim3(static_cast<unsigned>(p.batch * (MODE < kStep ? p.tiles_sym : p.tiles_step) * p.splits), 1, 1), kOrthoTileThreads,
                                    kOrthoTileSmem, c.stream, attr, p.splits);
    return cudaLaunchKernelEx(&cfg, kern, a, b, p);
}

struct Schedule {
    bool pair;
    int32_t width;                           // columns of a tile
    int32_t tiles, tiles_i, splits;
};

// The faster schedule by a rough count of SM cycles.  A pair's 256 x 256 x 128 block
// takes 1024 at the tensor core's rate, a tile's epilogue 9000 beside the next
// tile's blocks.  A single CTA's 128 x 128 x 128 block takes as long, for it is bound
// by the 64 KB that it loads (64 a cycle); its epilogue 4500 and the exchange of a
// split 7500, both as the columns, and 3000 until the first block is there.  K is split
// up to `most_splits` (the first product alone: of the others, on 64 to 65536 rows and
// columns, this count never finds a split faster).
Schedule schedule(const OrthoCall& c, bool symmetric, int32_t least_width, int32_t most_splits, int64_t rows, int64_t cols,
                  int64_t k_blocks) {
    Schedule best = {};
    int64_t least = INT64_MAX;
    auto consider = [&](bool pair, int32_t width, int32_t splits) {
        const int64_t side = pair ? 256 : 128;
        const int64_t i = (rows + side - 1) / side, j = (cols + width - 1) / width;
        const int64_t tiles = symmetric && width == side ? i * (i + 1) / 2 : i * j;
        int64_t cycles;
        if (pair) {
            const int64_t blocks = k_blocks * 1024, pairs = c.sms / 2;
            cycles = (tiles * c.batch + pairs - 1) / pairs * (blocks > 9000 ? blocks : 9000) + 9000;
        } else {
            const int64_t block = (32768 + width * 256) / 64, waves = (tiles * c.batch * splits + c.sms - 1) / c.sms;
            cycles = waves * ((k_blocks + splits - 1) / splits * block + 3000 + 4500 * width / 128 +
                              (splits > 1 ? 2500 + 5000 * width / 128 : 0));
        }
        if (cycles < least) {
            least = cycles;
            best = Schedule{pair, width, static_cast<int32_t>(tiles), static_cast<int32_t>(i), splits};
        }
    };
    consider(true, 256, 1);
    for (int32_t width = 128; width >= least_width; width /= 2)
        for (int32_t n = 1; n <= most_splits && n <= k_blocks && n * 8 <= width; n *= 2)       // (8 columns at least to finish)
            consider(false, width, n);
    return best;
}

template <int MODE>
cudaError_t product(const OrthoCall& c, const Schedule& s, const CUtensorMap& a, const CUtensorMap& b,
                    const CUtensorMap& b_narrow, OrthoParams p) {
    p.tiles_sym = p.tiles_step = s.tiles;
    p.tiles_i_step = s.tiles_i;
    p.full = s.width < 128;
    p.splits = s.splits;
    p.log_width = s.width == 128 ? 7 : s.width == 64 ? 6 : 5;
    for (int32_t n = s.splits; n > 1; n >>= 1) --p.log_width;               // (kGram)
    if (s.width == 128) return launch_tile<MODE, 128>(c, a, b, p);
    if constexpr (MODE < kStep)
        if (s.width == 32) return launch_tile<MODE, 32>(c, a, b_narrow, p);
    return launch_tile<MODE, 64>(c, a, b_narrow, p);
}

template <typename T>
cudaError_t prepare(const OrthoCall& c, PrepParams p) {
    cudaLaunchAttribute attr[2];
    const int64_t share = c.sms * 8 / c.batch > 1 ? c.sms * 8 / c.batch : 1;    // CTAs of a matrix
    const int64_t pieces = static_cast<int64_t>(p.rows) * ((p.cols + 7) / 8);
    int64_t parts = (pieces + 2 * kPrepThreads - 1) / (2 * kPrepThreads);
    if (parts > share) parts = share;
    if (parts > kMostParts) parts = kMostParts;
    p.parts = static_cast<int32_t>(parts);
    const unsigned batch = static_cast<unsigned>(c.batch);
    cudaLaunchConfig_t cfg = config(dim3(static_cast<unsigned>(parts), batch, 1), kPrepThreads, 0, c.stream, attr, 1);
    cudaError_t e = cudaLaunchKernelEx(&cfg, ortho_norm_kernel<T>, p);
    if (e != cudaSuccess) return e;
    int64_t grid = (static_cast<int64_t>(p.xr) * (p.xc / 8) + 2 * kPrepThreads - 1) / (2 * kPrepThreads);
    if (grid > share) grid = share;
    cfg.gridDim = dim3(static_cast<unsigned>(grid), batch, 1);
    return cudaLaunchKernelEx(&cfg, ortho_scale_kernel<T>, p);
}

// The first steps, in which lo has its second byte: those before which a rounding of X is
// enlarged by more than kFineFrom by the steps that are left, of singular values near 0 by
// their a.  Below that the first byte's 2^-20, of which half is the usual error, comes to at
// most 0.0007 of the norm of O (512; the usual five steps: 484).
constexpr float kFineFrom = 512.0f;
int32_t fine_steps(const ortho_update_t& opt) {
    int32_t s = opt.steps - 1;
    float grow = fmaxf(1.0f, fabsf(opt.coefficients[3 * s]));
    for (; s > 0; --s) {
        grow *= fmaxf(1.0f, fabsf(opt.coefficients[3 * (s - 1)]));
        if (grow > kFineFrom) break;
    }
    return s;                                // (0 of one step)
}

// The first of the last steps, behind each of which a rounding is enlarged by up to 4.
constexpr float kLateFrom = 4.0f;
int32_t late_step(const ortho_update_t& opt) {
    int32_t s = opt.steps - 1;
    for (float grow = 1.0f; s > 0; --s) {
        grow *= fmaxf(1.0f, fabsf(opt.coefficients[3 * s]));
        if (grow > kLateFrom) break;
    }
    return s;
}

cudaError_t run(const OrthoCall& c) {
    const Layout l = layout(c.batch, c.rows, c.cols);
    __half* hi[2] = {reinterpret_cast<__half*>(c.ws + l.hi[0]), reinterpret_cast<__half*>(c.ws + l.hi[1])};
    uint8_t* lo = c.ws + l.lo;
    __half* a = reinterpret_cast<__half*>(c.ws + l.a);
    __half* b = reinterpret_cast<__half*>(c.ws + l.b);
    const bool tall = c.rows > c.cols;
    const int64_t es = c.g_dtype == GEMM_F32 ? 4 : 2;
    auto vector = [&](const void* q, int64_t ld, int64_t stride, int64_t bytes) {
        return (reinterpret_cast<uintptr_t>(q) & 15u) == 0 && ld * bytes % 16 == 0 &&
               (c.batch == 1 || stride * bytes % 16 == 0);
    };

    PrepParams q = {};
    q.G = c.G, q.ldg = c.ldg, q.stride_g = c.stride_g;
    q.rows = static_cast<int32_t>(c.rows), q.cols = static_cast<int32_t>(c.cols);
    q.vec = vector(c.G, c.ldg, c.stride_g, es);
    q.xr = static_cast<int32_t>(l.xr), q.xc = static_cast<int32_t>(l.xc);
    q.sums = reinterpret_cast<double*>(c.ws + l.sums);
    q.eps = c.opt->eps;
    const int32_t fine = fine_steps(*c.opt);
    q.hi = hi[0], q.lo = lo, q.down = fine > 0 ? hi[1] : nullptr;
    q.done = reinterpret_cast<int32_t*>(c.ws + l.done), q.products = 3 * c.opt->steps;
    cudaError_t e = c.g_dtype == GEMM_F32    ? prepare<float>(c, q)
                    : c.g_dtype == GEMM_BF16 ? prepare<__nv_bfloat16>(c, q)
                                             : prepare<__half>(c, q);
    if (e != cudaSuccess) return e;

    Maps m;
    if (!encode_map(c, &m.x[0], hi[0], l.xr, l.xc) || !encode_map(c, &m.x[1], hi[1], l.xr, l.xc) ||
        !encode_map(c, &m.a, a, l.np, l.np) || !encode_map(c, &m.b, b, l.np, l.np))
        return cudaErrorInvalidValue;

    OrthoParams p = {};
    p.batch = static_cast<int32_t>(c.batch);
    p.np = static_cast<int32_t>(l.np), p.xr = q.xr, p.xc = q.xc;
    p.rows = q.rows, p.cols = q.cols;
    p.tall = tall;
    p.lo = lo;
    p.diag_a = reinterpret_cast<float*>(c.ws + l.diag_a);
    p.diag = reinterpret_cast<float*>(c.ws + l.diag);
    p.O = static_cast<__nv_bfloat16*>(c.O), p.ldo = c.ldo, p.stride_o = c.stride_o;
    p.vec = vector(c.O, c.ldo, c.stride_o, 2);
    p.scale = c.opt->scale;
    p.err = c.err, p.wait_limit_ns = c.wait_limit_ns;
    const int32_t steps = c.opt->steps;
    p.k_gram = static_cast<int32_t>(((tall ? l.xr : l.xc) + 127) / 128);
    p.k_other = static_cast<int32_t>((l.np + 127) / 128);
    // (an MN-major B comes in boxes of 64 columns)
    const Schedule sched[3] = {schedule(c, true, tall ? 64 : 32, 8, l.np, l.np, p.k_gram),
                               schedule(c, true, 32, 1, l.np, l.np, p.k_other),
                               schedule(c, false, 64, 1, l.xr, l.xc, p.k_other)};
    p.steps = steps, p.fine = fine, p.late = late_step(*c.opt);
    p.x[0] = hi[0], p.x[1] = hi[1], p.mat_a = a, p.mat_b = b, p.done = q.done;
    std::memcpy(p.abc, c.opt->coefficients, static_cast<size_t>(steps) * 3 * sizeof(float));
    bool ok = true;
    for (int i = 0; i < 2; ++i) {
        if (sched[0].width < 128 && !tall) ok = ok && encode_map(c, &m.x_few[i], hi[i], l.xr, l.xc, sched[0].width, 2);
        if (sched[tall ? 0 : 2].width < 128) ok = ok && encode_map(c, &m.x_narrow[i], hi[i], l.xr, l.xc, 128, 1);
    }
    if (sched[1].width < 128) ok = ok && encode_map(c, &m.a_few, a, l.np, l.np, sched[1].width, 2);
    if (sched[2].width < 128 && tall) ok = ok && encode_map(c, &m.b_few, b, l.np, l.np, sched[2].width, 2);
    if (!ok) return cudaErrorInvalidValue;
    auto square = [](int64_t side) { return (side + 255) / 256; };
    p.tiles_sym = static_cast<int32_t>(square(l.np) * (square(l.np) + 1) / 2);
    p.tiles_i_step = static_cast<int32_t>(square(l.xr));
    p.tiles_step = static_cast<int32_t>(square(l.xr) * square(l.xc));
    p.debug_flags = c.debug_flags;
    if (sched[0].pair && sched[1].pair && sched[2].pair) {
        p.first = 0, p.last = 3 * steps;
        return fine > 0 ? launch_pair<true>(c, m, p) : launch_pair<false>(c, m, p);
    }
    for (int32_t i = 0; i < 3 * steps; ++i) {
        const int32_t s = i / 3, k = i % 3;
        if (i > 0) p.debug_flags = 0;
        if (sched[k].pair) {
            p.first = i, p.last = i + 1;
            e = k == 2 && s < fine ? launch_pair<true>(c, m, p) : launch_pair<false>(c, m, p);
        } else {
            OrthoParams o = p;
            o.first = i, o.last = i + 1;
            const CUtensorMap &x = m.x[s & 1], &xn = m.x_narrow[s & 1];
            if (k == 0) e = product<kGram>(c, sched[k], x, x, tall ? xn : m.x_few[s & 1], o);
            else if (k == 1) e = product<kPoly>(c, sched[k], m.a, m.a, m.a_few, o);
            else if (s + 1 < steps && s < fine)
                e = tall ? product<kFine>(c, sched[k], x, m.b, m.b_few, o) : product<kFine>(c, sched[k], m.b, x, xn, o);
            else if (s + 1 < steps)
                e = tall ? product<kStep>(c, sched[k], x, m.b, m.b_few, o) : product<kStep>(c, sched[k], m.b, x, xn, o);
            else
                e = tall ? product<kLast>(c, sched[k], x, m.b, m.b_few, o) : product<kLast>(c, sched[k], m.b, x, xn, o);
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

int64_t ortho_bytes(int64_t batch, int64_t rows, int64_t cols) { return layout(batch, rows, cols).bytes; }

gemm_status_t ortho_enqueue(const OrthoCall& c) {
    if (run(c) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

}  // namespace gemm103
