// ortho_kern.cuh -- the products of the orthogonalised update
// (include/ortho_sm103.h) on tcgen05, with their epilogues.
//
// The workspace holds every matrix as it is stored (X, xr x xc), both sides padded with
// zeros to multiples of 64: products of zeros are zeros, so the padding keeps itself
// and only the last epilogue looks at the true sizes.  The short side, padded, is np.
// Everything is FP16 times a power of two, kScale = 2^11: entries of X are as small
// as 1 / sqrt(n m), near FP16's subnormals without it, and up to 32 is held.
//
// One step is three products (X wide; X tall):
//   kGram  A = X X^T;  X^T X        upper tiles only; each is stored twice, as it is
//   kPoly  B = b A + c A A          and mirrored
//   kStep  X = a X + B X;  X B      X = hi + lo; the product reads hi, from one of two
//   kFine  the same, finer          buffers to the other, lo stays in place
//   kLast  O = scale (...)
// lo, at most half a step of hi, is a byte: a 254th of a step of its own hi, so that X is
// rounded by 2^-20 (eight more operations per element than an E5M2 lo, 446 us for 423,
// which rounds X by 2^-14; FP16, 2^-22, would be half as much again of what kStep reads and
// writes beside its operands).  It matters because every step enlarges what a rounding left
// in the directions of small singular values by a (3.4): rank 1, five steps, 0.0007 of the
// norm of O (E5M2 0.007).  Where the steps that are left enlarge it by more than 512, kFine
// carries 8 more bits (eight steps of 16 x 1023 x 777: 892 us, 615 without, and 0.1 of the
// norm of O for 0.002).  These lie where nothing else is: before step 0 in the second buffer
// of hi (each thread reads its own before it writes hi there), from then on in O's rows, so
// kLast, which writes O, has none.
// A and B are stored without their diagonals D and d, which are kept in FP32: B = b A +
// c (A - D)^2 + c (D A + A D) - c D^2, and X' = a X + d hi + (B - d) hi.  d multiplies what
// the rest of B multiplies, for they may cancel (with d lo beside it O of rank 1 is off by
// 0.002 after five steps and 0.05 after eight), but where little more enlarges what does not,
// in the last two steps usually: there d is most of B if G is noise, of which O is off by
// 0.0007 for 0.0012 (all in FP16: 0.0026).
// Operands come as boxes of 128 rows by two K chunks (32 KB) through 4-D maps (64
// elements, rows, chunk, matrix).  The same box is 128 rows of a K-major operand, or
// 128 columns of one with K along its rows (MN-major): both in the tall kGram, the
// right one in the wide kStep.
//
// Two kernels.  ortho_pair_kernel: 256 x 256 tiles on CTA pairs, double-buffered
// accumulators, for many tiles; it runs through a range of products, of all the steps
// where all of them have many tiles.  A tile then waits for the tiles of its own
// matrix in the product before, which others have done: those of a batch follow one
// another without a gap (16 x 1023 x 777, 76 pairs: 38 rounds of tiles for 50, and one
// launch for 15).  ortho_tile_kernel: one tile of 128 rows and 128 columns per CTA, for few
// tiles; for fewer still 64 or 32 columns, which shortens the epilogue, and all tiles of
// the symmetric products, without mirroring.  Of kGram, whose K is the long side, the tile is
// a cluster's, whose 1 to 8 CTAs split K and add up through distributed shared memory; the
// others' K is the short side, short where tiles are few.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "f32x2.cuh"
#include "ortho_sm103.h"
#include "ptx.cuh"

namespace gemm103 {

enum : int { kGram = 0, kPoly = 1, kStep = 2, kLast = 3, kFine = 4 };

constexpr float kOrthoScale = 2048.0f;
constexpr float kLoParts = 254.0f;                   // lo's byte: parts of a step of hi
constexpr int kOrthoStages = 3;
constexpr uint32_t kOrthoBox = 32768;                // 128 rows x 128 bytes x 2 chunks
constexpr uint32_t kOrthoStage = 2 * kOrthoBox;      // A's and B's
constexpr uint32_t kOrthoTurn = 32768;                // pairs: 4 KB per epilogue warp behind the stages
constexpr uint32_t kOrthoTileSmem = kOrthoStages * kOrthoStage + 1024 + 256;
constexpr uint32_t kOrthoPairSmem = kOrthoTileSmem + kOrthoTurn;
constexpr int kOrthoPairThreads = 384;               // warp 0 TMA, 1 MMA, 4-11 epilogue
// Registers per thread of the pairs' kernel: 168 at the launch, then as the roles
// need them (128 x 40 + 256 x 232 of the launch's 384 x 168): with 168 the epilogues'
// inputs ahead spill to memory that no cache has room for beside the stages, 8000
// cycles a tile.
constexpr int kOrthoFewRegs = 40, kOrthoManyRegs = 232;
static_assert(128 * kOrthoFewRegs + 256 * kOrthoManyRegs <= 384 * 168, "the launch's registers");
constexpr int kOrthoTileThreads = 192;               // warp 0 TMA, 1 MMA, 2-5 epilogue

// Products [first, last): product 3 s of step s is kGram, 3 s + 1 kPoly, 3 s + 2 kFine in
// the first `fine` steps, then kStep, and kLast in the last step.  From step `late` on B's
// diagonal multiplies lo too.
struct OrthoParams {
    int32_t batch;                      // matrices
    int32_t np, xr, xc;                 // padded: the short side; X's rows and columns
    int32_t k_gram, k_other;            // pairs of K chunks
    int32_t steps, fine, late, first, last;
    int32_t tiles_sym, tiles_step, tiles_i_step;    // tiles of a matrix; along its rows
    int32_t full;                       // symmetric products: all tiles, not the upper ones
    int32_t splits, log_width;          // ortho_tile_kernel, kGram: CTAs per tile; log2(columns / splits)
    __half *x[2], *mat_a, *mat_b;       // X's first numbers before even and odd steps
    uint8_t* lo;
    float *diag_a, *diag;               // A's and B's diagonals
    __nv_bfloat16* O;                   // kLast
    int64_t ldo, stride_o;
    int32_t rows, cols, tall, vec;      // true sides; rows > cols; O's rows are vectors
    float scale;
    int32_t* done;                      // [product][matrix]: epilogue warps through with it
    int* err;
    uint64_t wait_limit_ns;
    uint32_t debug_flags;
    float abc[3 * ORTHO_MAX_STEPS];
};

struct OrthoTile {
    int32_t b, i, j;
};

// Work item -> matrix and tile.  Symmetric products: the upper tiles (i <= j), by
// columns.  Others: by columns, so that the tiles of a wave share few columns of X.
template <int MODE>
__device__ __forceinline__ OrthoTile ortho_tile(const OrthoParams& p, int32_t item) {
    const int32_t tiles = MODE < kStep ? p.tiles_sym : p.tiles_step;
    OrthoTile t;
    t.b = item / tiles;
    const int32_t k = item - t.b * tiles;
    if (MODE < kStep && !p.full) {
        int32_t j = static_cast<int32_t>((sqrtf(8.0f * static_cast<float>(k) + 1.0f) - 1.0f) * 0.5f);
        while (j * (j + 1) / 2 > k) --j;
        while ((j + 1) * (j + 2) / 2 <= k) ++j;
        t.j = j;
        t.i = k - j * (j + 1) / 2;
    } else {
        t.j = k / p.tiles_i_step;
        t.i = k - t.j * p.tiles_i_step;
    }
    return t;
}

// Eight FP16 numbers as four FP32 pairs, and back, rounded.
__device__ __forceinline__ void half8(uint4 u, F2 (&f)[4]) {
    f[0] = unpack2<__half>(u.x), f[1] = unpack2<__half>(u.y), f[2] = unpack2<__half>(u.z), f[3] = unpack2<__half>(u.w);
}
__device__ __forceinline__ uint4 pack8(const F2 (&f)[4]) {
    return make_uint4(pack2<__half>(f[0]), pack2<__half>(f[1]), pack2<__half>(f[2]), pack2<__half>(f[3]));
}

// The epilogue works on 8 columns of a row at a time, 8 rows by 32 columns a warp, four
// neighbouring lanes a row: eight lanes, which the load/store unit takes at once, touch
// two lines.  (With a row per lane, as the accumulator comes, or another order of the
// lanes, eight: 33 wavefronts an access for 8; 16 x 1023 x 777 631 us for 536.)  The
// sums take a turn through shared memory to get there.

// lo in units of a step of its hi: a byte of kLoParts to the step, 128 for 0; with a second
// byte of 256 parts to each of these, again 128 for 0.
//
// Times `scale`, the steps of eight FP16 numbers x, or one over them: 2^-10 of the power of
// two below, at least FP16's smallest.
template <bool INVERSE>
__device__ __forceinline__ void low_unit(const F2 (&x)[4], float scale, F2 (&u)[4]) {
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        get2(x[i], lo, hi);
        lo = fmaxf(__uint_as_float(__float_as_uint(lo) & 0x7f800000u), 0x1p-14f);
        hi = fmaxf(__uint_as_float(__float_as_uint(hi) & 0x7f800000u), 0x1p-14f);
        if constexpr (INVERSE) {
            lo = __uint_as_float(0x7f000000u - __float_as_uint(lo));
            hi = __uint_as_float(0x7f000000u - __float_as_uint(hi));
        }
        u[i] = mul2(mk2(lo, hi), mk2(INVERSE ? scale * 0x1p10f : scale * 0x1p-10f));
    }
}
// Whole numbers of 0 .. 65535 become FP32 and back as the low bits of 2^23 + them.
constexpr uint32_t kWhole = 0x4b000000u;
__device__ __forceinline__ void low8(uint2 up, F2 (&f)[4]) {
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = i < 2 ? up.x : up.y;
        f[i] = add2(mk2(__uint_as_float(__byte_perm(w, kWhole, i & 1 ? 0x7442 : 0x7440)),
                        __uint_as_float(__byte_perm(w, kWhole, i & 1 ? 0x7443 : 0x7441))), mk2(-(0x1p23f + 128.0f)));
    }
}
__device__ __forceinline__ void low16(uint2 up, uint2 down, F2 (&f)[4]) {
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = __byte_perm(i < 2 ? down.x : down.y, i < 2 ? up.x : up.y, i & 1 ? 0x7362 : 0x5140);
        f[i] = add2(mk2(__uint_as_float(__byte_perm(w, kWhole, 0x7410)), __uint_as_float(__byte_perm(w, kWhole, 0x7432))),
                    mk2(-(0x1p23f + 32768.0f + 128.0f)));
    }
}
// lo as bytes; `up` alone is rounded to nearest as well.
__device__ __forceinline__ void pack_low8(const F2 (&x)[4], const F2 (&lo)[4], uint2& up, uint2& down) {
    F2 u[4];
    low_unit<true>(x, kLoParts * 256.0f, u);
    uint32_t w[4];
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        get2(fma2(lo[i], u[i], mk2(0x1p23f + 32768.0f + 128.0f)), a, b);
        w[i] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5140);          // down, down, up, up
    }
    up = make_uint2(__byte_perm(w[0], w[1], 0x7632), __byte_perm(w[2], w[3], 0x7632));
    down = make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
}

// What it reads: A (kPoly), or hi and lo, whose second byte only kFine has.
template <int MODE>
struct OrthoIn {
    uint4 x;
    uint2 y;
};
template <>
struct OrthoIn<kFine> {
    uint4 x;
    uint2 y, z;
};
// ... for 32 rows and 32 columns, with a row's and a column's part of the factors
// (ortho_factors) per lane.
template <int MODE>
struct OrthoBlock {
    OrthoIn<MODE> in[4];
    float row, col;
};
// The padded sides of a product's result: multiples of 64, so that whole blocks of 32
// lie in it or do not.
template <int MODE>
__device__ __forceinline__ int32_t ortho_rows(const OrthoParams& p) { return MODE < kStep ? p.np : p.xr; }
template <int MODE>
__device__ __forceinline__ int32_t ortho_cols(const OrthoParams& p) { return MODE < kStep ? p.np : p.xc; }
template <int MODE>
__device__ __forceinline__ bool ortho_inside(const OrthoParams& p, int32_t row, int32_t col) {
    return row < ortho_rows<MODE>(p) && col < ortho_cols<MODE>(p);
}
// lo's second bytes in 8 columns of a row before step s.  In O (s > 0) they lie at the
// row's first multiple of 8 bytes: of a row's 2 cols bytes that takes up to 6, and the last
// 8 up to 7 behind the last column, which from 16 columns on is never more than there
// are.  Rows of fewer columns: from the first byte on, one at a time.
__device__ __forceinline__ uint8_t* ortho_down(const OrthoParams& p, int32_t b, int32_t row, int32_t col) {
    uint8_t* at = reinterpret_cast<uint8_t*>(p.O + b * p.stride_o + row * p.ldo);
    if (p.cols >= 16) at += -reinterpret_cast<uintptr_t>(at) & 7;
    return at + col;
}
__device__ __forceinline__ uint2 ortho_read_down(const OrthoParams& p, int32_t s, int32_t b, int32_t row, int32_t col) {
    uint2 z = make_uint2(0x80808080u, 0x80808080u);
    if (row >= p.rows || col >= p.cols) return z;
    if (s == 0) return __ldcg(reinterpret_cast<const uint2*>(p.x[1] + (static_cast<int64_t>(b) * p.xr + row) * p.xc + col));
    const uint8_t* at = ortho_down(p, b, row, col);
    if (p.cols >= 16) return __ldcg(reinterpret_cast<const uint2*>(at));
    #pragma unroll 1
    for (int32_t i = 0; i < 8 && col + i < p.cols; ++i) {
        const uint32_t down = __ldcg(at + i), shift = (i & 3) * 8;
        uint32_t& w = i < 4 ? z.x : z.y;
        w = (w & ~(0xffu << shift)) | down << shift;
    }
    return z;
}
__device__ __forceinline__ void ortho_write_down(const OrthoParams& p, int32_t b, int32_t row, int32_t col, uint2 z) {
    if (row >= p.rows || col >= p.cols) return;
    uint8_t* at = ortho_down(p, b, row, col);
    if (p.cols >= 16) {
        *reinterpret_cast<uint2*>(at) = z;
    } else {
        #pragma unroll 1
        for (int32_t i = 0; i < 8 && col + i < p.cols; ++i)
            at[i] = static_cast<uint8_t>((i < 4 ? z.x : z.y) >> ((i & 3) * 8));
    }
}

template <int MODE>
__device__ __forceinline__ OrthoIn<MODE> ortho_read(const OrthoParams& p, int32_t s, int32_t b, int32_t row, int32_t col) {
    OrthoIn<MODE> in;
    in.x = make_uint4(0u, 0u, 0u, 0u);
    in.y = make_uint2(0u, 0u);
    if constexpr (MODE == kPoly) {
        in.x = __ldcg(reinterpret_cast<const uint4*>(p.mat_a + (static_cast<int64_t>(b) * p.np + row) * p.np + col));
    } else if constexpr (MODE != kGram) {
        const int64_t at = (static_cast<int64_t>(b) * p.xr + row) * p.xc + col;
        in.x = __ldcg(reinterpret_cast<const uint4*>(p.x[s & 1] + at));
        in.y = __ldcg(reinterpret_cast<const uint2*>(p.lo + at));
        if constexpr (MODE == kFine) in.z = ortho_read_down(p, s, b, row, col);
    }
    return in;
}

// An element of the diagonal, whose sum counts as 0 from here on (A's was read as 0).
template <int MODE>
__device__ __forceinline__ void ortho_diagonal(const OrthoParams& p, int32_t s, int32_t b, int32_t row, float sum) {
    const int64_t at = static_cast<int64_t>(b) * p.np + row;
    const float x = sum * (1.0f / (kOrthoScale * kOrthoScale));
    if constexpr (MODE == kGram) {
        p.diag_a[at] = x;
    } else {
        const float c = p.abc[3 * s + 2], d = __ldcg(p.diag_a + at);
        p.diag[at] = fmaf(d, fmaf(c, d, p.abc[3 * s + 1]), c * x);
    }
}

// Sums v (of scaled products) of 8 columns to the result, in v, and out to where it
// is stored by rows.
template <int MODE>
__device__ __forceinline__ void ortho_finish(const OrthoParams& p, int32_t s, int32_t b, int32_t row, int32_t col,
                                             const OrthoIn<MODE>& in, const F2 (&c0)[4], F2 (&v)[4]) {
    constexpr float kDown = 1.0f / kOrthoScale;
    F2 x[4];
    if constexpr (MODE < kStep) {
        if constexpr (MODE == kPoly) {
            half8(in.x, x);
            const F2 c2 = mk2(p.abc[3 * s + 2] * kDown);
            #pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = fma2(c0[i], x[i], mul2(c2, v[i]));
        } else {
            #pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], mk2(kDown));
        }
        __half* out = MODE == kGram ? p.mat_a : p.mat_b;
        *reinterpret_cast<uint4*>(out + (static_cast<int64_t>(b) * p.np + row) * p.np + col) = pack8(v);
    } else {
        F2 y[4], u[4];
        half8(in.x, x);
        if constexpr (MODE == kFine) low16(in.y, in.z, y);
        else low8(in.y, y);
        low_unit<false>(x, MODE == kFine ? 1.0f / (kLoParts * 256.0f) : 1.0f / kLoParts, u);
        // lo counts to hi, or apart from it: times a alone
        const bool late = MODE == kLast || s >= p.late;
        const F2 to_hi = mk2(late ? 1.0f : 0.0f), apart = mk2(late ? 0.0f : p.abc[3 * s]);
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[i] = mul2(u[i], y[i]);
            v[i] = mul2(v[i], mk2(kDown));
            if constexpr (MODE != kLast) v[i] = fma2(apart, y[i], v[i]);
            v[i] = fma2(c0[i], fma2(to_hi, y[i], x[i]), v[i]);
        }
        if constexpr (MODE != kLast) {
            const uint4 h = pack8(v);
            half8(h, x);
            #pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = fma2(x[i], mk2(-1.0f), v[i]);
            const int64_t at = (static_cast<int64_t>(b) * p.xr + row) * p.xc + col;
            *reinterpret_cast<uint4*>(p.x[(s & 1) ^ 1] + at) = h;
            uint2 up, down;
            pack_low8(x, y, up, down);
            *reinterpret_cast<uint2*>(p.lo + at) = up;
            if (MODE == kFine && s + 1 < p.fine) ortho_write_down(p, b, row, col, down);
        } else {
            const F2 scale = mk2(p.scale);
            #pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = mul2(mul2(v[i], mk2(kDown)), scale);
            if (p.vec && row < p.rows && col < p.cols) {
                __nv_bfloat16* d = p.O + b * p.stride_o + row * p.ldo + col;
                if (col + 8 <= p.cols) {
                    *reinterpret_cast<uint4*>(d) = make_uint4(pack2<__nv_bfloat16>(v[0]), pack2<__nv_bfloat16>(v[1]),
                                                              pack2<__nv_bfloat16>(v[2]), pack2<__nv_bfloat16>(v[3]));
                } else {
                    #pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float lo, hi;
                        get2(v[i], lo, hi);
                        if (col + 2 * i < p.cols) d[2 * i] = __float2bfloat16_rn(lo);
                        if (col + 2 * i + 1 < p.cols) d[2 * i + 1] = __float2bfloat16_rn(hi);
                    }
                }
            }
        }
    }
}
// Eight sums as two float4s of shared memory.
__device__ __forceinline__ void ortho_load8(const float4* a, const float4* b, F2 (&v)[4]) {
    const float4 x = *a, y = *b;
    v[0] = mk2(x.x, x.y), v[1] = mk2(x.z, x.w), v[2] = mk2(y.x, y.y), v[3] = mk2(y.z, y.w);
}
__device__ __forceinline__ void ortho_store8(float4* a, float4* b, const F2 (&v)[4]) {
    float4 x, y;
    get2(v[0], x.x, x.y), get2(v[1], x.z, x.w), get2(v[2], y.x, y.y), get2(v[3], y.z, y.w);
    *a = x, *b = y;
}

// Whether the results are stored in another way too, mirrored, or only in another,
// as rows that are not vectors.
template <int MODE>
__device__ __forceinline__ bool ortho_again(const OrthoParams& p, const OrthoTile& t) {
    if constexpr (MODE < kStep) return !p.full && t.i != t.j;
    else return MODE == kLast && !p.vec;
}
// Four columns of one row to the mirrored place (lanes: neighbouring rows).
template <int MODE>
__device__ __forceinline__ void ortho_mirror(const OrthoParams& p, int32_t b, int32_t row, int32_t col, float4 v) {
    __half* d = (MODE == kGram ? p.mat_a : p.mat_b) + (static_cast<int64_t>(b) * p.np + col) * p.np + row;
    d[0] = __float2half_rn(v.x);
    d[p.np] = __float2half_rn(v.y);
    d[2 * p.np] = __float2half_rn(v.z);
    d[3 * p.np] = __float2half_rn(v.w);
}

// A warp's 32 rows (the first is row0) and 32 columns: `r` one row per lane, from
// tensor memory; `in` four of eight rows.  `buf` is 4 KB of its own: row r's float4 u
// lies at u ^ (r & 7), which no access of 8 lanes meets twice in a bank.
template <int MODE>
__device__ __forceinline__ void ortho_block(const OrthoParams& p, int32_t s, const OrthoTile& t, int32_t row0, int32_t col0,
                                            const uint32_t (&r)[32], const OrthoBlock<MODE>& in, float4* buf) {
    const int lane = threadIdx.x & 31, l7 = lane & 7, g = lane & 3, line = lane >> 2;
    __syncwarp();
    #pragma unroll
    for (int u = 0; u < 8; ++u)
        buf[lane * 8 + (u ^ l7)] = make_float4(__uint_as_float(r[4 * u]), __uint_as_float(r[4 * u + 1]),
                                               __uint_as_float(r[4 * u + 2]), __uint_as_float(r[4 * u + 3]));
    __syncwarp();
    if constexpr (MODE < kStep) {
        if (row0 == col0) {
            float* e = reinterpret_cast<float*>(buf) + lane * 32 + (((lane >> 2) ^ l7) << 2) + (lane & 3);
            ortho_diagonal<MODE>(p, s, t.b, row0 + lane, *e);
            *e = 0.0f;
            __syncwarp();
        }
    }
    const bool again = ortho_again<MODE>(p, t);
    F2 col[4];
    if constexpr (MODE != kGram) {
        if (MODE == kPoly || p.tall) {
            #pragma unroll
            for (int i = 0; i < 4; ++i)
                col[i] = mk2(__shfl_sync(0xffffffffu, in.col, g * 8 + 2 * i),
                             __shfl_sync(0xffffffffu, in.col, g * 8 + 2 * i + 1));
        } else {
            col[0] = col[1] = col[2] = col[3] = mk2(0.0f);
        }
    }
    #pragma unroll
    for (int q = 0; q < 4; ++q) {
        float4* at = buf + (q * 8 + line) * 8;
        F2 v[4];
        ortho_load8(at + ((2 * g) ^ line), at + ((2 * g + 1) ^ line), v);
        F2 c0[4];
        if constexpr (MODE != kGram) {
            const F2 r = mk2(__shfl_sync(0xffffffffu, in.row, q * 8 + line));
            #pragma unroll
            for (int i = 0; i < 4; ++i) c0[i] = add2(r, col[i]);
        }
        ortho_finish<MODE>(p, s, t.b, row0 + q * 8 + line, col0 + g * 8, in.in[q], c0, v);
        if (again) ortho_store8(at + ((2 * g) ^ line), at + ((2 * g + 1) ^ line), v);
    }
    if (!again) return;
    __syncwarp();
    if constexpr (MODE == kLast) {
        // rows that are not vectors: a row at a time, one element per lane
        const float* f = reinterpret_cast<const float*>(buf);
        const int32_t col = col0 + lane;
        __nv_bfloat16* d = p.O + t.b * p.stride_o + col;
        #pragma unroll 4
        for (int k = 0; k < 32; ++k)
            if (row0 + k < p.rows && col < p.cols)
                d[(row0 + k) * p.ldo] = __float2bfloat16_rn(f[k * 32 + (((lane >> 2) ^ (k & 7)) << 2) + (lane & 3)]);
    } else {
        #pragma unroll 2
        for (int u = 0; u < 8; ++u) ortho_mirror<MODE>(p, t.b, row0 + lane, col0 + 4 * u, buf[lane * 8 + (u ^ l7)]);
    }
}

// The inputs of such a block.
template <int MODE>
__device__ __forceinline__ void ortho_read_block(const OrthoParams& p, int32_t s, int32_t b, int32_t row0, int32_t col0,
                                                 OrthoBlock<MODE>& in) {
    const int lane = threadIdx.x & 31;
    #pragma unroll
    for (int q = 0; q < 4; ++q) in.in[q] = ortho_read<MODE>(p, s, b, row0 + q * 8 + (lane >> 2), col0 + (lane & 3) * 8);
    if constexpr (MODE == kPoly) {
        const float* d = p.diag_a + static_cast<int64_t>(b) * p.np + lane;
        const float c1 = p.abc[3 * s + 1], c2 = p.abc[3 * s + 2];
        in.row = fmaf(c2, __ldcg(d + row0), c1);
        in.col = c2 * __ldcg(d + col0);
    } else if constexpr (MODE >= kStep) {
        const float* d = p.diag + static_cast<int64_t>(b) * p.np + lane;
        in.row = p.abc[3 * s];
        in.col = 0.0f;
        if (p.tall) in.col = __ldcg(d + col0);
        else in.row += __ldcg(d + row0);
    }
}

// A warp's 32 rows by up to 128 columns of a tile: `taddr` their accumulator; `in0`
// and `in1` the inputs of the first two blocks, on their way since before the sums
// were there.  Those of the next two follow when their registers are free (one at a
// time, handed on, cost the latency of a load per block: 5 us of 10 a tile).  A loop,
// and its body short: code that runs once per tile is bound by its fetching.
template <int MODE>
__device__ __forceinline__ void ortho_blocks(const OrthoParams& p, int32_t s, const OrthoTile& t, int32_t row0, int32_t col0,
                                             int32_t blocks, uint32_t taddr, OrthoBlock<MODE>& in0,
                                             OrthoBlock<MODE>& in1, float4* buf) {
    #pragma unroll 1
    for (int32_t c = 0; c < blocks; c += 2) {
        uint32_t r[32];
        __syncwarp();
        tmem_ld_32x32b_x32(taddr + c * 32, r);
        tmem_ld_wait();
        ortho_block<MODE>(p, s, t, row0, col0 + c * 32, r, in0, buf);
        if (c + 1 >= blocks) break;
        if (c + 2 < blocks) ortho_read_block<MODE>(p, s, t.b, row0, col0 + c * 32 + 64, in0);
        __syncwarp();
        tmem_ld_32x32b_x32(taddr + c * 32 + 32, r);
        tmem_ld_wait();
        ortho_block<MODE>(p, s, t, row0, col0 + c * 32 + 32, r, in1, buf);
        if (c + 3 < blocks) ortho_read_block<MODE>(p, s, t.b, row0, col0 + c * 32 + 96, in1);
    }
}
// Blocks of 32 columns from col0 on, of at most `most`.
template <int MODE>
__device__ __forceinline__ int32_t ortho_block_count(const OrthoParams& p, int32_t row0, int32_t col0, int32_t most) {
    const int32_t left = (ortho_cols<MODE>(p) - col0) >> 5;
    return row0 >= ortho_rows<MODE>(p) || left <= 0 ? 0 : left < most ? left : most;
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

// The MMAs of one stage (128 of K) into d: 256 x 256 on a pair, or 128 x NB.  AMN, BMN:
// the operand's K is along its rows.
template <bool AMN, bool BMN, bool PAIR, int NB>
__device__ __forceinline__ void ortho_mma(uint32_t d, uint32_t sa, bool first) {
    constexpr uint32_t idesc = instr_desc(0, AMN, BMN, PAIR ? 256 : 128, NB);
    constexpr uint32_t kRows = PAIR ? NB / 2 : NB;            // of B in this CTA's memory
    const uint32_t sb = sa + kOrthoBox;
    #pragma unroll
    for (uint32_t kk = 0; kk < 8; ++kk) {
        const uint64_t ad = AMN ? smem_desc_sw128(sa + kk * 2048u, 16384u, 1024u)
                                : smem_desc_sw128(sa + (kk >> 2) * 16384u + (kk & 3u) * 32u, 16u, 1024u);
        const uint64_t bd = BMN ? smem_desc_sw128(sb + kk * 2048u, 16384u, 1024u)
                                : smem_desc_sw128(sb + (kk >> 2) * (kRows * 128u) + (kk & 3u) * 32u, 16u, 1024u);
        const uint32_t acc = first && kk == 0 ? 0u : 1u;
        if constexpr (PAIR) tc_mma_f16_pair(d, ad, bd, idesc, acc);
        else tc_mma_f16(d, ad, bd, idesc, acc);
    }
}
// How a product reads its operands.
__device__ __forceinline__ bool ortho_a_mn(const OrthoParams& p, int mode) { return mode == kGram && p.tall; }
__device__ __forceinline__ bool ortho_b_mn(const OrthoParams& p, int mode) {
    return p.tall ? mode == kGram : mode >= kStep;
}

// ------------------------------------------------------------------- CTA pairs

// Product q: its mode, and its tiles of a matrix.
__device__ __forceinline__ int ortho_mode(const OrthoParams& p, int32_t q) {
    const int32_t s = q / 3, m = q - 3 * s;
    return m < 2 ? m : s + 1 == p.steps ? kLast : s < p.fine ? kFine : kStep;
}
__device__ __forceinline__ int32_t ortho_tiles(const OrthoParams& p, int mode) {
    return mode < kStep ? p.tiles_sym : p.tiles_step;
}
__device__ __forceinline__ OrthoTile ortho_tile_of(const OrthoParams& p, int mode, int32_t item) {
    return mode < kStep ? ortho_tile<kGram>(p, item) : ortho_tile<kStep>(p, item);
}
// This pair's first tile of a product: tiles are numbered through the products.
__device__ __forceinline__ int32_t ortho_first(int64_t before, int32_t mine, int32_t pairs) {
    const int32_t at = static_cast<int32_t>(before % pairs);
    return mine >= at ? mine - at : mine - at + pairs;
}

// Until the product before q is done for matrix b (bounded); one thread.  Tiles wait
// for earlier tiles only, every pair takes its own in order, and all pairs are
// resident (a cooperative launch), so some pair always can go on.
__device__ __forceinline__ bool ortho_ready(const OrthoParams& p, int32_t q, int32_t b, volatile int* abort_flag) {
    if (q == p.first) return true;
    const int32_t want = ortho_tiles(p, ortho_mode(p, q - 1)) * 16;                // 8 warps, 2 CTAs
    const int32_t* at = p.done + static_cast<int64_t>(q - 1) * p.batch + b;
    uint64_t t0 = 0;
    for (uint32_t i = 0;; ++i) {
        int32_t v;
        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(at) : "memory");
        if (v >= want) return true;
        __nanosleep(100);                // (1400 warps may be waiting at one address)
        if ((i & 63u) == 63u) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            if (*abort_flag || now - t0 > p.wait_limit_ns) break;
        }
    }
    ortho_give_up(p, abort_flag);
    return false;
}
// Between writes through the generic proxy and TMA's reads of them, on both sides.
__device__ __forceinline__ void ortho_proxy_fence() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

template <int MODE>
__device__ __forceinline__ bool ortho_epilogue(const OrthoParams& p, int32_t s, const OrthoTile& t, int32_t row0,
                                               int32_t col0, uint32_t taddr, uint64_t* acc_full, uint32_t parity,
                                               float4* turn, volatile int* abort_flag) {
    const int32_t blocks = ortho_block_count<MODE>(p, row0, col0, 4);
    // inputs are on their way before the accumulator is there
    OrthoBlock<MODE> in0, in1;
    if (blocks > 0) ortho_read_block<MODE>(p, s, t.b, row0, col0, in0);
    if (blocks > 1) ortho_read_block<MODE>(p, s, t.b, row0, col0 + 32, in1);
    // each lane waits for itself, and the warp goes on together or not at all: what follows
    // is collective
    if (!__all_sync(0xffffffffu, ortho_wait(acc_full, parity, abort_flag, p))) return false;
    tc_fence_after_sync();
    ortho_blocks<MODE>(p, s, t, row0, col0, blocks, taddr, in0, in1, turn);
    return true;
}

// FINE: some products are kFine.  (Their code in the same kernel costs all others their
// registers: 16 x 1023 x 777, five steps, 519 us for 439.)
template <bool FINE>
__global__ void __launch_bounds__(kOrthoPairThreads, 1)
    ortho_pair_kernel(const __grid_constant__ CUtensorMap map_x0, const __grid_constant__ CUtensorMap map_x1,
                      const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ OrthoParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOrthoStages * kOrthoStage + kOrthoTurn);
    uint64_t* empty = full + kOrthoStages;
    uint64_t* acc_full = empty + kOrthoStages;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    __shared__ volatile int abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int32_t pairs = static_cast<int32_t>(gridDim.x >> 1), mine = static_cast<int32_t>(blockIdx.x >> 1);

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

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOrthoFewRegs));
        if (warp == 0) {
            if (lane == 0) {
                const uint64_t keep = l2_policy_evict_last();
                uint32_t armed = 0;
                bool ok = true;
                int64_t before = 0;
                for (int32_t q = p.first; q < p.last && ok; ++q) {
                    const int mode = ortho_mode(p, q);
                    const CUtensorMap* x = (q / 3) & 1 ? &map_x1 : &map_x0;
                    const CUtensorMap* mb = mode == kPoly ? &map_a : x;
                    const CUtensorMap* ma = mode >= kStep ? &map_b : mb;
                    if (mode >= kStep && p.tall) ma = x, mb = &map_b;
                    const bool amn = ortho_a_mn(p, mode), bmn = ortho_b_mn(p, mode);
                    const int32_t items = p.batch * ortho_tiles(p, mode), k_blocks = mode == kGram ? p.k_gram : p.k_other;
                    const int32_t item0 = ortho_first(before, mine, pairs);
                    before += items;
                    for (int32_t item = item0; item < items && ok; item += pairs) {
                        const OrthoTile t = ortho_tile_of(p, mode, item);
                        const int32_t r0 = t.i * 256 + static_cast<int32_t>(rank) * 128;
                        const int32_t c0 = t.j * 256 + static_cast<int32_t>(rank) * 128;
                        if (q > p.first) {
                            ok = ortho_ready(p, q, t.b, &abort_flag);
                            if (!ok) break;
                            ortho_proxy_fence();
                        }
                        for (int32_t kb = 0; kb < k_blocks; ++kb, ++armed) {
                            const uint32_t s = armed % kOrthoStages, round = armed / kOrthoStages;
                            ok = ortho_wait(&empty[s], (round & 1u) ^ 1u, &abort_flag, p);
                            if (!ok) break;
                            uint8_t* sa = smem + s * kOrthoStage;
                            const uint32_t fb = map_to_rank(smem_addr(&full[s]), 0);
                            // the even CTA's barrier counts the bytes of both
                            if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kOrthoStage);
                            if ((p.debug_flags & 1u) && armed == 0 && blockIdx.x == 0) continue;   // test hook: no load
                            const int32_t k0 = kb * 128, kc = kb * 2;
                            tma_load_4d_pair(sa, ma, fb, 0, amn ? k0 : r0, amn ? r0 >> 6 : kc, t.b, keep);
                            tma_load_4d_pair(sa + kOrthoBox, mb, fb, 0, bmn ? k0 : c0, bmn ? c0 >> 6 : kc, t.b, keep);
                        }
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
                int64_t before = 0;
                for (int32_t q = p.first; q < p.last && ok; ++q) {
                    const int mode = ortho_mode(p, q);
                    const int32_t items = p.batch * ortho_tiles(p, mode), k_blocks = mode == kGram ? p.k_gram : p.k_other;
                    const bool amn = ortho_a_mn(p, mode), bmn = ortho_b_mn(p, mode);
                    const int32_t item0 = ortho_first(before, mine, pairs);
                    before += items;
                    for (int32_t item = item0; item < items && ok; item += pairs, ++acc_i) {
                        const uint32_t buf = acc_i & 1u;
                        ok = ortho_wait<true>(&acc_empty[buf], ((acc_i >> 1) & 1u) ^ 1u, &abort_flag, p);
                        if (!ok) break;
                        tc_fence_after_sync();
                        for (int32_t kb = 0; kb < k_blocks; ++kb, ++used) {
                            const uint32_t s = used % kOrthoStages, round = used / kOrthoStages;
                            ok = ortho_wait(&full[s], round & 1u, &abort_flag, p);
                            if (!ok) break;
                            tc_fence_after_sync();
                            const uint32_t d = tmem + buf * 256u, sa = base + s * kOrthoStage;
                            if (!bmn) ortho_mma<false, false, true, 256>(d, sa, kb == 0);
                            else if (!amn) ortho_mma<false, true, true, 256>(d, sa, kb == 0);
                            else ortho_mma<true, true, true, 256>(d, sa, kb == 0);
                            tc_commit_pair_multicast(&empty[s], 3);
                        }
                        if (ok) tc_commit_pair_multicast(&acc_full[buf], 3);
                    }
                }
                // all MMAs issued have completed, also when the loop was left early
                tc_commit_pair(drain);
                if (!mbar_wait(drain, 0, p.wait_limit_ns)) ortho_give_up(p, &abort_flag);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kOrthoManyRegs));
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        float4* turn = reinterpret_cast<float4*>(smem + kOrthoStages * kOrthoStage) + (warp - 4) * 256;
        uint32_t acc_i = 0;
        bool ok = true;
        int64_t before = 0;
        for (int32_t q = p.first; q < p.last && ok; ++q) {
            const int mode = ortho_mode(p, q);
            const int32_t items = p.batch * ortho_tiles(p, mode);
            const int32_t item0 = ortho_first(before, mine, pairs);
            before += items;
            for (int32_t item = item0; item < items; item += pairs, ++acc_i) {
                const OrthoTile t = ortho_tile_of(p, mode, item);
                const uint32_t buf = acc_i & 1u, parity = (acc_i >> 1) & 1u;
                const int32_t row0 = t.i * 256 + static_cast<int32_t>(rank) * 128 + quarter * 32;
                const int32_t col0 = t.j * 256 + half * 128;
                const uint32_t taddr = tmem + buf * 256u + (static_cast<uint32_t>(quarter * 32) << 16) + half * 128u;
                if (q > p.first) {
                    int ready = 0;
                    if (lane == 0) ready = ortho_ready(p, q, t.b, &abort_flag) ? 1 : 0;
                    ok = __shfl_sync(0xffffffffu, ready, 0) != 0;
                    if (!ok) break;
                    __syncwarp();        // all lanes read behind the acquire of one (a shuffle orders nothing)
                }
                if (mode == kGram)
                    ok = ortho_epilogue<kGram>(p, q / 3, t, row0, col0, taddr, &acc_full[buf], parity, turn,
                                               &abort_flag);
                else if (mode == kPoly)
                    ok = ortho_epilogue<kPoly>(p, q / 3, t, row0, col0, taddr, &acc_full[buf], parity, turn,
                                               &abort_flag);
                else if (mode == kStep)
                    ok = ortho_epilogue<kStep>(p, q / 3, t, row0, col0, taddr, &acc_full[buf], parity, turn,
                                               &abort_flag);
                else if (FINE && mode == kFine)
                    ok = ortho_epilogue<kFine>(p, q / 3, t, row0, col0, taddr, &acc_full[buf], parity, turn,
                                               &abort_flag);
                else
                    ok = ortho_epilogue<kLast>(p, q / 3, t, row0, col0, taddr, &acc_full[buf], parity, turn,
                                               &abort_flag);
                if (!ok) break;
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_addr(&acc_empty[buf]), 0));
                if (q + 1 < p.last) {
                    // what this warp wrote is there for the next product's loads (the
                    // release is cumulative: it covers what the warp's barrier ordered)
                    ortho_proxy_fence();
                    __syncwarp();
                    if (lane == 0)
                        asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(
                                         p.done + static_cast<int64_t>(q) * p.batch + t.b)
                                     : "memory");
                }
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();                                   // the peer is through with our memory
    tc_fence_after_sync();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ------------------------------------------------------- one tile per cluster

// kGram with K split: the sums of S CTAs, each of which finishes 128 rows and its part of
// the tile's columns, in units of 8 columns of a row.
template <int NB>
__device__ __forceinline__ void ortho_join(const OrthoParams& p, const OrthoTile& t, int32_t S, uint32_t rank, uint32_t taddr,
                                           uint8_t* smem, volatile int* abort_flag) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t log4 = p.log_width - 2, log8 = p.log_width - 3;            // log2 of the fours and eights of columns
    const int32_t first_row = t.i * 128, first_col = t.j * NB + (static_cast<int32_t>(rank) << p.log_width);
    float4* xbuf = reinterpret_cast<float4*>(smem);
    auto at_of = [&](int32_t src, int32_t c4, int32_t rr) {
        return xbuf + ((src << log4) + c4) * 128 + (rr ^ (((c4 >> 1) << (3 - log8)) & 7));
    };
    if (warp >= 2) {
        const int r_in = (warp & 3) * 32 + lane;
        #pragma unroll 1
        for (int c = 0; c < NB; c += 32) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(taddr + c, r);
            tmem_ld_wait();
            #pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const int32_t c4 = (c + j) >> 2;
                const uint32_t q = static_cast<uint32_t>(c4 >> log4);
                float4* at = at_of(static_cast<int32_t>(rank), c4 & ((1 << log4) - 1), r_in);
                const float4 v = make_float4(__uint_as_float(r[j]), __uint_as_float(r[j + 1]),
                                             __uint_as_float(r[j + 2]), __uint_as_float(r[j + 3]));
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
    if (*abort_flag) return;
    {
        const int32_t rr = static_cast<int32_t>(threadIdx.x), cc = first_row + rr - first_col;
        if (rr < 128 && cc >= 0 && cc < 1 << p.log_width && first_row + rr < p.np) {
            float sum = 0.0f;
            for (int32_t s = 0; s < S; ++s) {
                float* e = reinterpret_cast<float*>(at_of(s, cc >> 2, rr)) + (cc & 3);
                sum += *e;
                *e = 0.0f;
            }
            ortho_diagonal<kGram>(p, 0, t.b, first_row + rr, sum);
        }
        __syncthreads();
    }
    const bool again = ortho_again<kGram>(p, t);
    if (warp >= 2) {
        #pragma unroll 4
        for (int32_t k = 0; k < 1 << log8; ++k) {
            const int32_t e = k * 128 + static_cast<int32_t>(threadIdx.x) - 64;          // (by rows)
            const int32_t g = e & ((1 << log8) - 1), rr = e >> log8;
            if (!ortho_inside<kGram>(p, first_row + rr, first_col + g * 8)) continue;
            F2 v[4];
            ortho_load8(at_of(0, 2 * g, rr), at_of(0, 2 * g + 1, rr), v);
            #pragma unroll 2
            for (int32_t s = 1; s < S; ++s) {
                F2 o[4];
                ortho_load8(at_of(s, 2 * g, rr), at_of(s, 2 * g + 1, rr), o);
                #pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = add2(v[i], o[i]);
            }
            const F2 none[4] = {};
            ortho_finish<kGram>(p, 0, t.b, first_row + rr, first_col + g * 8, OrthoIn<kGram>{}, none, v);
            // in the place of the first source's sums, which this thread alone reads
            if (again) ortho_store8(at_of(0, 2 * g, rr), at_of(0, 2 * g + 1, rr), v);
        }
    }
    if (!again) return;
    __syncthreads();
    #pragma unroll 1
    for (int32_t e = threadIdx.x; e < 128 << log4; e += kOrthoTileThreads) {
        const int32_t rr = e & 127, c4 = e >> 7;
        if (ortho_inside<kGram>(p, first_row + rr, first_col + 4 * c4))
            ortho_mirror<kGram>(p, t.b, first_row + rr, first_col + 4 * c4, *at_of(0, c4, rr));
    }
}

// NB: its columns, 32 (not where B's boxes are of 64 columns: ortho_b_mn), 64 or 128.
template <int MODE, int NB>
__global__ void __launch_bounds__(kOrthoTileThreads, 1)
    ortho_tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ OrthoParams p) {
    static_assert(NB == 128 || NB == 64 || (NB == 32 && MODE < kStep), "columns");
    const bool amn = ortho_a_mn(p, MODE), bmn = ortho_b_mn(p, MODE);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOrthoStages * kOrthoStage);
    uint64_t* empty = full + kOrthoStages;
    uint64_t* done = empty + kOrthoStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    __shared__ volatile int abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t S = MODE == kGram ? p.splits : 1;
    const uint32_t rank = S > 1 ? cluster_ctarank() : 0u;
    const OrthoTile t = ortho_tile<MODE>(p, static_cast<int32_t>(blockIdx.x) / S);
    const int32_t step = p.first / 3, k_blocks = MODE == kGram ? p.k_gram : p.k_other;
    const int32_t kb0 = static_cast<int32_t>(rank) * k_blocks / S;
    const int32_t kb1 = static_cast<int32_t>(rank + 1) * k_blocks / S;

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
        tmem_alloc(tmem_slot, NB);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();
    grid_dependents_launch();

    // The epilogue's place: 32 rows and, unless K is split, blocks of 32 columns, of which
    // the first two's inputs are on their way while the products run.
    const int quarter = warp & 3;
    const int32_t row0 = t.i * 128 + quarter * 32;
    const int32_t blocks = S > 1 ? 0 : ortho_block_count<MODE>(p, row0, t.j * NB, NB / 32);
    OrthoBlock<MODE> in0, in1;
    if (warp >= 2) {
        if (blocks > 0) ortho_read_block<MODE>(p, step, t.b, row0, t.j * NB, in0);
        if (blocks > 1) ortho_read_block<MODE>(p, step, t.b, row0, t.j * NB + 32, in1);
    }

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t keep = l2_policy_evict_last();
            uint32_t armed = 0;
            for (int32_t kb = kb0; kb < kb1; ++kb, ++armed) {
                const uint32_t s = armed % kOrthoStages, round = armed / kOrthoStages;
                if (!ortho_wait(&empty[s], (round & 1u) ^ 1u, &abort_flag, p)) break;
                uint8_t* sa = smem + s * kOrthoStage;
                mbar_arrive_expect_tx(&full[s], kOrthoBox + NB * 256u);
                if ((p.debug_flags & 1u) && armed == 0 && blockIdx.x == 0) continue;   // test hook: no load
                const int32_t k0 = kb * 128, kc = kb * 2;
                tma_load_4d(sa, &tmA, &full[s], 0, amn ? k0 : t.i * 128, amn ? t.i * 2 : kc, t.b, keep);
                tma_load_4d(sa + kOrthoBox, &tmB, &full[s], 0, bmn ? k0 : t.j * NB, bmn ? t.j * (NB / 64) : kc, t.b, keep);
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
                const uint32_t sa = base + s * kOrthoStage;
                if constexpr (MODE == kGram && NB > 32) {
                    if (bmn) ortho_mma<true, true, false, NB>(tmem, sa, used == 0);
                    else ortho_mma<false, false, false, NB>(tmem, sa, used == 0);
                } else if constexpr (MODE >= kStep) {
                    if (bmn) ortho_mma<false, true, false, NB>(tmem, sa, used == 0);
                    else ortho_mma<false, false, false, NB>(tmem, sa, used == 0);
                } else {
                    ortho_mma<false, false, false, NB>(tmem, sa, used == 0);
                }
                tc_commit(&empty[s]);
            }
            tc_commit(done);
            if (!mbar_wait(done, 0, p.wait_limit_ns)) ortho_give_up(p, &abort_flag);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (S > 1) cluster_sync_all();
    tc_fence_after_sync();
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    if (S > 1) {
        // Every CTA of the cluster is through with its stages: their memory becomes the
        // exchange buffer [source][four columns of mine][row] of float4s, the rows of
        // different columns turned against each other, so that the units of eight lanes
        // meet in no bank.
        if constexpr (MODE == kGram) ortho_join<NB>(p, t, S, rank, taddr, smem, &abort_flag);
    } else if (warp >= 2 && !abort_flag) {
        float4* turn = reinterpret_cast<float4*>(smem) + (warp - 2) * 256;      // the stages are free
        ortho_blocks<MODE>(p, step, t, row0, t.j * NB, blocks, taddr, in0, in1, turn);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 1) tmem_dealloc(tmem, NB);
}

}  // namespace gemm103
