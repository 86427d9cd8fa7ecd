// stream_k.h -- who takes what of a stream-K schedule: the k-blocks of all tiles
// in a line, tile after tile, cut into one range of L for each unit (a CTA or a
// CTA pair).
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define GEMM103_HD __host__ __device__ __forceinline__
#else
#define GEMM103_HD inline
#endif

namespace gemm103 {

// The unit that block (or pair of blocks) `b` of `units` is.  A tile that several
// units share is finished by the first of them, which waits for the others' sums:
// for units behind its own.  So the last blocks are the first units: blocks are
// started in order (measured, of clusters too), and one that waits does so for
// blocks started before it, which wait for none behind them in turn.  It never
// keeps an SM from a block that it waits for, whatever else runs on the GPU -- two
// such kernels on two streams, say, each of which has only part of its blocks
// started.  The number is its own inverse: block b is unit stream_k_unit(b), and
// unit u is block stream_k_unit(u).
GEMM103_HD int32_t stream_k_unit(int32_t b, int32_t units) { return units - 1 - b; }

// The first and the last unit with k-blocks of a tile of KB.
GEMM103_HD int32_t stream_k_first(int32_t tile, int32_t KB, int32_t L) {
    return static_cast<int32_t>(static_cast<int64_t>(tile) * KB / L);
}
GEMM103_HD int32_t stream_k_last(int32_t tile, int32_t KB, int32_t L) {
    return static_cast<int32_t>((static_cast<int64_t>(tile + 1) * KB - 1) / L);
}

}  // namespace gemm103
