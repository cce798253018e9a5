// How the 8-bit pair kernel cuts a group's rows into tiles, for host and device, and what
// that costs.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define FP8_TILES_FN __host__ __device__ inline
#else
#define FP8_TILES_FN inline
#endif

namespace fp8_dev {

// Rows are up to GEMM_F16_MAX_DIM (2^31 - 2^16), and up to 2^26 parts of them: the sums
// that round a quotient up are taken without a sign, or they would pass 2^31.
FP8_TILES_FN int parts_of(int rows, int w) { return static_cast<int>((static_cast<uint32_t>(rows) + w - 1) / w); }

FP8_TILES_FN int width_of(int rows, int parts)
{
    return parts ? static_cast<int>(((static_cast<uint32_t>(rows) + parts - 1) / parts + 31) & ~31u) : 0;
}

// What the clusters' turns cost in cycles: a step of 128 values brings 16 KB of weights and
// 64 bytes a column to either CTA, at 64 bytes a cycle 256 + W cycles, which is no less
// than its 2 W cycles of MMA (measured: 321 cycles at W = 64, 376 at 128, 485 at 224), and a
// tile costs some 600 more, with one accumulator 3000.
FP8_TILES_FN int64_t cost_of(int tiles, int widest, int clusters, int steps)
{
    const int turns = (tiles + clusters - 1) / clusters;
    return turns * (static_cast<int64_t>(steps) * (widest + 256) + (widest > 224 && turns > 1 ? 3000 : 600));
}

}  // namespace fp8_dev

#undef FP8_TILES_FN
