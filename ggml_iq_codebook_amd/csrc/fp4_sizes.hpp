// fp4_sizes.hpp -- how many rows and channels a workgroup of a product with 4-bit
// weights takes: the size with the least expected time.  Host code only.
//
// Sizes of 64 channels and more are the tile kernel's (64 x 64, 64 x 256 and 128 x
// 256), the others those of the kernel for few rows, which has its operands in
// registers and reads a weight again for each of its row tiles.  The constants are fits
// to measured times like those of int8_tiles.hpp, made by perf/fp4_sizes.py from
// profiles/sizes_fp4.json.  Sizes that were tried and are not worth their code: 2 x 16,
// 64 x 128 and 128 x 128 (under 0.3 % on average, 64 x 128 1.2 % by expert in bf16).
// The times hold for 256 compute units, a whole card: the choice also sizes the
// workspace, which has to be the same wherever it is asked.
#pragma once

#include "int8_tiles.hpp"
#include "iq_codec.h"

namespace iqk {

// To 420 products of bf16 activations, 1 to 4096 rows: 0.3 % longer than the fastest
// on average, 16 % at worst.
constexpr TileTime kDenseBf16[] = {
    {1, 16, 3.07, 0.32, 0.22, 0.47, 0.0},
    {4, 16, 3.14, 0.38, 0.28, 0.34, 0.0},
    {8, 16, 3.2, 0.44, 0.33, 0.32, 0.03},
    {16, 16, 3.29, 0.54, 0.42, 0.19, 0.07},
    {16, 32, 2.31, 2.37, 0.64, 0.2, 0.27},
    {32, 32, 2.27, 3.14, 0.77, 0.0, 0.6},
    {64, 32, 2.02, 4.9, 1.45, 0.0, 0.79},
    {64, 64, 5.13, 0.0, 3.23, 1.69, 0.0},
    {64, 256, 3.08, 2.99, 7.63, 4.43, 1.17},
    {128, 256, 3.16, 4.99, 9.1, 5.52, 3.13}};
// To 320 of fp16 ones: 0.7 %, 25 % at worst.
constexpr TileTime kDenseF16[] = {
    {1, 16, 3.36, 0.24, 0.28, 0.52, 0.01},
    {4, 16, 3.39, 0.33, 0.43, 0.52, 0.0},
    {8, 16, 3.54, 0.2, 0.63, 0.57, 0.0},
    {16, 16, 3.87, 0.23, 1.0, 0.6, 0.0},
    {16, 32, 2.05, 3.06, 1.18, 0.0, 0.43},
    {32, 32, 2.11, 4.08, 1.99, 0.02, 0.65},
    {64, 64, 8.07, 0.0, 6.63, 1.67, 0.0},
    {64, 256, 7.27, 1.87, 14.9, 5.96, 2.49},
    {128, 256, 10.14, 0.43, 19.78, 11.59, 2.69}};
// To 320 of fp32 ones: 0.5 %, 46 % at worst.
constexpr TileTime kDenseF32[] = {
    {1, 16, 3.53, 0.01, 0.35, 0.63, 0.05},
    {4, 16, 3.46, 0.37, 0.57, 0.43, 0.0},
    {8, 16, 3.47, 0.3, 0.84, 0.45, 0.0},
    {16, 16, 1.86, 2.26, 1.36, 0.42, 0.17},
    {16, 32, 2.42, 2.31, 1.66, 0.9, 0.25},
    {32, 32, 2.73, 3.68, 3.09, 0.0, 1.84},
    {64, 64, 9.09, 0.0, 9.76, 1.98, 0.0},
    {64, 256, 9.99, 0.0, 19.95, 9.24, 4.96},
    {128, 256, 12.32, 0.68, 28.93, 15.41, 3.6}};
// To 360 products by expert of bf16 activations, 8 to 128 experts, chosen evenly and
// not: 2.7 %, 45 % at worst.
constexpr TileTime kExpertBf16[] = {
    {1, 16, 3.41, 0.0, 0.22, 0.98, 0.04},
    {4, 16, 3.76, 0.0, 0.19, 1.4, 0.19},
    {8, 16, 3.68, 0.0, 0.3, 1.43, 0.16},
    {16, 16, 3.98, 0.0, 0.4, 1.6, 0.15},
    {16, 32, 3.05, 1.95, 0.72, 1.99, 0.38},
    {32, 32, 2.46, 4.51, 0.71, 0.58, 0.74},
    {64, 64, 5.74, 0.0, 2.34, 2.35, 1.18},
    {64, 256, 2.93, 3.45, 7.4, 4.57, 1.41},
    {128, 256, 4.22, 4.35, 9.21, 5.15, 2.46}};
// To 280 of fp16 ones: 3.1 %, 62 % at worst.
constexpr TileTime kExpertF16[] = {
    {1, 16, 3.44, 0.0, 0.13, 1.11, 0.15},
    {4, 16, 3.66, 0.0, 0.44, 1.65, 0.0},
    {8, 16, 3.47, 0.11, 0.6, 1.58, 0.0},
    {16, 16, 4.06, 0.0, 0.92, 1.9, 0.0},
    {16, 32, 3.46, 1.91, 0.68, 2.47, 1.04},
    {32, 32, 2.9, 5.38, 0.47, 0.19, 2.28},
    {64, 64, 8.06, 0.0, 5.42, 2.75, 0.66},
    {64, 256, 5.41, 2.01, 14.69, 6.91, 0.4},
    {128, 256, 9.66, 2.47, 19.92, 7.04, 2.51}};
// To 280 of fp32 ones: 3.2 %, 48 % at worst.
constexpr TileTime kExpertF32[] = {
    {1, 16, 3.37, 1.1, 0.0, 0.0, 0.35},
    {4, 16, 3.77, 1.12, 0.32, 0.56, 0.21},
    {8, 16, 3.61, 1.25, 0.57, 0.35, 0.19},
    {16, 16, 3.22, 2.49, 0.75, 0.82, 0.83},
    {16, 32, 2.36, 4.49, 0.55, 0.0, 1.53},
    {32, 32, 3.77, 5.13, 0.0, 0.0, 4.87},
    {64, 64, 8.85, 0.0, 7.4, 3.11, 1.52},
    {64, 256, 8.33, 1.39, 15.9, 5.94, 6.43},
    {128, 256, 4.13, 9.26, 29.45, 5.74, 2.33}};

template <int kN>
inline int fastest_size(int64_t rows, int64_t channels, int64_t depth, int experts,
                        const TileTime (&sizes)[kN])
{
    const TileTime& t = sizes[fastest_tile(rows, channels, depth, experts, 256, sizes)];
    return t.rows * 1000 + t.channels;
}

// As rows * 1000 + channels.
inline int fp4_size(int dtype, int64_t rows, int64_t channels, int64_t depth, int experts)
{
    if (experts)
        return dtype == IQ_DTYPE_BF16  ? fastest_size(rows, channels, depth, experts, kExpertBf16)
               : dtype == IQ_DTYPE_F16 ? fastest_size(rows, channels, depth, experts, kExpertF16)
                                       : fastest_size(rows, channels, depth, experts, kExpertF32);
    return dtype == IQ_DTYPE_BF16  ? fastest_size(rows, channels, depth, 0, kDenseBf16)
           : dtype == IQ_DTYPE_F16 ? fastest_size(rows, channels, depth, 0, kDenseF16)
                                   : fastest_size(rows, channels, depth, 0, kDenseF32);
}

}  // namespace iqk
