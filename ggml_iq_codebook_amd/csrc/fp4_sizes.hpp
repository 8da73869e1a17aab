// fp4_sizes.hpp -- how many rows, channels and waves a workgroup of a product with
// 4-bit weights has: the size with the least expected time.  Host code only.
//
// Sizes of 64 channels and more are the tile kernel's, the others those of the kernel
// of few rows, which reads a weight again for each of its row tiles and is taken up to
// 12 of them.  (That limit was set by hand, these sizes were hardly timed beyond it, and just
// beyond it is the worst choice of all: fp32 193 x 1092 x 4800 takes 32 x 64 and 56 us, where
// 16 x 32 took 28.)  Dense products of few rows have a workgroup to a compute unit, whose
// eight waves share the depth; those by expert have many, and smaller ones hide each
// other's start (16 tokens, 2 of 16 experts of 1536 x 4096, at the time this was decided:
// 20.7 us with eight waves of 4 x 16, 15.1 with four of 4 x 32; 8 x 32 took the latter's
// place).  The constants are fits to measured times, made by perf/fp4_sizes.py from
// profiles/sizes_fp4.json.  The times are those of earlier kernels than these: fp32 and
// bf16 from before fp16 activations were multiplied as fp16, fp16 from after that, all from
// before the tile kernel's slots without bank conflicts and its loop in fewer registers,
// which made tiles up to 10 % faster.  They hold for 256 compute units, a whole card: the
// choice also sizes the workspace, which has to be the same wherever it is asked.
#pragma once

#include <cmath>
#include <cstdint>

#include "iq_codec.h"

namespace iqk {

// The expected time in microseconds: `once` for the product, for each turn of `slots`
// workgroups that share a compute unit `start` and, for every 1024 of the depth, `depth`;
// `start_full` and `depth_full` count with the workgroups that a unit has on average.
struct Fp4Size {
    int rows, channels, waves, slots;
    double once, start, depth, start_full, depth_full;
};

// To 420 products of bf16 activations, 1 to 4096 rows: 0.8 % longer than the fastest
// on average, 37 % at worst.
constexpr Fp4Size kDenseBf16[] = {
    {1, 16, 8, 2, 2.59, 1.02, 0.16, 0.34, 0.15},
    {4, 16, 8, 1, 3.1, 0.57, 0.26, 0.1, 0.04},
    {8, 16, 8, 1, 3.29, 0.4, 0.32, 0.32, 0.05},
    {16, 16, 4, 4, 3.03, 0.58, 0.56, 0.25, 0.32},
    {16, 16, 8, 1, 3.35, 0.51, 0.44, 0.22, 0.06},
    {32, 32, 8, 1, 2.47, 2.94, 0.81, 0.1, 0.55},
    {32, 64, 4, 5, 3.49, 0.78, 2.41, 0.64, 1.17},
    {32, 128, 4, 3, 2.39, 2.17, 3.29, 0.56, 2.24},
    {64, 128, 4, 2, 2.5, 2.62, 4.84, 1.17, 2.84},
    {128, 256, 8, 1, 3.66, 4.04, 8.85, 5.51, 4.72}};
// To 320 of fp16 ones: 1.1 %, 27 % at worst.
constexpr Fp4Size kDenseF16[] = {
    {1, 16, 8, 1, 3.05, 0.67, 0.25, 0.06, 0.0},
    {4, 16, 8, 1, 3.35, 0.28, 0.32, 0.42, 0.0},
    {8, 16, 8, 2, 2.73, 1.09, 0.3, 0.32, 0.26},
    {16, 16, 4, 4, 2.92, 0.83, 0.65, 0.19, 0.34},
    {16, 16, 8, 2, 2.72, 1.27, 0.4, 0.34, 0.33},
    {32, 32, 8, 1, 2.0, 3.51, 0.99, 0.0, 0.45},
    {32, 64, 4, 4, 2.43, 2.44, 3.09, 0.47, 1.32},
    {32, 128, 4, 3, 2.53, 2.57, 4.46, 0.86, 2.17},
    {64, 128, 4, 2, 2.84, 2.64, 7.39, 1.84, 2.51},
    {128, 256, 8, 1, 2.93, 5.5, 9.31, 5.88, 3.23}};
// To 320 of fp32 ones: 0.8 %, 100 % at worst.
constexpr Fp4Size kDenseF32[] = {
    {1, 16, 8, 2, 2.64, 0.94, 0.32, 0.45, 0.23},
    {4, 16, 8, 1, 3.47, 0.43, 0.53, 0.29, 0.04},
    {8, 16, 8, 2, 2.9, 0.96, 0.69, 0.4, 0.49},
    {16, 16, 4, 3, 3.55, 0.62, 1.66, 0.25, 0.8},
    {16, 16, 8, 1, 2.06, 2.31, 1.24, 0.0, 0.42},
    {16, 32, 8, 1, 2.31, 2.78, 1.49, 0.0, 0.63},
    {32, 64, 4, 3, 7.15, 0.0, 8.85, 1.46, 1.58},
    {32, 128, 4, 3, 7.2, 0.0, 10.25, 2.62, 4.14},
    {64, 128, 4, 2, 6.57, 1.45, 16.21, 5.5, 4.71},
    {128, 256, 8, 1, 12.11, 1.8, 26.83, 13.8, 9.59}};
// To 360 products by expert of bf16 activations, 8 to 128 experts, chosen evenly and
// not: 1.9 %, 57 % at worst.
constexpr Fp4Size kExpertBf16[] = {
    {1, 16, 4, 8, 2.43, 2.12, 0.07, 0.17, 0.22},
    {4, 16, 4, 5, 3.45, 1.22, 0.17, 0.22, 0.33},
    {8, 16, 4, 4, 3.01, 1.86, 0.17, 0.11, 0.43},
    {8, 32, 4, 3, 3.19, 2.25, 0.39, 0.28, 0.65},
    {16, 32, 4, 3, 3.27, 2.63, 0.56, 0.39, 0.72},
    {32, 64, 4, 5, 3.91, 1.45, 2.6, 0.73, 1.33},
    {32, 128, 4, 3, 4.36, 1.09, 3.83, 1.19, 2.11},
    {64, 128, 4, 2, 3.1, 3.14, 5.47, 1.23, 2.91},
    {128, 256, 8, 1, 2.5, 7.13, 8.53, 3.08, 3.61}};
// To 280 of fp16 ones: 1.6 %, 37 % at worst.
constexpr Fp4Size kExpertF16[] = {
    {1, 16, 4, 5, 3.0, 1.26, 0.33, 0.27, 0.2},
    {4, 16, 4, 4, 3.37, 0.88, 0.57, 0.45, 0.23},
    {8, 16, 4, 4, 3.51, 0.72, 0.62, 0.5, 0.29},
    {16, 32, 4, 2, 3.15, 2.61, 0.78, 0.68, 0.72},
    {32, 64, 4, 4, 3.78, 1.59, 4.0, 0.77, 1.43},
    {32, 128, 4, 3, 4.04, 1.87, 4.52, 1.05, 2.31},
    {64, 128, 4, 2, 2.53, 4.37, 6.32, 1.07, 2.85},
    {128, 256, 8, 1, 4.19, 5.33, 9.12, 6.39, 2.29}};
// To 280 of fp32 ones: 2.0 %, 51 % at worst.
constexpr Fp4Size kExpertF32[] = {
    {1, 16, 4, 5, 2.64, 1.73, 0.38, 0.25, 0.23},
    {4, 16, 4, 5, 3.57, 0.97, 0.67, 0.57, 0.42},
    {8, 16, 4, 4, 3.57, 0.97, 1.07, 0.52, 0.5},
    {8, 32, 4, 2, 3.81, 1.19, 1.38, 1.18, 0.63},
    {16, 32, 4, 2, 3.32, 3.44, 1.32, 0.38, 1.15},
    {32, 64, 4, 5, 6.11, 1.55, 7.68, 1.1, 3.06},
    {32, 128, 4, 3, 7.52, 0.0, 10.44, 2.46, 3.86},
    {64, 128, 4, 2, 7.56, 0.55, 17.47, 4.08, 3.53},
    {128, 256, 8, 1, 8.53, 3.01, 27.83, 12.5, 5.22}};

// A size as one number.
constexpr int size_key(int rows, int channels, int waves)
{
    return (rows * 1000 + channels) * 100 + waves;
}
// Whether it is the tile kernel's.
constexpr bool is_tile(int key) { return key / 100 % 1000 >= 64; }

template <int kN>
inline int fastest_size(int64_t rows, int64_t channels, int64_t depth, int experts,
                        const Fp4Size (&sizes)[kN])
{
    int best = 0;
    double least = 0.0;
    for (const Fp4Size& s : sizes) {
        double tiles = (double)((rows + s.rows - 1) / s.rows), each = (double)rows;
        if (experts) {
            // As if every row chose its expert evenly: the last tile of an expert that
            // has rows is half full.
            each /= experts;
            const double used = experts * (1.0 - std::exp(-each));
            tiles = std::fmax(used, (double)rows / s.rows + 0.5 * used);
        }
        if (s.channels < 64 && each > 12.0 * s.rows) continue;
        const double average = tiles * (double)((channels + s.channels - 1) / s.channels) / 256.0;
        const double k = depth / 1024.0;
        const double time = s.once + std::ceil(average / s.slots) * (s.start + s.depth * k) +
                            average * (s.start_full + s.depth_full * k);
        if (!best || time < least) {
            least = time;
            best = size_key(s.rows, s.channels, s.waves);
        }
    }
    return best;
}

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
