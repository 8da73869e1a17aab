// int8_tiles.hpp -- which tile an 8-bit product takes: the one with the least
// expected time.  Host code only.
//
// The constants are least-squares fits to measured times, with no negative
// constant, of relative errors weighted by sqrt(fastest time / time) and without
// times over twice the fastest.  perf/tiles.py makes the tables from the times in
// profiles/tiles_int8.json and compares the choice with the fastest tile.
#pragma once

#include <cmath>
#include <cstdint>

namespace iqk {

// The expected time of a tile size in microseconds: `once` for the product, and
// for each tile that a compute unit takes in turn `start` (its first loads and
// its results) and `depth` for every 1024 of the depth.  Where not all units are
// busy to the end those that are go faster, the small tiles because they share
// L2 and LDS, the large ones the card's power: `start_full` and `depth_full`
// count with the tiles a unit has on average, not the most that one has.
struct TileTime {
    int rows, channels;
    double once, start, depth, start_full, depth_full;
};

inline double expected_time(int64_t rows, int64_t channels, int64_t depth, int experts, int cus,
                            const TileTime& t)
{
    double row_tiles = (double)((rows + t.rows - 1) / t.rows);
    if (experts) {
        // As if every row chose its expert evenly: the last tile of an expert
        // that has rows is half full.
        const double each = (double)rows / experts;
        const double used = experts * (1.0 - std::exp(-each));
        row_tiles = std::fmax(used, (double)rows / t.rows + 0.5 * used);
    }
    const double average = row_tiles * ((channels + t.channels - 1) / t.channels) / cus;
    const double k = depth / 1024.0;
    return t.once + std::ceil(average) * (t.start + t.depth * k) +
           average * (t.start_full + t.depth_full * k);
}

// Fitted to 700 products of 1 to 4096 tokens, 256 to 5632 channels and depths of
// 512 to 5632.  The tile with the least expected time took 0.2 % longer than the
// fastest on average, 7 % at worst (of 695: in five it was not timed); without the
// four sizes with a side of 192 1.5 % and 38 %, 128 x 128 alone 77 %.
constexpr TileTime kDense[] = {
    {16, 16, 3.10, 0.06, 0.34, 0.10, 0.0},
    {32, 32, 3.08, 0.22, 0.71, 0.39, 0.0},
    {64, 64, 2.11, 2.04, 1.33, 0.93, 0.26},
    {64, 128, 2.29, 1.86, 2.43, 1.80, 0.05},
    {64, 192, 2.52, 2.44, 3.23, 2.06, 0.11},
    {128, 128, 2.66, 2.39, 3.14, 2.45, 0.39},
    {128, 192, 2.87, 3.81, 4.16, 2.63, 0.53},
    {192, 128, 2.73, 3.28, 3.93, 2.76, 0.70},
    {128, 256, 2.79, 3.13, 5.56, 4.49, 1.71},
    {192, 192, 3.49, 4.42, 5.03, 3.57, 2.50},
    {256, 256, 3.42, 8.79, 5.83, 4.41, 5.17}};
// To 540 products by expert, 1 to 4096 tokens of 1, 2 and 8 choices, 8 to 128
// experts, chosen evenly and not, weights out of HBM: 4 % longer than the fastest
// of fifteen tiles on average, 55 % at worst, where a distribution needs just over
// a round of tiles.  Tiles take longer than in a dense product.
constexpr TileTime kByExpert[] = {
    {16, 16, 4.28, 0.0, 0.58, 0.55, 0.0},
    {32, 64, 4.91, 0.0, 1.62, 1.24, 0.41},
    {32, 128, 7.13, 0.0, 1.85, 1.17, 1.47},
    {64, 64, 5.04, 0.0, 1.98, 1.78, 0.32},
    {64, 128, 4.59, 0.0, 2.82, 4.69, 1.23},
    {64, 192, 5.45, 0.0, 3.83, 5.50, 1.58},
    {128, 128, 4.74, 0.0, 3.06, 6.10, 2.20},
    {128, 192, 3.32, 3.04, 4.62, 5.46, 2.22},
    {192, 192, 1.31, 6.45, 4.83, 3.57, 4.39},
    {256, 256, 6.35, 6.70, 5.26, 3.39, 8.68}};
// To 510 dense products whose rows do not start on 16 bytes: 2 % longer than the
// fastest of six tiles, 20 % at worst.  Products by expert with such rows take this
// table too; it was not fitted to times of theirs.
constexpr TileTime kUnaligned[] = {
    {16, 16, 7.38, 0.34, 0.84, 0.46, 0.0},
    {32, 32, 7.09, 2.27, 1.74, 0.0, 0.0},
    {64, 64, 7.37, 2.78, 3.30, 0.41, 0.0},
    {128, 128, 2.94, 9.96, 6.87, 2.17, 0.0},
    {128, 256, 2.95, 9.78, 14.62, 4.83, 0.0}};

// The entry with the least expected time.
template <int kN>
inline int fastest_tile(int64_t rows, int64_t channels, int64_t depth, int experts, int cus,
                        const TileTime (&tiles)[kN])
{
    int best = 0;
    double least = expected_time(rows, channels, depth, experts, cus, tiles[0]);
    for (int i = 1; i < kN; ++i) {
        const double time = expected_time(rows, channels, depth, experts, cus, tiles[i]);
        if (time < least) {
            least = time;
            best = i;
        }
    }
    return best;
}

}  // namespace iqk
