// expert_tiles.hpp -- which rows and channels a workgroup of a product takes,
// dense or with a weight per expert, shared by the 8-bit and 4-bit products.  A
// Product has rows, tokens, order, offsets, experts, top_k and first_tile.
#pragma once

#include "layers_common.hpp"

namespace iqk {

struct Tile {
    int64_t row0;      // first row of y
    int64_t row_end;   // rows of this tile end here (exclusive)
    int channel_tile;
    int expert;        // -1: dropped rows, written as zeros; -2: no tile
};

__device__ __forceinline__ int64_t clamp_offset(int32_t v, int64_t rows)
{
    return min(max((int64_t)v, (int64_t)0), rows);
}

// Rows of segment e: expert e, or the dropped rows where e == experts.
template <class Product>
__device__ __forceinline__ void segment(const Product& p, int e, int64_t* lo, int64_t* hi)
{
    *lo = clamp_offset(p.offsets[e], p.rows);
    *hi = e < p.experts ? clamp_offset(p.offsets[e + 1], p.rows) : p.rows;
}

// Consecutive tiles go to one XCD (workgroup i runs on XCD i % 8), so those
// that share a panel of the weight share an L2.
__device__ __forceinline__ int64_t by_xcd(int64_t pid, int64_t total)
{
    const int64_t each = total / 8, more = total % 8;
    const int64_t xcd = pid % 8;
    return xcd * each + min(xcd, more) + pid / 8;
}

template <int kRows, class Product>
__device__ __forceinline__ Tile dense_tile(const Product& p, int channel_tiles)
{
    // Bands of kBand row tiles, channel tile by channel tile.
    constexpr int kBand = 8;
    const int64_t row_tiles = (p.rows + kRows - 1) / kRows;
    const int64_t id = by_xcd(p.first_tile + blockIdx.x, row_tiles * channel_tiles);
    const int64_t band = id / (kBand * (int64_t)channel_tiles);
    const int64_t in_band = id - band * kBand * channel_tiles;
    const int64_t height = min((int64_t)kBand, row_tiles - band * kBand);
    Tile t;
    t.row0 = (band * kBand + in_band % height) * kRows;
    t.row_end = p.rows;
    t.channel_tile = (int)(in_band / height);
    t.expert = 0;
    return t;
}

// Tiles of each expert one after another; the grid is as large as any
// distribution of the rows could need, and the rest of it ends at once.  Every
// wave finds its tile by itself: lane l counts the tiles of segment l, and the
// counts are summed up across the lanes, 64 segments at a time (up to 63
// experts the offsets are read once).
template <int kRows, class Product>
__device__ __forceinline__ Tile expert_tile(const Product& p, int channel_tiles)
{
    const int lane = threadIdx.x % kWave;
    int64_t lo = 0, hi = 0;
    int count = 0, last = 0;          // of this lane's segment, and up to it
    auto count_from = [&](int e0) {
        const int e = e0 + lane;
        lo = hi = 0;
        if (e <= p.experts) segment(p, e, &lo, &hi);
        count = hi > lo ? (int)((hi - lo + kRows - 1) / kRows) : 0;
        last = count;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int up = __shfl_up(last, d);
            if (lane >= d) last += up;
        }
        return __shfl(last, kWave - 1);
    };
    int total = count_from(0);
    if (p.experts >= kWave) {
        for (int e0 = kWave; e0 <= p.experts; e0 += kWave) total += count_from(e0);
    }
    Tile t = {0, 0, 0, -2};
    const int64_t tiles = (int64_t)total * channel_tiles;
    if (p.first_tile + blockIdx.x >= tiles) return t;
    const int64_t id = by_xcd(p.first_tile + blockIdx.x, tiles);
    const int row_tile = (int)(id / channel_tiles);
    t.channel_tile = (int)(id - (int64_t)row_tile * channel_tiles);
    int before = 0;
    for (int e0 = 0; e0 <= p.experts; e0 += kWave) {
        const int all = p.experts >= kWave ? count_from(e0) : total;
        const int first = before + last - count;
        const uint64_t mine = __ballot(row_tile >= first && row_tile < first + count);
        if (mine) {
            const int l = __ffsll((unsigned long long)mine) - 1;
            const int at = row_tile - __shfl(first, l);
            t.expert = e0 + l < p.experts ? e0 + l : -1;
            t.row0 = (int64_t)__shfl((int)lo, l) + (int64_t)at * kRows;
            t.row_end = __shfl((int)hi, l);
            return t;
        }
        before += all;
    }
    return t;
}

// The row of x that row r of y takes.
template <class Product>
__device__ __forceinline__ int64_t token_of(const Product& p, int64_t r)
{
    if (!p.order) return r;
    const int64_t t = (uint32_t)p.order[r] / (uint32_t)p.top_k;
    return min(t, p.tokens - 1);
}

}  // namespace iqk
