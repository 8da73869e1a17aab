// int8_matmul.hip -- products in 8-bit integers on the matrix cores, with a
// scale per token and per output channel, dense or with a weight per expert:
//   y[t][n] = (float)(sum_i x[t][i] * w[n][i]) * x_scale[t] * w_scale[n].
//
// The sums are exact in 32-bit integers, so neither tiling nor the order of the
// depth changes a result.  Both operands hold their depth innermost, which is
// how the matrix instructions take it: lane l of v_mfma_i32_32x32x32_i8
// supplies row l%32, depth 16*(l/32)..+15, as one 16-byte register group.
// The weight is the first operand, so a lane's results are 4 consecutive
// channels of one token and go out as one store.
#include <hip/hip_runtime.h>

#include "iq_layers.h"
#include "layers_common.hpp"
#include "layers_launch.hpp"

namespace iqk {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

constexpr int kDepth = 128;           // bytes of a row in a staged tile

// ---------------------------------------------------------------------------
// Which rows a tile works on
// ---------------------------------------------------------------------------

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
__device__ __forceinline__ void segment(const Int8Product& p, int e, int64_t* lo, int64_t* hi)
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

template <int kRows>
__device__ __forceinline__ Tile dense_tile(const Int8Product& p, int channel_tiles)
{
    // Bands of kBand row tiles, channel tile by channel tile.
    constexpr int kBand = 4;
    const int64_t row_tiles = (p.rows + kRows - 1) / kRows;
    const int64_t id = by_xcd(blockIdx.x, row_tiles * channel_tiles);
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
// wave finds its tile by itself, 64 segments at a time.
template <int kRows>
__device__ __forceinline__ Tile expert_tile(const Int8Product& p, int channel_tiles)
{
    const int lane = threadIdx.x % kWave;
    int64_t total = 0;
    for (int e0 = 0; e0 <= p.experts; e0 += kWave) {
        const int e = e0 + lane;
        int64_t lo = 0, hi = 0;
        if (e <= p.experts) segment(p, e, &lo, &hi);
        int count = hi > lo ? (int)((hi - lo + kRows - 1) / kRows) : 0;
#pragma unroll
        for (int d = kWave / 2; d; d >>= 1) count += __shfl_xor(count, d);
        total += count;
    }
    Tile t = {0, 0, 0, -2};
    if ((int64_t)blockIdx.x >= total * channel_tiles) return t;
    const int64_t id = by_xcd(blockIdx.x, total * channel_tiles);
    const int64_t row_tile = id / channel_tiles;
    t.channel_tile = (int)(id - row_tile * channel_tiles);
    int64_t before = 0;
    for (int e0 = 0; e0 <= p.experts; e0 += kWave) {
        const int e = e0 + lane;
        int64_t lo = 0, hi = 0;
        if (e <= p.experts) segment(p, e, &lo, &hi);
        const int count = hi > lo ? (int)((hi - lo + kRows - 1) / kRows) : 0;
        int sum = count;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int up = __shfl_up(sum, d);
            if (lane >= d) sum += up;
        }
        const int64_t first = before + sum - count;
        const uint64_t mine = __ballot(row_tile >= first && row_tile < first + count);
        if (mine) {
            const int l = __ffsll((unsigned long long)mine) - 1;
            const int64_t at = row_tile - __shfl((int)first, l);
            t.expert = e0 + l < p.experts ? e0 + l : -1;
            segment(p, e0 + l, &lo, &hi);
            t.row0 = lo + at * kRows;
            t.row_end = hi;
            return t;
        }
        before += __shfl(sum, kWave - 1);
    }
    return t;
}

// The row of x that row r of y takes.
__device__ __forceinline__ int64_t token_of(const Int8Product& p, int64_t r)
{
    if (!p.order) return r;
    const int64_t t = (uint32_t)p.order[r] / (uint32_t)p.top_k;
    return min(t, p.tokens - 1);
}

// ---------------------------------------------------------------------------
// Writing results
// ---------------------------------------------------------------------------

// Four consecutive channels of one row of y.
__device__ __forceinline__ void store4(const Int8Product& p, int64_t row, int channel,
                                       const float (&f)[4])
{
    const int64_t at = row * p.ldy + channel;
    if (p.out_dtype == IQ_DTYPE_F32) {
        float* to = static_cast<float*>(p.y) + at;
        if (channel + 4 <= p.channels)
            __builtin_memcpy(to, f, 16);
        else
            for (int i = 0; i < 4; ++i)
                if (channel + i < p.channels) to[i] = f[i];
        return;
    }
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = p.out_dtype == IQ_DTYPE_BF16 ? Value<IQ_DTYPE_BF16>::store(f[i])
                                            : Value<IQ_DTYPE_F16>::store(f[i]);
    uint16_t* to = static_cast<uint16_t*>(p.y) + at;
    if (channel + 4 <= p.channels)
        __builtin_memcpy(to, h, 8);
    else
        for (int i = 0; i < 4; ++i)
            if (channel + i < p.channels) to[i] = h[i];
}

template <int kRows, int kChannels, int kThreads>
__device__ __forceinline__ void store_zeros(const Int8Product& p, const Tile& t)
{
    const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = threadIdx.x; i < kRows * (kChannels / 4); i += kThreads) {
        const int64_t row = t.row0 + i / (kChannels / 4);
        const int channel = t.channel_tile * kChannels + i % (kChannels / 4) * 4;
        if (row < t.row_end && channel < p.channels) store4(p, row, channel, zero);
    }
}

// ---------------------------------------------------------------------------
// The tile kernel
// ---------------------------------------------------------------------------

__device__ const uint4 zeros[1] = {{0u, 0u, 0u, 0u}};

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) void global_void;

// 16 bytes a lane from global memory into LDS at `to` + 16 * lane.
__device__ __forceinline__ void copy_to_lds(const int8_t* from, int8_t* to)
{
    __builtin_amdgcn_global_load_lds((global_void*)(uintptr_t)from, (lds_void*)to, 16, 0, 0);
}

// 16 bytes of a row from depth `at`, zeros beyond its end, at any alignment.
__device__ __forceinline__ uint4 load_codes(const int8_t* row, int at, int depth)
{
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (at + 16 <= depth) {
        __builtin_memcpy(&v, row + at, 16);
    } else if (at < depth) {
        uint32_t u[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (at + i < depth) u[i / 4] |= (uint32_t)(uint8_t)row[at + i] << (8 * (i % 4));
        v = make_uint4(u[0], u[1], u[2], u[3]);
    }
    return v;
}

// kWT x kWC waves share a tile of kRows rows of y by kChannels channels, each
// a part of kRows/kWT by kChannels/kWC, in steps of 128 of the depth.  The
// tiles of both operands are double buffered in LDS: the next step is on its
// way while this one is multiplied.  A row of 128 bytes is stored as 8 pieces
// of 16, piece c in slot c ^ (row % 8), so that lanes reading one piece of
// consecutive rows meet different banks.  kDirect: rows start on 16 bytes and
// the depth is a multiple of 16, and the pieces go straight into LDS;
// otherwise they pass through registers, with the ends of rows cut byte by byte.
template <int kRows, int kChannels, int kWT, int kWC, bool kDirect, bool kExperts>
__global__ __launch_bounds__(kWT* kWC* kWave) void int8_tile_kernel(Int8Product p,
                                                                    int channel_tiles)
{
    constexpr int kWaves = kWT * kWC, kThreads = kWaves * kWave;
    constexpr int kFT = kRows / kWT / 32, kFC = kChannels / kWC / 32;
    constexpr int kLoads = (kRows + kChannels) / 8 / kWaves;   // a wave's, 8 rows each
    static_assert((kRows + kChannels) % (8 * kWaves) == 0 && kChannels % 8 == 0, "tile");
    __shared__ __align__(1024) int8_t staged[2][(kRows + kChannels) * kDepth];

    const Tile t = kExperts ? expert_tile<kRows>(p, channel_tiles)
                            : dense_tile<kRows>(p, channel_tiles);
    if (t.expert == -2) return;
    if (t.expert == -1) {
        store_zeros<kRows, kChannels, kThreads>(p, t);
        return;
    }
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int lane = threadIdx.x % kWave;
    const int channel0 = t.channel_tile * kChannels;
    const int8_t* w = p.w + (int64_t)t.expert * p.w_stride;

    // Staged rows: the weight's channels, then the tokens.  Rows beyond the
    // last repeat it: their results are not stored.
    const int8_t* from[kLoads];
    int piece[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int r = (wave * kLoads + i) * 8 + lane / 8;
        piece[i] = ((lane % 8) ^ (r % 8)) * 16;
        if (r < kChannels) {
            from[i] = w + (int64_t)min(channel0 + r, p.channels - 1) * p.ldw;
        } else {
            const int64_t row = min(t.row0 + r - kChannels, t.row_end - 1);
            from[i] = p.x + (kExperts ? token_of(p, row) : row) * p.ldx;
        }
    }

    uint4 passing[kDirect ? 1 : kLoads];
    auto fetch = [&](int b, int step) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int at = step * kDepth + piece[i];
            if constexpr (kDirect)
                copy_to_lds(at < p.depth ? from[i] + at : reinterpret_cast<const int8_t*>(zeros),
                            &staged[b][(wave * kLoads + i) * 1024]);
            else
                passing[i] = load_codes(from[i], at, p.depth);
        }
    };
    auto arrive = [&](int b) {
        if constexpr (!kDirect) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                *reinterpret_cast<uint4*>(&staged[b][(wave * kLoads + i) * 1024 + lane * 16]) =
                    passing[i];
        }
    };

    v16i acc[kFC][kFT] = {};
    const int wt = wave % kWT, wc = wave / kWT;
    const int row_c = wc * kFC * 32 + lane % 32;
    const int row_t = kChannels + wt * kFT * 32 + lane % 32;
    const int half = lane / 32;
    auto multiply = [&](int b) {
#pragma unroll
        for (int k = 0; k < kDepth / 32; ++k) {
            v4i a[kFC], x[kFT];
#pragma unroll
            for (int i = 0; i < kFC; ++i)
                a[i] = *reinterpret_cast<const v4i*>(
                    &staged[b][(row_c + i * 32) * kDepth + ((2 * k + half) ^ (row_c % 8)) * 16]);
#pragma unroll
            for (int j = 0; j < kFT; ++j)
                x[j] = *reinterpret_cast<const v4i*>(
                    &staged[b][(row_t + j * 32) * kDepth + ((2 * k + half) ^ (row_t % 8)) * 16]);
#pragma unroll
            for (int i = 0; i < kFC; ++i)
#pragma unroll
                for (int j = 0; j < kFT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[i], x[j], acc[i][j], 0, 0, 0);
        }
    };

    const int steps = (p.depth + kDepth - 1) / kDepth;
    fetch(0, 0);
    arrive(0);
    __syncthreads();
    for (int s = 0; s < steps; s += 2) {
        if (s + 1 < steps) fetch(1, s + 1);
        multiply(0);
        if (s + 1 < steps) arrive(1);
        __syncthreads();
        if (s + 1 >= steps) break;
        if (s + 2 < steps) fetch(0, s + 2);
        multiply(1);
        if (s + 2 < steps) arrive(0);
        __syncthreads();
    }

#pragma unroll
    for (int j = 0; j < kFT; ++j) {
        const int64_t row = t.row0 + wt * kFT * 32 + j * 32 + lane % 32;
        if (row >= t.row_end) continue;
        const float sx = p.x_scale[kExperts ? token_of(p, row) : row];
        const float* sw = p.w_scale + (int64_t)t.expert * p.channels;
#pragma unroll
        for (int i = 0; i < kFC; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int channel = channel0 + wc * kFC * 32 + i * 32 + 8 * g + 4 * half;
                if (channel >= p.channels) continue;
                float f[4];
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    f[v] = (float)acc[i][j][4 * g + v] * sx *
                           sw[min(channel + v, p.channels - 1)];
                store4(p, row, channel, f);
            }
    }
}

template <int kRows, int kChannels, int kWT, int kWC>
hipError_t launch_tiles(const Int8Product& p, bool direct, hipStream_t stream)
{
    const int channel_tiles = (p.channels + kChannels - 1) / kChannels;
    // Every expert (and the dropped rows) may end in a tile that is not full.
    const int64_t row_tiles = p.experts ? min(p.rows, p.rows / kRows + p.experts + 1)
                                        : (p.rows + kRows - 1) / kRows;
    const int64_t wgs = row_tiles * channel_tiles;
    if (wgs > INT32_MAX) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)wgs), threads(kWT * kWC * kWave);
    if (p.experts) {
        if (direct)
            hipLaunchKernelGGL((int8_tile_kernel<kRows, kChannels, kWT, kWC, true, true>), grid,
                               threads, 0, stream, p, channel_tiles);
        else
            hipLaunchKernelGGL((int8_tile_kernel<kRows, kChannels, kWT, kWC, false, true>), grid,
                               threads, 0, stream, p, channel_tiles);
    } else {
        if (direct)
            hipLaunchKernelGGL((int8_tile_kernel<kRows, kChannels, kWT, kWC, true, false>), grid,
                               threads, 0, stream, p, channel_tiles);
        else
            hipLaunchKernelGGL((int8_tile_kernel<kRows, kChannels, kWT, kWC, false, false>), grid,
                               threads, 0, stream, p, channel_tiles);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_product(const Int8Product& p, int cus, hipStream_t stream)
{
    const bool direct = p.depth % 16 == 0 && p.ldx % 16 == 0 && p.ldw % 16 == 0 &&
                        p.w_stride % 16 == 0 && reinterpret_cast<uintptr_t>(p.x) % 16 == 0 &&
                        reinterpret_cast<uintptr_t>(p.w) % 16 == 0;
    (void)cus;
    return launch_tiles<128, 128, 2, 2>(p, direct, stream);
}

}  // namespace iqk
