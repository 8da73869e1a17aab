// int8_matmul.hip -- products in 8-bit integers on the matrix cores, with a
// scale per token and per output channel, dense or with a weight per expert:
//   y[t][n] = (float)(sum_i x[t][i] * w[n][i]) * x_scale[t] * w_scale[n].
//
// The sums are exact in 32-bit integers, so neither tiling nor the order of the
// depth changes a result.  Both operands hold their depth innermost, which is
// how the matrix instructions take it: lane l of v_mfma_i32_16x16x64_i8
// supplies row l%16, depth 16*(l/16)..+15, as one 16-byte register group.
// The weight is the first operand, so a lane's results are 4 consecutive
// channels of one token and go out as one store.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "int8_tiles.hpp"
#include "iq_layers.h"
#include "layers_common.hpp"
#include "layers_launch.hpp"

namespace iqk {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

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
template <int kRows>
__device__ __forceinline__ Tile expert_tile(const Int8Product& p, int channel_tiles)
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
__device__ __forceinline__ int64_t token_of(const Int8Product& p, int64_t r)
{
    if (!p.order) return r;
    const int64_t t = (uint32_t)p.order[r] / (uint32_t)p.top_k;
    return min(t, p.tokens - 1);
}

// ---------------------------------------------------------------------------
// Writing results
// ---------------------------------------------------------------------------

// kN consecutive channels of one row of y, in its type.
template <int kDT, int kN>
__device__ __forceinline__ void store_channels(const Int8Product& p, int64_t row, int channel,
                                               const float (&f)[kN])
{
    typedef typename Value<kDT>::raw raw;
    raw* to = static_cast<raw*>(p.y) + row * p.ldy + channel;
    raw v[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = Value<kDT>::store(f[i]);
    if (channel + kN <= p.channels) {
        __builtin_memcpy(to, v, sizeof(v));
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i)
            if (channel + i < p.channels) to[i] = v[i];
    }
}

// The dropped rows of a tile: zeros are zeros in every type.
template <int kRows, int kChannels, int kThreads>
__device__ __forceinline__ void store_zeros(const Int8Product& p, const Tile& t)
{
    const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = threadIdx.x; i < kRows * (kChannels / 4); i += kThreads) {
        const int64_t row = t.row0 + i / (kChannels / 4);
        const int channel = t.channel_tile * kChannels + i % (kChannels / 4) * 4;
        if (row >= t.row_end || channel >= p.channels) continue;
        if (p.out_dtype == IQ_DTYPE_F32)
            store_channels<IQ_DTYPE_F32>(p, row, channel, zero);
        else
            store_channels<IQ_DTYPE_F16>(p, row, channel, zero);
    }
}

// ---------------------------------------------------------------------------
// The tile kernel
// ---------------------------------------------------------------------------

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) void global_void;

// 16 bytes a lane from global memory into LDS at `to` + 16 * lane.
__device__ __forceinline__ void copy_to_lds(const int8_t* from, int8_t* to)
{
    __builtin_amdgcn_global_load_lds((global_void*)(uintptr_t)from, (lds_void*)to, 16, 0, 0);
}

// 16 bytes at any alignment.
__device__ __forceinline__ uint4 load16(const int8_t* from)
{
    uint4 v;
    __builtin_memcpy(&v, from, 16);
    return v;
}

// 16 bytes of a row from depth `at`, zeros beyond its end, at any alignment.
__device__ __forceinline__ uint4 load_codes(const int8_t* row, int at, int depth)
{
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (at + 16 <= depth) {
        v = load16(row + at);
    } else if (at < depth) {
        uint64_t u[2] = {0u, 0u};
#pragma unroll 1
        for (int i = 0; i < depth - at; ++i) {
            const uint64_t byte = (uint64_t)(uint8_t)row[at + i] << (8 * (i % 8));
            u[0] |= i < 8 ? byte : 0u;
            u[1] |= i < 8 ? 0u : byte;
        }
        v = make_uint4((uint32_t)u[0], (uint32_t)(u[0] >> 32), (uint32_t)u[1],
                       (uint32_t)(u[1] >> 32));
    }
    return v;
}

// A staged row of kDepth bytes is stored in pieces of 16, piece c in slot
// c ^ swizzle(row): eight lanes that read one piece of consecutive rows meet
// eight different groups of banks.
template <int kDepth>
__device__ __forceinline__ int swizzle(int row)
{
    return kDepth == 64 ? (row >> 1) & 3 : row & (kDepth / 16 - 1);
}

// Waits until at most kLeft of this wave's loads are under way and all its LDS
// reads have arrived, then for the other waves.
template <int kLeft>
__device__ __forceinline__ void wait_and_meet()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLeft) : "memory");
}

// kWT x kWC waves share a tile of kRows rows of y by kChannels channels, each
// a part of kRows/kWT by kChannels/kWC, in steps of kDepth of the depth.  On the
// two smallest tiles kWK waves share a part, each on its share of every step, and
// add their sums at the end.  The tiles of both operands go through a ring of
// buffers in LDS; what the depth leaves beyond whole steps has a buffer of its
// own, filled at the start.
//
// kDirect: rows start on 16 bytes, and pieces are copied straight into LDS,
// kStages - 1 steps ahead.  Otherwise they pass through registers, four steps
// ahead (two for the largest tile), into two buffers.
//
// kPingPong (8 waves, two on a SIMD): the second four waves run half a step
// behind, so on each SIMD one wave multiplies while the other reads its
// operands; a step is two barriers long.
//
// Results go through LDS too where a wave has 32 channels or more: written as
// the matrix instructions leave them, 4 channels a lane, and read back as
// whole rows of its channels, 16 bytes a lane, so that stores fill cache lines
// (4096^3 to bf16: 67 us; stored as they are left: 76).
//
// Measured, codes of activations with a few large channels: 16384 x 4096 x 4096
// 257 us (2140 TOP/s), 4096^3 62 us.  What bounds the large tiles is the card's
// power: the matrix instructions alone, on random codes and without memory,
// reach 3250 TOP/s (4480 on zeros), and this kernel takes 51 us for 4096^3 zeros.
// Ping-pong against waves that all wait, read and multiply together: 62 us
// against 74; v_mfma_i32_32x32x32_i8 in its place: 71.
// Small tiles are bound by the latency of their first loads and by what a compute
// unit loads from the L2 (about 38 bytes a clock), so small products take many
// small tiles: 24 x 1536 x 4096 in a graph 4.3 us with 16 x 16 tiles, 6.1 with
// 32 x 32.  Products by expert of few rows are bound by HBM (16 tokens, 2 of 16
// experts of 1536 x 4096: 95 MB read in 18 us, 5.3 TB/s).
template <int kRows, int kChannels, int kWT, int kWC, int kWK, int kDepth, int kStages,
          bool kPingPong, bool kDirect, bool kExperts>
__global__ __launch_bounds__(kWT* kWC* kWK* kWave, kWT* kWC* kWK / 4) void int8_tile_kernel(
    Int8Product p, int channel_tiles)
{
    constexpr int kWaves = kWT * kWC * kWK, kThreads = kWaves * kWave;
    constexpr int kFT = kRows / kWT / 16, kFC = kChannels / kWC / 16;
    constexpr int kPieces = kDepth / 16;
    constexpr int kRowsPerLoad = kWave / kPieces;
    constexpr int kLoads = (kRows + kChannels) / kRowsPerLoad / kWaves;   // a wave's
    constexpr int kBuffers = kDirect ? kStages : 2;
    static_assert(kLoads * kRowsPerLoad * kWaves == kRows + kChannels && kFT > 0 && kFC > 0, "tile");
    constexpr int kBytes = (kRows + kChannels) * kDepth;
    __shared__ __align__(1024) int8_t staged[kBuffers + 1][kBytes];

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
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int r = (wave * kLoads + i) * kRowsPerLoad + lane / kPieces;
        const int at = ((lane % kPieces) ^ swizzle<kDepth>(r)) * 16;
        if (r < kChannels) {
            from[i] = w + (int64_t)min(channel0 + r, p.channels - 1) * p.ldw + at;
        } else {
            const int64_t row = min(t.row0 + r - kChannels, t.row_end - 1);
            from[i] = p.x + (kExperts ? token_of(p, row) : row) * p.ldx + at;
        }
    }
    const int steps = p.depth / kDepth;
    const int rest = p.depth - steps * kDepth;
    // The rest of the depth: through registers, its end cut byte by byte.
    auto stage_rest = [&]() {
        if (rest == 0) return;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = (wave * kLoads + i) * kRowsPerLoad + lane / kPieces;
            const int at = ((lane % kPieces) ^ swizzle<kDepth>(r)) * 16;
            *reinterpret_cast<uint4*>(&staged[kBuffers][(wave * kLoads + i) * 1024 + lane * 16]) =
                load_codes(from[i] + (int64_t)steps * kDepth - at, at, rest);
        }
    };

    v4i acc[kFC][kFT] = {};
    const int wt = wave % kWT, wc = wave / kWT % kWC, wk = wave / (kWT * kWC);
    const int quarter = lane / 16;
    const int row_c = wc * kFC * 16 + lane % 16;
    const int row_t = kChannels + wt * kFT * 16 + lane % 16;
    // A step's parts of 64 that are this wave's: wk, wk + kWK, ...
    constexpr int kParts = kDepth / 64 / kWK;
    static_assert(kParts > 0 && (kWK == 1 || kFC == 1), "waves that share a part");
    auto read = [&](int b, int k, v4i (&a)[kFC], v4i (&x)[kFT]) {
        const int piece = 4 * (kWK * k + wk) + quarter;
#pragma unroll
        for (int i = 0; i < kFC; ++i)
            a[i] = *reinterpret_cast<const v4i*>(
                &staged[b][(row_c + i * 16) * kDepth + (piece ^ swizzle<kDepth>(row_c)) * 16]);
#pragma unroll
        for (int j = 0; j < kFT; ++j)
            x[j] = *reinterpret_cast<const v4i*>(
                &staged[b][(row_t + j * 16) * kDepth + (piece ^ swizzle<kDepth>(row_t)) * 16]);
    };
    auto multiply = [&](const v4i (&a)[kFC], const v4i (&x)[kFT]) {
#pragma unroll
        for (int i = 0; i < kFC; ++i)
#pragma unroll
            for (int j = 0; j < kFT; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], x[j], acc[i][j], 0, 0, 0);
    };

    if constexpr (kDirect) {
        // Where a weight is read once, each channel tile begins at a step of its
        // own and ends with those before it: rows that are a power of two apart
        // share HBM channels, and tiles that go through the depth together meet
        // there (16 tokens, 2 of 8 experts of 2048 x 4096: 20 us, so 16).  Large
        // tiles share the tokens' L2 lines by going together (58 us so, 55).
        const int shift = (kExperts ? kRows <= 128 : p.rows <= kRows) && steps
                              ? t.channel_tile * 7 % steps : 0;
        auto fetch = [&](int b, int step) {
            step += step + shift < steps ? shift : shift - steps;
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                copy_to_lds(from[i] + (int64_t)step * kDepth,
                            &staged[b][(wave * kLoads + i) * 1024]);
        };
        constexpr int kLeft = (kStages - 2) * kLoads;
        static_assert(kLeft < 64, "vmcnt holds 6 bits");
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i)
            if (i < steps) fetch(i, i);
        stage_rest();
        if constexpr (kPingPong) {
            const bool late = wave >= kWaves / 2;
            if (steps >= kStages - 1)
                wait_and_meet<kLeft>();
            else
                wait_and_meet<0>();
            if (late) asm volatile("s_barrier" ::: "memory");
            for (int s0 = 0; s0 < steps; s0 += kStages) {
#pragma unroll
                for (int u = 0; u < kStages; ++u) {
                    const int s = s0 + u;
                    if (s >= steps) break;
                    v4i a[kParts][kFC], x[kParts][kFT];
#pragma unroll
                    for (int k = 0; k < kParts; ++k) read(u, k, a[k], x[k]);
                    // Into the buffer of step s - 1, which both halves read before
                    // the last barrier.  Step s + 1 has to be there for the next.
                    if (s + kStages - 1 < steps) {
                        fetch((u + kStages - 1) % kStages, s + kStages - 1);
                        wait_and_meet<kLeft>();
                    } else {
                        wait_and_meet<0>();
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    __builtin_amdgcn_s_setprio(1);
#pragma unroll
                    for (int k = 0; k < kParts; ++k) multiply(a[k], x[k]);
                    __builtin_amdgcn_s_setprio(0);
                    __builtin_amdgcn_sched_barrier(0);
                    asm volatile("s_barrier" ::: "memory");
                }
            }
            if (!late) asm volatile("s_barrier" ::: "memory");
        } else {
            for (int s0 = 0; s0 < steps; s0 += kStages) {
#pragma unroll
                for (int u = 0; u < kStages; ++u) {
                    const int s = s0 + u;
                    if (s >= steps) break;
                    if (s + kStages - 2 < steps)
                        wait_and_meet<kLeft>();
                    else
                        wait_and_meet<0>();
                    if (s + kStages - 1 < steps)
                        fetch((u + kStages - 1) % kStages, s + kStages - 1);
#pragma unroll
                    for (int k = 0; k < kParts; ++k) {
                        v4i a[kFC], x[kFT];
                        read(u, k, a, x);
                        multiply(a, x);
                    }
                }
            }
        }
    } else {
        // As far ahead as the registers go.
        constexpr int kAhead = kRows * kChannels > 128 * 128 ? 2 : 4;
        uint4 passing[kAhead][kLoads];
        auto fetch = [&](int set, int step) {
            // Beyond the last step the last one again: not used.
            const int64_t at = (int64_t)min(step, max(steps - 1, 0)) * kDepth;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) passing[set][i] = load16(from[i] + at);
        };
        if (steps > 0) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) fetch(i, i);
        }
        stage_rest();
        for (int s0 = 0; s0 < steps; s0 += kAhead) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int s = s0 + u;
                if (s >= steps) break;
                // This buffer was last read in step s - 2, before the last barrier.
#pragma unroll
                for (int i = 0; i < kLoads; ++i)
                    *reinterpret_cast<uint4*>(
                        &staged[u % 2][(wave * kLoads + i) * 1024 + lane * 16]) = passing[u][i];
                asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                fetch(u, s + kAhead);
#pragma unroll
                for (int k = 0; k < kParts; ++k) {
                    v4i a[kFC], x[kFT];
                    read(u % 2, k, a, x);
                    multiply(a, x);
                }
            }
        }
    }
    if (rest) {
        wait_and_meet<0>();
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
            v4i a[kFC], x[kFT];
            read(kBuffers, k, a, x);
            multiply(a, x);
        }
    }

    if constexpr (kWK > 1) {
        wait_and_meet<0>();
        v4i* sums = reinterpret_cast<v4i*>(&staged[0][0]) + (wave % (kWT * kWC)) * kFT * kWave + lane;
        constexpr int kNext = kWT * kWC * kFT * kWave;
        if (wk) {
#pragma unroll
            for (int j = 0; j < kFT; ++j) sums[(wk - 1) * kNext + j * kWave] = acc[0][j];
        }
        wait_and_meet<0>();
        if (wk) return;
#pragma unroll
        for (int k = 0; k < kWK - 1; ++k)
#pragma unroll
            for (int j = 0; j < kFT; ++j) acc[0][j] += sums[k * kNext + j * kWave];
    }
    const int wave_channel = channel0 + wc * kFC * 16;
    const float* sw = p.w_scale + (int64_t)t.expert * p.channels;
    float scale[kFC][4];
#pragma unroll
    for (int i = 0; i < kFC; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v)
            scale[i][v] = sw[min(wave_channel + i * 16 + 4 * quarter + v, p.channels - 1)];
    // Every wave is done with the staged tiles.
    if (kFC > 1) wait_and_meet<0>();
    auto write = [&](auto dt) {
        constexpr int kDT = decltype(dt)::value;
        typedef typename Value<kDT>::raw raw;
        constexpr int kN = 16 / (int)sizeof(raw);
        // A row of the wave's channels, and some more so that rows start on
        // different banks.
        constexpr int kRow = kFC * 16 + kN;
        constexpr int kLanes = kFC * 16 / kN;             // lanes to a row
        static_assert(kFC == 1 || kWaves * 16 * kRow * (int)sizeof(raw) <= (kBuffers + 1) * kBytes,
                      "results fit the staged tiles");
        raw* mine = reinterpret_cast<raw*>(&staged[0][0]) + wave * 16 * kRow;
#pragma unroll
        for (int j = 0; j < kFT; ++j) {
            const int64_t row0 = t.row0 + (wt * kFT + j) * 16;
            const int64_t row = min(row0 + lane % 16, t.row_end - 1);
            const float sx = p.x_scale[kExperts ? token_of(p, row) : row];
#pragma unroll
            for (int i = 0; i < kFC; ++i) {
                float f[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) f[v] = (float)acc[i][j][v] * sx * scale[i][v];
                if constexpr (kFC == 1) {
                    const int channel = wave_channel + 4 * quarter;
                    if (row0 + lane % 16 < t.row_end && channel < p.channels)
                        store_channels<kDT>(p, row, channel, f);
                } else {
                    raw o[4];
#pragma unroll
                    for (int v = 0; v < 4; ++v) o[v] = Value<kDT>::store(f[v]);
                    __builtin_memcpy(__builtin_assume_aligned(
                                         mine + lane % 16 * kRow + i * 16 + 4 * quarter, 4 * sizeof(raw)),
                                     o, sizeof(o));
                }
            }
            if constexpr (kFC > 1) {
                // A wave's own LDS accesses are done in order.
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int s = 0; s < 16 * kLanes / kWave; ++s) {
                    const int r = (s * kWave + lane) / kLanes, c = (s * kWave + lane) % kLanes * kN;
                    raw o[kN];
                    __builtin_memcpy(o, __builtin_assume_aligned(mine + r * kRow + c, 16), 16);
                    const int channel = wave_channel + c;
                    if (row0 + r >= t.row_end || channel >= p.channels) continue;
                    raw* to = static_cast<raw*>(p.y) + (row0 + r) * p.ldy + channel;
                    if (channel + kN <= p.channels) {
                        __builtin_memcpy(to, o, 16);
                    } else {
#pragma unroll
                        for (int v = 0; v < kN; ++v)
                            if (channel + v < p.channels) to[v] = o[v];
                    }
                }
                __builtin_amdgcn_wave_barrier();
            }
        }
    };
    if (p.out_dtype == IQ_DTYPE_BF16)
        write(Int<IQ_DTYPE_BF16>());
    else if (p.out_dtype == IQ_DTYPE_F16)
        write(Int<IQ_DTYPE_F16>());
    else
        write(Int<IQ_DTYPE_F32>());
}

// Every expert (and the dropped rows) may end in a tile that is not full.
int64_t workgroups(const Int8Product& p, int rows, int channel_tiles)
{
    const int64_t row_tiles = p.experts ? std::min(p.rows, p.rows / rows + p.experts + 1)
                                        : (p.rows + rows - 1) / rows;
    return row_tiles * channel_tiles;
}

template <int kRows, int kChannels, int kWT, int kWC, int kWK, int kDepth, int kStages,
          bool kPingPong, bool kDirect, bool kExperts>
hipError_t launch_tiles(const Int8Product& p, hipStream_t stream)
{
    const int channel_tiles = (p.channels + kChannels - 1) / kChannels;
    constexpr int kThreads = kWT * kWC * kWK * kWave;
    Int8Product part = p;
    return in_parts(workgroups(p, kRows, channel_tiles), kThreads, [&](int64_t first, dim3 wgs) {
        part.first_tile = first;
        hipLaunchKernelGGL((int8_tile_kernel<kRows, kChannels, kWT, kWC, kWK, kDepth, kStages,
                                             kPingPong, kDirect, kExperts>),
                           wgs, dim3(kThreads), 0, stream, part, channel_tiles);
        return hipGetLastError();
    });
}

// The tile for a product, as rows * 1000 + channels.
template <int kN>
int choose_tile(const Int8Product& p, int cus, const TileTime (&tiles)[kN])
{
    const TileTime& t = tiles[fastest_tile(p.rows, p.channels, p.depth, p.experts, cus, tiles)];
    return t.rows * 1000 + t.channels;
}

template <bool kExperts>
hipError_t launch_unaligned(const Int8Product& p, int cus, hipStream_t stream)
{
    switch (choose_tile(p, cus, kUnaligned)) {
    case 16016: return launch_tiles<16, 16, 1, 1, 4, 256, 2, false, false, kExperts>(p, stream);
    case 32032: return launch_tiles<32, 32, 2, 2, 2, 256, 2, false, false, kExperts>(p, stream);
    case 64064: return launch_tiles<64, 64, 4, 2, 1, 128, 2, false, false, kExperts>(p, stream);
    case 128128: return launch_tiles<128, 128, 4, 4, 1, 128, 2, false, false, kExperts>(p, stream);
    default: return launch_tiles<128, 256, 2, 4, 1, 64, 2, false, false, kExperts>(p, stream);
    }
}

// The tiles that both kinds of product take; `tile` as choose_tile gives it.
template <bool kExperts>
hipError_t launch_direct(int tile, const Int8Product& p, hipStream_t stream)
{
    switch (tile) {
    case 16016: return launch_tiles<16, 16, 1, 1, 4, 256, 4, false, true, kExperts>(p, stream);
    case 64128: return launch_tiles<64, 128, 2, 4, 1, 128, 4, true, true, kExperts>(p, stream);
    case 64192: return launch_tiles<64, 192, 4, 2, 1, 128, 4, true, true, kExperts>(p, stream);
    case 128128: return launch_tiles<128, 128, 4, 2, 1, 128, 4, true, true, kExperts>(p, stream);
    case 128192: return launch_tiles<128, 192, 4, 2, 1, 128, 3, true, true, kExperts>(p, stream);
    case 192192: return launch_tiles<192, 192, 4, 2, 1, 64, 4, true, true, kExperts>(p, stream);
    default: return launch_tiles<256, 256, 4, 2, 1, 64, 4, true, true, kExperts>(p, stream);
    }
}

}  // namespace

hipError_t launch_int8_product(const Int8Product& p, int cus, hipStream_t stream)
{
    const bool direct = (p.tokens == 1 || p.ldx % 16 == 0) &&
                        (p.channels == 1 || p.ldw % 16 == 0) &&
                        (p.experts <= 1 || p.w_stride % 16 == 0) &&
                        reinterpret_cast<uintptr_t>(p.x) % 16 == 0 &&
                        reinterpret_cast<uintptr_t>(p.w) % 16 == 0;
    if (!direct)
        return p.experts ? launch_unaligned<true>(p, cus, stream)
                         : launch_unaligned<false>(p, cus, stream);
    if (p.experts) {
        // Tiles of few rows, several workgroups to a compute unit: it is the
        // number of loads under way that counts on weights out of HBM.
        switch (const int tile = choose_tile(p, cus, kByExpert)) {
        case 32064: return launch_tiles<32, 64, 1, 4, 1, 128, 4, false, true, true>(p, stream);
        case 32128: return launch_tiles<32, 128, 1, 4, 1, 128, 3, false, true, true>(p, stream);
        case 64064: return launch_tiles<64, 64, 2, 2, 1, 128, 4, false, true, true>(p, stream);
        default: return launch_direct<true>(tile, p, stream);
        }
    }
    switch (const int tile = choose_tile(p, cus, kDense)) {
    case 32032: return launch_tiles<32, 32, 2, 2, 2, 256, 4, false, true, false>(p, stream);
    case 64064: return launch_tiles<64, 64, 4, 2, 1, 256, 4, true, true, false>(p, stream);
    case 192128: return launch_tiles<192, 128, 4, 2, 1, 128, 3, true, true, false>(p, stream);
    case 128256: return launch_tiles<128, 256, 2, 4, 1, 64, 4, true, true, false>(p, stream);
    default: return launch_direct<false>(tile, p, stream);
    }
}

}  // namespace iqk
