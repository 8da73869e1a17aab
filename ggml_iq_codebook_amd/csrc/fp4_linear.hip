// fp4_linear.hip -- products with 4-bit weights whose groups of 32 share a power
// of two, dense or with a weight per expert:
//   y[t][n] = sum_k x[t][k] * value(w[n][k]).
//
// The weight's values are exact in bf16, so the matrix cores take them as they
// are.  bf16 activations are an operand as they come; fp16 ones are split into
// two bf16 parts and fp32 ones into three (v = hi + mid + lo exactly), each
// multiplied in turn, so every product is exact and only the fp32 sums and the
// one rounding of the result differ from the formula.  (The parts of fp32 values
// below 2^-110 reach below bf16's smallest number, 2^-133, and are cut there.)
#include <hip/hip_runtime.h>

#include <algorithm>

#include "expert_tiles.hpp"
#include "fp4_common.hpp"
#include "layers_launch.hpp"

namespace iqk {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kPiece = 128;           // depth of a step: four groups, 64 bytes of codes a row

__device__ __forceinline__ v4f mfma16(v8bf a, v8bf b, v4f c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// bf16 parts that a type is split into.
template <int kDT>
constexpr int kSplit = kDT == IQ_DTYPE_BF16 ? 1 : (kDT == IQ_DTYPE_F16 ? 2 : 3);

// 8 activations as operands.  hi is v cut to 8 significant bits, mid what is
// left cut likewise, lo the rest; of a NaN or an infinity hi is all.
template <int kDT>
__device__ __forceinline__ void split_values(const typename Value<kDT>::raw (&r)[8],
                                             v8bf (&part)[kSplit<kDT>])
{
    if constexpr (kDT == IQ_DTYPE_BF16) {
        part[0] = __builtin_bit_cast(v8bf, r);
    } else {
        constexpr int kN = kSplit<kDT>;
        uint32_t u[kN][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float left = Value<kDT>::load(r[i]);
            const uint32_t bits = __float_as_uint(left);
            const bool finite = (bits & 0x7f800000u) != 0x7f800000u;
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                u[k][i] = __float_as_uint(left) & 0xffff0000u;
                left = left - __uint_as_float(u[k][i]);
            }
            if (!finite) {
                u[0][i] |= bits & 0xffffu ? 0x400000u : 0u;
#pragma unroll
                for (int k = 1; k < kN; ++k) u[k][i] = 0u;
            }
        }
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = (u[k][2 * i] >> 16) | u[k][2 * i + 1];
            part[k] = __builtin_bit_cast(v8bf, w);
        }
    }
}

// kN consecutive channels of one row of y, in its type.
template <int kDT>
__device__ __forceinline__ void store_channels(const Fp4Product& p, int64_t row, int channel, v4f f)
{
    typedef typename Value<kDT>::raw raw;
    raw* to = static_cast<raw*>(p.y) + row * p.ldy + channel;
    raw v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = Value<kDT>::store(f[i]);
    if (channel + 4 <= p.channels) {
        __builtin_memcpy(to, v, sizeof(v));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (channel + i < p.channels) to[i] = v[i];
    }
}

template <int kDT, int kRows, int kChannels, int kThreads>
__device__ __forceinline__ void store_zeros(const Fp4Product& p, const Tile& t)
{
    for (int i = threadIdx.x; i < kRows * (kChannels / 4); i += kThreads) {
        const int64_t row = t.row0 + i / (kChannels / 4);
        const int channel = t.channel_tile * kChannels + i % (kChannels / 4) * 4;
        if (row < t.row_end && channel < p.channels)
            store_channels<kDT>(p, row, channel, v4f{0.0f, 0.0f, 0.0f, 0.0f});
    }
}

// Few rows: a workgroup takes 16 kFC channels of 16 kFT rows and its waves share
// the depth, so both operands go straight into registers and nothing waits for
// another wave until the sums are added at the end.  Lane l has row l % 16 of
// both operands and group l / 16 of a step: 16 bytes of codes and 32 activations.
template <int kDT, int kFC, int kFT, int kWaves, bool kExperts>
__global__ __launch_bounds__(kWaves* kWave) void fp4_rows_kernel(Fp4Product p, int channel_tiles)
{
    typedef typename Value<kDT>::raw raw;
    constexpr int kN = kSplit<kDT>;
    __shared__ __align__(16) v4f sums[kWaves - 1][kFC * kFT][kWave];
    const Tile t = kExperts ? expert_tile<16 * kFT>(p, channel_tiles)
                            : dense_tile<16 * kFT>(p, channel_tiles);
    if (t.expert == -2) return;
    if (t.expert == -1) {
        store_zeros<kDT, 16 * kFT, 16 * kFC, kWaves * kWave>(p, t);
        return;
    }
    const int lane = threadIdx.x % kWave, quarter = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int channel0 = t.channel_tile * 16 * kFC;

    const uint8_t *w[kFC], *scale[kFC];
#pragma unroll
    for (int i = 0; i < kFC; ++i) {
        const int64_t n = min(channel0 + 16 * i + lane % 16, p.channels - 1);
        w[i] = p.w + t.expert * p.w_stride + n * p.ldw + 16 * quarter;
        scale[i] = p.scale + t.expert * p.s_stride + n * p.lds;
    }
    const raw* x[kFT];
    bool live[kFT];
#pragma unroll
    for (int j = 0; j < kFT; ++j) {
        const int64_t row = t.row0 + 16 * j + lane % 16;
        live[j] = row < t.row_end;
        const int64_t token = live[j] ? (kExperts ? token_of(p, row) : row) : 0;
        x[j] = static_cast<const raw*>(p.x) + token * p.ldx + kGroup * quarter;
    }

    const int groups = p.depth / kGroup;
    const int steps = (groups + 3) / 4;
    const int first = (int)((int64_t)steps * wave / kWaves);
    const int last = (int)((int64_t)steps * (wave + 1) / kWaves);
    v4f acc[kFC][kFT] = {};
    for (int s = first; s < last; ++s) {
        const int group = 4 * s + quarter;
        const bool there = group < groups;
        uint4 codes[kFC];
        float power[kFC];
#pragma unroll
        for (int i = 0; i < kFC; ++i) {
            codes[i] = make_uint4(0u, 0u, 0u, 0u);
            if (there) __builtin_memcpy(&codes[i], w[i] + (int64_t)s * (kPiece / 2), 16);
            power[i] = group_scale(scale[i][min(group, groups - 1)]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v8bf b[kFT][kN];
#pragma unroll
            for (int j = 0; j < kFT; ++j) {
                raw r[8] = {};
                if (there && live[j])
                    __builtin_memcpy(r, x[j] + (int64_t)s * kPiece + 8 * k, sizeof(r));
                split_values<kDT>(r, b[j]);
            }
#pragma unroll
            for (int i = 0; i < kFC; ++i) {
                const uint32_t word = k == 0 ? codes[i].x : k == 1 ? codes[i].y
                                    : k == 2 ? codes[i].z : codes[i].w;
                const v8bf a = values_of(word, power[i]);
#pragma unroll
                for (int j = 0; j < kFT; ++j)
#pragma unroll
                    for (int q = kN - 1; q >= 0; --q) acc[i][j] = mfma16(a, b[j][q], acc[i][j]);
            }
        }
    }
    if (wave) {
#pragma unroll
        for (int i = 0; i < kFC; ++i)
#pragma unroll
            for (int j = 0; j < kFT; ++j) sums[wave - 1][i * kFT + j][lane] = acc[i][j];
    }
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int i = 0; i < kFC; ++i)
#pragma unroll
        for (int j = 0; j < kFT; ++j) {
            v4f sum = acc[i][j];
#pragma unroll
            for (int v = 0; v < kWaves - 1; ++v) sum += sums[v][i * kFT + j][lane];
            const int64_t row = t.row0 + 16 * j + lane % 16;
            const int channel = channel0 + 16 * i + 4 * quarter;
            if (row < t.row_end && channel < p.channels) store_channels<kDT>(p, row, channel, sum);
        }
}

// Every expert (and the dropped rows) may end in a tile that is not full.
int64_t workgroups(const Fp4Product& p, int rows, int channel_tiles)
{
    const int64_t row_tiles = p.experts ? std::min(p.rows, p.rows / rows + p.experts + 1)
                                        : (p.rows + rows - 1) / rows;
    return row_tiles * channel_tiles;
}

template <int kDT, int kFC, int kFT, int kWaves, bool kExperts>
hipError_t launch_rows(const Fp4Product& p, hipStream_t stream)
{
    const int channel_tiles = (p.channels + 16 * kFC - 1) / (16 * kFC);
    Fp4Product part = p;
    return in_parts(workgroups(p, 16 * kFT, channel_tiles), kWaves * kWave,
                    [&](int64_t first, dim3 wgs) {
        part.first_tile = first;
        hipLaunchKernelGGL((fp4_rows_kernel<kDT, kFC, kFT, kWaves, kExperts>), wgs,
                           dim3(kWaves * kWave), 0, stream, part, channel_tiles);
        return hipGetLastError();
    });
}

}  // namespace

int64_t fp4_workspace(int dtype, const void* x, int64_t ldx, int64_t tokens, int64_t rows,
                      int experts, int64_t channels, int64_t depth)
{
    return 0;
}

hipError_t launch_fp4_product(const Fp4Product& p, void* workspace, int cus, hipStream_t stream)
{
    return with_dtype(p.dtype, [&](auto dt) {
        constexpr int kDT = decltype(dt)::value;
        return p.experts ? launch_rows<kDT, 1, 1, 8, true>(p, stream)
                         : launch_rows<kDT, 1, 1, 8, false>(p, stream);
    });
}

}  // namespace iqk
