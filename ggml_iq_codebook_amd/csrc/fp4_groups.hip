// fp4_groups.hip -- rows rounded to 4-bit floats in groups of 32 that share a
// power of two, and read back.
//   m = max|x| over the group, s = clamp(floor(log2 m) - 2, -127, 127),
//   code = the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6 to |x| 2^-s, halves to the
//   even code, 6 beyond 6, with the sign of x.
// 2^s is a power of two, so x 2^-s is exact and the one rounding is the code's.
//
// Bound by HBM: 4096 x 4096 of fp32 13 us to codes and 15 back, 24576 x 4096 of bf16
// 57 and 37 (both ways 5.0 and 4.9 TB/s, a large copy 5.1).  A lane has four pieces of
// 8 values on the way, 16 bytes a load; rows without gaps are one row, so that no wave
// is partly empty.
#include <hip/hip_runtime.h>

#include "fp4_common.hpp"
#include "layers_launch.hpp"
#include "row_codes.hpp"

namespace iqk {
namespace {

constexpr int kThreads = 256;
constexpr int kParts = 4;             // pieces of 8 values that a lane has under way
constexpr int kPerWave = kWave * kChunk * kParts;

// A wave's row and its first value there.
struct Place {
    int64_t row, col;
};

__device__ __forceinline__ Place place_of(int64_t wave, int64_t per_row)
{
    const int64_t row = wave / per_row;
    return {row, (wave - row * per_row) * kPerWave};
}

// A quad has a group: 8 values a lane.
template <int kDT>
__global__ __launch_bounds__(kThreads) void quantize_groups_kernel(
    const void* __restrict__ x, int64_t ldx, int64_t rows, int64_t cols,
    uint8_t* __restrict__ codes, int64_t ldc, uint8_t* __restrict__ scales, int64_t lds,
    int64_t first, int64_t per_row, int32_t* status)
{
    typedef typename Value<kDT>::raw raw;
    const int lane = threadIdx.x % kWave;
    const int64_t wave = (first + blockIdx.x) * (kThreads / kWave) +
                         __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const Place p = place_of(wave, per_row);
    if (p.row >= rows) return;
    const raw* xr = static_cast<const raw*>(x) + p.row * ldx;
    Chunk<kDT, true> v[kParts];
#pragma unroll
    for (int i = 0; i < kParts; ++i) v[i].load(xr, p.col + (i * kWave + lane) * kChunk, cols);
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        const int64_t at = p.col + (i * kWave + lane) * kChunk;
        uint32_t top = v[i].top();
        top = max(top, (uint32_t)quad_xchg<kQuadXor1>((int)top));
        top = max(top, (uint32_t)quad_xchg<kQuadXor2>((int)top));
        // floor(log2 m) is the exponent field less 127; values below 2^-126 have
        // none and take the lowest scale, as all below 2^-124 do.
        const bool bad = top >= 0x7f800000u;
        const uint32_t byte = bad || top < (3u << 23) ? 0u : (top >> 23) - 2u;
        uint32_t word = 0u;
        if (!bad) {
            const float scale = group_scale(byte);
            word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[i][0], v[i][1], scale, 0);
            word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[i][2], v[i][3], scale, 1);
            word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[i][4], v[i][5], scale, 2);
            word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[i][6], v[i][7], scale, 3);
        }
        if (at < cols) {
            __builtin_memcpy(codes + p.row * ldc + at / 2, &word, 4);
            if (lane % 4 == 0) {
                scales[p.row * lds + at / kGroup] = (uint8_t)byte;
                if (bad) report_generic(status, IQ_ERR_NONFINITE);
            }
        }
    }
}

template <int kDT>
__global__ __launch_bounds__(kThreads) void dequantize_groups_kernel(
    const uint8_t* __restrict__ codes, int64_t ldc, const uint8_t* __restrict__ scales,
    int64_t lds, int64_t rows, int64_t cols, void* __restrict__ y, int64_t ldy, int64_t first,
    int64_t per_row)
{
    typedef typename Value<kDT>::raw raw;
    const int lane = threadIdx.x % kWave;
    const int64_t wave = (first + blockIdx.x) * (kThreads / kWave) +
                         __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const Place p = place_of(wave, per_row);
    if (p.row >= rows) return;
    uint32_t word[kParts], byte[kParts];
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        const int64_t at = p.col + (i * kWave + lane) * kChunk;
        word[i] = byte[i] = 0u;
        if (at < cols) {
            __builtin_memcpy(&word[i], codes + p.row * ldc + at / 2, 4);
            byte[i] = scales[p.row * lds + at / kGroup];
        }
    }
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        const int64_t at = p.col + (i * kWave + lane) * kChunk;
        const v8bf v = values_of(word[i], group_scale(byte[i]));
        raw out[kChunk];
#pragma unroll
        for (int j = 0; j < kChunk; ++j) out[j] = Value<kDT>::store((float)v[j]);
        if (at < cols) __builtin_memcpy(static_cast<raw*>(y) + p.row * ldy + at, out, sizeof(out));
    }
}

}  // namespace

hipError_t launch_quantize_groups(int dtype, const void* x, int64_t ldx, int64_t rows, int64_t cols,
                                  uint8_t* codes, int64_t ldc, uint8_t* scale, int64_t lds,
                                  int32_t* status, hipStream_t stream)
{
    if (ldx == cols && ldc == cols / 2 && lds == cols / kGroup) {
        cols *= rows;
        rows = 1;
    }
    const int64_t per_row = (cols + kPerWave - 1) / kPerWave;
    constexpr int kWaves = kThreads / kWave;
    return with_dtype(dtype, [&](auto dt) {
        constexpr int kDT = decltype(dt)::value;
        return in_parts((rows * per_row + kWaves - 1) / kWaves, kThreads,
                        [&](int64_t first, dim3 wgs) {
            hipLaunchKernelGGL(quantize_groups_kernel<kDT>, wgs, dim3(kThreads), 0, stream, x, ldx,
                               rows, cols, codes, ldc, scale, lds, first, per_row, status);
            return hipGetLastError();
        });
    });
}

hipError_t launch_dequantize_groups(const uint8_t* codes, int64_t ldc, const uint8_t* scale,
                                    int64_t lds, int64_t rows, int64_t cols, int dtype, void* y,
                                    int64_t ldy, hipStream_t stream)
{
    if (ldy == cols && ldc == cols / 2 && lds == cols / kGroup) {
        cols *= rows;
        rows = 1;
    }
    const int64_t per_row = (cols + kPerWave - 1) / kPerWave;
    constexpr int kWaves = kThreads / kWave;
    return with_dtype(dtype, [&](auto dt) {
        constexpr int kDT = decltype(dt)::value;
        return in_parts((rows * per_row + kWaves - 1) / kWaves, kThreads,
                        [&](int64_t first, dim3 wgs) {
            hipLaunchKernelGGL(dequantize_groups_kernel<kDT>, wgs, dim3(kThreads), 0, stream, codes,
                               ldc, scale, lds, rows, cols, y, ldy, first, per_row);
            return hipGetLastError();
        });
    });
}

}  // namespace iqk
