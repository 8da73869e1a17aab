// quantize_rows.hip -- rows rounded to 8-bit integers with a scale each:
// scale = max|x| * (1/127), q = round_half_even(x / scale), in fp32: the
// reciprocal and the product rounded to nearest, the division correctly rounded.
//
// Bound by HBM: a row is read once, kept in registers while its maximum is
// found, and written as one byte per value.  16384 bf16 rows of 4096: 38 us,
// 5.3 TB/s read and written together (a large copy: 5.1); 4096 rows: 11.5 us.
// A correctly rounded division for each value, in place of the reciprocal and
// its check, took 19 us for these 4096 rows.
#include <hip/hip_runtime.h>

#include "layers_launch.hpp"
#include "row_codes.hpp"

namespace iqk {
namespace {

constexpr int kThreads = 256;

template <int kDT, bool kWhole>
__device__ __forceinline__ void store_chunk(int8_t* row, int64_t at, int64_t cols,
                                            const Chunk<kDT, kWhole>& v, float scale, float inv)
{
    uint32_t b[kChunk / 4];
    codes_of(v, scale, inv, b);
    if (kWhole || at + kChunk <= cols) {
        __builtin_memcpy(row + at, b, kChunk);
    } else {
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
            if (at + i < cols) row[at + i] = (int8_t)(b[i / 4] >> (8 * (i % 4)));
    }
}

// kLanes lanes share a row (64: a wave; 256: the workgroup); each keeps kKeep
// chunks of it in registers, and rows longer than that are read again.
template <int kDT, int kLanes, int kKeep, bool kWhole>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(
    const void* __restrict__ x, int64_t ldx, int64_t rows, int64_t cols, int8_t* __restrict__ q,
    int64_t ldq, float* __restrict__ scales, int32_t* status)
{
    typedef typename Value<kDT>::raw raw;
    __shared__ uint32_t tops[kThreads / kWave];
    const int lane = threadIdx.x % kLanes;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    // Rows beyond the last only occur where a row is a wave's: no barrier then.
    if (row >= rows) return;
    const raw* xr = static_cast<const raw*>(x) + row * ldx;
    int8_t* qr = q + row * ldq;

    Chunk<kDT, kWhole> kept[kKeep];
    uint32_t top = 0u;
#pragma unroll
    for (int c = 0; c < kKeep; ++c) kept[c].load(xr, (c * kLanes + lane) * kChunk, cols);
#pragma unroll
    for (int c = 0; c < kKeep; ++c) top = max(top, kept[c].top());
    constexpr int64_t kKept = (int64_t)kKeep * kLanes * kChunk;
    for (int64_t at = kKept + lane * kChunk; at < cols; at += kLanes * kChunk) {
        Chunk<kDT, kWhole> u;
        u.load(xr, at, cols);
        top = max(top, u.top());
    }
#pragma unroll
    for (int d = kWave / 2; d; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    if (kLanes > kWave) {
        if (threadIdx.x % kWave == 0) tops[threadIdx.x / kWave] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kThreads / kWave; ++i) top = max(top, tops[i]);
    }

    const float scale = row_scale(top);
    if (lane == 0) {
        scales[row] = scale;
        if (top >= 0x7f800000u) report_generic(status, IQ_ERR_NONFINITE);
    }
    if (!(scale > 0.0f)) {
        // A row of zeros, or one that is refused.
        for (int64_t at = lane; at < cols; at += kLanes) qr[at] = 0;
        return;
    }
    const float inv = 1.0f / scale;
#pragma unroll
    for (int c = 0; c < kKeep; ++c) {
        const int64_t at = (c * kLanes + lane) * kChunk;
        if (at < cols) store_chunk(qr, at, cols, kept[c], scale, inv);
    }
    for (int64_t at = kKept + lane * kChunk; at < cols; at += kLanes * kChunk) {
        Chunk<kDT, kWhole> u;
        u.load(xr, at, cols);
        store_chunk(qr, at, cols, u, scale, inv);
    }
}

template <int kDT, int kLanes, int kKeep>
hipError_t launch(const void* x, int64_t ldx, int64_t rows, int64_t cols, int8_t* q, int64_t ldq,
                  float* scale, int32_t* status, hipStream_t stream)
{
    constexpr int kRows = kThreads / kLanes;
    const auto kernel = cols % kChunk == 0 ? quantize_rows_kernel<kDT, kLanes, kKeep, true>
                                           : quantize_rows_kernel<kDT, kLanes, kKeep, false>;
    return in_parts((rows + kRows - 1) / kRows, kThreads, [&](int64_t first, dim3 wgs) {
        const int64_t row = first * kRows;
        hipLaunchKernelGGL(kernel, wgs, dim3(kThreads), 0, stream,
                           static_cast<const typename Value<kDT>::raw*>(x) + row * ldx, ldx,
                           rows - row, cols, q + row * ldq, ldq, scale + row, status);
        return hipGetLastError();
    });
}

}  // namespace

// A wave per row up to 4096 values (8 chunks of 8 a lane: no barrier) where
// there are rows enough to hide a wave's latency; the workgroup where rows are
// longer or fewer.  bf16 rows of 4096, by waves and by workgroups: 1024 rows
// 7.2 and 6.9 us, 4096 rows 15.7 and 11.5 us, 16384 rows 37.7 and 40.9 us.
hipError_t launch_quantize_rows(int dtype, const void* x, int64_t ldx, int64_t rows, int64_t cols,
                                int8_t* q, int64_t ldq, float* scale, int32_t* status,
                                hipStream_t stream)
{
    return with_dtype(dtype, [&](auto dt) {
        constexpr int kDT = decltype(dt)::value;
        if (cols <= 1024)
            return launch<kDT, 64, 2>(x, ldx, rows, cols, q, ldq, scale, status, stream);
        if (cols <= 4096 && rows > 8192)
            return launch<kDT, 64, 8>(x, ldx, rows, cols, q, ldq, scale, status, stream);
        if (cols <= 4096)
            return launch<kDT, 256, 2>(x, ldx, rows, cols, q, ldq, scale, status, stream);
        return launch<kDT, 256, 4>(x, ldx, rows, cols, q, ldq, scale, status, stream);
    });
}

}  // namespace iqk
