// quantize_rows.hip -- rows rounded to 8-bit integers with a scale each:
// scale = max|x| * (1/127), q = round_half_even(x / scale), in fp32: the
// reciprocal and the product rounded to nearest, the division correctly rounded.
//
// Bound by HBM: a row is read once, kept in registers while its maximum is
// found, and written as one byte per value.  The maximum is taken over the
// bits of |x| as integers, which also orders infinities and NaN above every
// finite value, so one comparison finds a row that has to be refused.
#include <hip/hip_runtime.h>

#include "layers_common.hpp"
#include "layers_launch.hpp"

namespace iqk {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8;             // values a lane reads and writes at once

template <int kDT>
__device__ __forceinline__ uint32_t load_chunk(const typename Value<kDT>::raw* row, int64_t at,
                                               int64_t cols, float (&v)[kChunk])
{
    typedef typename Value<kDT>::raw raw;
    Pack<raw, kChunk> p;
    if (at + kChunk <= cols) {
        p.load(row + at);
    } else {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) p.v[i] = at + i < cols ? row[at + i] : raw(0);
    }
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
        v[i] = Value<kDT>::load(p.v[i]);
        top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    }
    return top;
}

__device__ __forceinline__ void store_chunk(int8_t* row, int64_t at, int64_t cols,
                                            const float (&v)[kChunk], float scale)
{
    Pack<int8_t, kChunk> q;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
        // |x| / scale rounds to 127 at most, but for scales among the smallest
        // subnormals, whose own rounding is coarse.
        const float r = scale > 0.0f ? rintf(v[i] / scale) : 0.0f;
        q.v[i] = (int8_t)fminf(fmaxf(r, -127.0f), 127.0f);
    }
    if (at + kChunk <= cols) {
        q.store(row + at);
    } else {
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
            if (at + i < cols) row[at + i] = q.v[i];
    }
}

// kLanes lanes share a row (64: a wave; 256: the workgroup); each keeps kKeep
// chunks of it in registers, and rows longer than that are read again.
template <int kDT, int kLanes, int kKeep>
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

    float v[kKeep][kChunk];
    uint32_t top = 0u;
#pragma unroll
    for (int c = 0; c < kKeep; ++c)
        top = max(top, load_chunk<kDT>(xr, ((int64_t)c * kLanes + lane) * kChunk, cols, v[c]));
    constexpr int64_t kKept = (int64_t)kKeep * kLanes * kChunk;
    for (int64_t at = kKept + lane * kChunk; at < cols; at += kLanes * kChunk) {
        float u[kChunk];
        top = max(top, load_chunk<kDT>(xr, at, cols, u));
    }
#pragma unroll
    for (int d = kWave / 2; d; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    if (kLanes > kWave) {
        if (threadIdx.x % kWave == 0) tops[threadIdx.x / kWave] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kThreads / kWave; ++i) top = max(top, tops[i]);
    }

    const bool finite = top < 0x7f800000u;
    const float scale = finite ? __uint_as_float(top) * (1.0f / 127.0f) : 0.0f;
    if (lane == 0) {
        scales[row] = scale;
        if (!finite) report_generic(status, IQ_ERR_NONFINITE);
    }
#pragma unroll
    for (int c = 0; c < kKeep; ++c) {
        const int64_t at = ((int64_t)c * kLanes + lane) * kChunk;
        if (at < cols) store_chunk(qr, at, cols, v[c], scale);
    }
    for (int64_t at = kKept + lane * kChunk; at < cols; at += kLanes * kChunk) {
        float u[kChunk];
        load_chunk<kDT>(xr, at, cols, u);
        store_chunk(qr, at, cols, u, scale);
    }
}

template <int kDT, int kLanes, int kKeep>
hipError_t launch(const void* x, int64_t ldx, int64_t rows, int64_t cols, int8_t* q, int64_t ldq,
                  float* scale, int32_t* status, hipStream_t stream)
{
    const int64_t wgs = (rows + kThreads / kLanes - 1) / (kThreads / kLanes);
    hipLaunchKernelGGL((quantize_rows_kernel<kDT, kLanes, kKeep>), dim3((unsigned)wgs),
                       dim3(kThreads), 0, stream, x, ldx, rows, cols, q, ldq, scale, status);
    return hipGetLastError();
}

}  // namespace

// A wave per row up to 4096 values (8 chunks of 8 a lane: no barrier), the
// workgroup beyond.
hipError_t launch_quantize_rows(int dtype, const void* x, int64_t ldx, int64_t rows, int64_t cols,
                                int8_t* q, int64_t ldq, float* scale, int32_t* status,
                                hipStream_t stream)
{
    return with_dtype(dtype, [&](auto dt) {
        constexpr int kDT = decltype(dt)::value;
        if (cols <= 1024)
            return launch<kDT, 64, 2>(x, ldx, rows, cols, q, ldq, scale, status, stream);
        if (cols <= 4096)
            return launch<kDT, 64, 8>(x, ldx, rows, cols, q, ldq, scale, status, stream);
        return launch<kDT, 256, 4>(x, ldx, rows, cols, q, ldq, scale, status, stream);
    });
}

}  // namespace iqk
