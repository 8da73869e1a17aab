// int8_decode.hip -- the 8-bit layer for a few tokens, as one launch: every
// workgroup rounds the tokens to 8 bits itself while its part of the weight is
// on its way.
//
// Bound by the weight's bytes and by latency: at these sizes a launch of its
// own for the rounding costs more than repeating it in every workgroup (a
// token of 4096 values is 8 KiB out of the L2).  A workgroup of 8 waves takes
// 16 channels; each wave takes an eighth of the depth and loads its weight
// rows straight into the operand registers of the matrix instruction, 8 pieces
// of 64 bytes a row under way at once.  The 8 partial sums are integers, so
// adding them in LDS is exact.
//
// One token through 4096 x 4096: 7.8 us in a graph with its weight in HBM, as two
// launches 10.0; called back to back on a weight that stays in the caches 6.2 us
// (16.8 MB at the rate of a large copy: 3.3 us).  32 or 64 channels to a
// workgroup, which halve the rounding of wide weights, took 9.4 and 14.0 us here
// and no less than two launches on 32768 channels.
#include <hip/hip_runtime.h>

#include "layers_launch.hpp"
#include "row_codes.hpp"

namespace iqk {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * kWave;
constexpr int kTokens = 16;           // columns of the matrix instruction
constexpr int kChannels = kDecodeChannels;   // and its rows
constexpr int kFlight = 8;            // pieces of the weight under way
constexpr int kPart = kWave * kChunk; // values a wave rounds at once

// 16 bytes of a row from depth `at`.  Beyond its end there are zeros, or, where
// the depth is a multiple of 16 (kWhole), the row's last values: the tokens'
// codes are zeros there.
template <bool kWhole>
__device__ __forceinline__ v4i load_codes(const int8_t* row, int at, int depth)
{
    v4i v = {0, 0, 0, 0};
    if (kWhole || at + 16 <= depth) {
        __builtin_memcpy(&v, row + (kWhole ? min(at, depth - 16) : at), 16);
    } else if (at < depth) {
        uint64_t u[2] = {0u, 0u};
#pragma unroll 1
        for (int i = 0; i < depth - at; ++i) {
            const uint64_t byte = (uint64_t)(uint8_t)row[at + i] << (8 * (i % 8));
            u[0] |= i < 8 ? byte : 0u;
            u[1] |= i < 8 ? 0u : byte;
        }
        v = {(int)u[0], (int)(u[0] >> 32), (int)u[1], (int)(u[1] >> 32)};
    }
    return v;
}

// kKeep: how many parts a wave rounds at most.  Its code is read once by every
// compute unit, so that its size shows: one token through 8192 x 512 takes 4.3 us
// with 4 KB of it; with 22 KB, for four parts and any depth, it took 5.6.
template <int kDT, bool kWhole, int kKeep>
__global__ __launch_bounds__(kThreads) void int8_decode_kernel(Int8Product p, const void* x,
                                                               int64_t ldx, int32_t* status)
{
    typedef typename Value<kDT>::raw raw;
    extern __shared__ __align__(16) int8_t codes[];   // [tokens][stride]
    __shared__ uint32_t tops[kTokens];
    __shared__ int sums[kWaves][kTokens][kChannels];
    const int tokens = (int)p.tokens;
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int stride = decode_stride(p.depth);

    // The weight: this wave's part of the depth, in whole pieces of 64.
    const int pieces = (p.depth + 63) / 64;
    const int first = (int)((int64_t)pieces * wave / kWaves);
    const int last = (int)((int64_t)pieces * (wave + 1) / kWaves);
    const int channel = blockIdx.x * kChannels + lane % 16;
    const int quarter = lane / 16;
    const int8_t* w = p.w + (int64_t)min(channel, p.channels - 1) * p.ldw;
    v4i a[kFlight] = {};
#pragma unroll
    for (int i = 0; i < kFlight; ++i)
        if (first + i < last)
            a[i] = load_codes<kWhole>(w, (first + i) * 64 + quarter * 16, p.depth);

    // The tokens, in parts of kPart values dealt out to the waves.
    const int parts = (p.depth + kPart - 1) / kPart;
    if (threadIdx.x < kTokens) tops[threadIdx.x] = 0u;
    __syncthreads();
    Chunk<kDT, kWhole> kept[kKeep];
#pragma unroll
    for (int c = 0; c < kKeep; ++c) {
        const int part = c * kWaves + wave;
        const int token = part / parts;
        if (token < tokens)
            kept[c].load(static_cast<const raw*>(x) + token * ldx,
                         (part - token * parts) * kPart + lane * kChunk, p.depth);
    }
#pragma unroll
    for (int c = 0; c < kKeep; ++c) {
        const int token = (c * kWaves + wave) / parts;
        if (token < tokens) {
            uint32_t top = kept[c].top();
#pragma unroll
            for (int d = kWave / 2; d; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
            if (lane == 0) atomicMax(&tops[token], top);
        }
    }
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x < tokens && tops[threadIdx.x] >= 0x7f800000u)
        report_generic(status, IQ_ERR_NONFINITE);
#pragma unroll
    for (int c = 0; c < kKeep; ++c) {
        const int part = c * kWaves + wave;
        const int token = part / parts;
        if (token < tokens) {
            const float scale = row_scale(tops[token]);
            const int at = (part - token * parts) * kPart + lane * kChunk;
            uint32_t b[kChunk / 4] = {};
            if (scale > 0.0f) codes_of(kept[c], scale, 1.0f / scale, b);
            // Values beyond the depth are zeros, and so are their codes.
            if (at < stride) *reinterpret_cast<uint2*>(codes + token * stride + at) = make_uint2(b[0], b[1]);
        }
    }
    __syncthreads();

    // Lanes of tokens there are none of repeat the last one: not stored.
    const int8_t* own = codes + min(lane % 16, tokens - 1) * stride + quarter * 16;
    v4i acc = {0, 0, 0, 0};
    for (int at = first; at < last; at += kFlight) {
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            if (at + i < last) {
                const v4i b = *reinterpret_cast<const v4i*>(own + (at + i) * 64);
                acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], b, acc, 0, 0, 0);
            }
            const int next = at + i + kFlight;
            if (next < last) a[i] = load_codes<kWhole>(w, next * 64 + quarter * 16, p.depth);
        }
    }
    *reinterpret_cast<v4i*>(&sums[wave][lane % 16][4 * quarter]) = acc;
    __syncthreads();
    const int token = threadIdx.x / kChannels, c = threadIdx.x % kChannels;
    const int at = blockIdx.x * kChannels + c;
    if (token < tokens && at < p.channels) {
        int sum = 0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) sum += sums[i][token][c];
        const float y = (float)sum * row_scale(tops[token]) * p.w_scale[at];
        static_cast<raw*>(p.y)[token * p.ldy + at] = Value<kDT>::store(y);
    }
}

template <int kKeep>
hipError_t launch_keeping(const Int8Product& p, int dtype, const void* x, int64_t ldx,
                          int32_t* status, hipStream_t stream)
{
    const unsigned wgs = (unsigned)((p.channels + kChannels - 1) / kChannels);
    const size_t lds = (size_t)p.tokens * decode_stride(p.depth);
    return with_dtype(dtype, [&](auto dt) {
        constexpr int kDT = decltype(dt)::value;
        if (p.depth % 16 == 0)
            hipLaunchKernelGGL((int8_decode_kernel<kDT, true, kKeep>), dim3(wgs), dim3(kThreads),
                               lds, stream, p, x, ldx, status);
        else
            hipLaunchKernelGGL((int8_decode_kernel<kDT, false, kKeep>), dim3(wgs), dim3(kThreads),
                               lds, stream, p, x, ldx, status);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_int8_decode(const Int8Product& p, int dtype, const void* x, int64_t ldx,
                              int32_t* status, hipStream_t stream)
{
    const int64_t parts = p.tokens * ((p.depth + kPart - 1) / kPart);
    if (parts <= kWaves) return launch_keeping<1>(p, dtype, x, ldx, status, stream);
    if (parts <= 2 * kWaves) return launch_keeping<2>(p, dtype, x, ldx, status, stream);
    return launch_keeping<kDecodeParts / kWaves>(p, dtype, x, ldx, status, stream);
}

}  // namespace iqk
