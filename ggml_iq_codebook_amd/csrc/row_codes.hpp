// row_codes.hpp -- values of a row rounded to 8-bit codes, shared by the row
// kernel and the product that rounds its few tokens itself.
#pragma once

#include "layers_common.hpp"

namespace iqk {

constexpr int kChunk = 8;             // values a lane reads and writes at once

// kChunk values of a row as they are stored, so that a kept row takes no more
// registers than it has bytes.  kWhole: rows are whole chunks.
template <int kDT, bool kWhole>
struct Chunk {
    typedef typename Value<kDT>::raw raw;
    static constexpr int kN = Row<kDT>::kN;
    Row<kDT> r[kChunk / kN];
    __device__ __forceinline__ void load(const raw* row, int64_t at, int64_t cols)
    {
#pragma unroll
        for (int h = 0; h < kChunk / kN; ++h) {
            if (!kWhole)
                r[h].load(row, at + h * kN, cols);
            else if (at < cols)
                __builtin_memcpy(r[h].u, row + at + h * kN, 16);
            else
                r[h].zero();
        }
    }
    __device__ __forceinline__ float operator[](int i) const { return r[i / kN][i % kN]; }
    // The largest magnitude's bits: as integers they order infinities and NaN
    // above every finite value.
    __device__ __forceinline__ uint32_t top() const
    {
        uint32_t t = 0u;
#pragma unroll
        for (int i = 0; i < kChunk; ++i) t = max(t, __float_as_uint((*this)[i]) & 0x7fffffffu);
        return t;
    }
};

// The scale of a row whose largest magnitude has the bits `top`: 0 where the
// row is refused (a NaN or an infinity).
__device__ __forceinline__ float row_scale(uint32_t top)
{
    return top < 0x7f800000u ? __uint_as_float(top) * (1.0f / 127.0f) : 0.0f;
}

// x / scale rounded to the nearest integer without a division: with inv the
// reciprocal of the scale, x * inv is within 3 units of 2^-24 of the correctly
// rounded quotient, less than 2^-15 for quotients up to 127.5, so both round to
// the same integer unless x * inv is that near to a half.  Only then the
// division is done.  Adding 1.5 * 2^23 rounds to an integer (halves to even)
// and leaves it in the low bits, from where the byte is taken.
template <int kDT, bool kWhole>
__device__ __forceinline__ void codes_of(const Chunk<kDT, kWhole>& v, float scale, float inv,
                                         uint32_t (&b)[kChunk / 4])
{
    constexpr float kMagic = 12582912.0f, kSure = 0.5f - 0x1p-15f;
    uint32_t u[kChunk];
    float worst = 0.0f;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
        // The bounds only act on scales among the subnormals, whose own
        // rounding is coarse.
        const float t = fminf(fmaxf(v[i] * inv, -127.0f), 127.0f);
        const float m = t + kMagic;
        worst = fmaxf(worst, fabsf(t - (m - kMagic)));
        u[i] = __float_as_uint(m);
    }
    // The reciprocal of a scale below 2^-126 may be infinite.
    if (!(worst <= kSure) || inv > 0x1p126f) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
            u[i] = __float_as_uint(fminf(fmaxf(v[i] / scale, -127.0f), 127.0f) + kMagic);
    }
    // The low bytes of four words, byte-permuted together.
#pragma unroll
    for (int i = 0; i < kChunk / 4; ++i) {
        const uint32_t lo = __builtin_amdgcn_perm(u[4 * i + 1], u[4 * i], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(u[4 * i + 3], u[4 * i + 2], 0x04000c0cu);
        b[i] = lo | hi;
    }
}

}  // namespace iqk
