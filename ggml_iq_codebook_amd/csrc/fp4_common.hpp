// fp4_common.hpp -- 4-bit floats in groups of 32 that share a power of two.
//
// A code is a sign and one of 0, 1/2, 1, 3/2, 2, 3, 4, 6 (bits: sign, two of
// exponent, one of mantissa); byte i of a row holds the codes of values 2i (low)
// and 2i + 1.  A group's scale byte s stands for 2^(s - 127), 255 for NaN.  The
// conversion instructions of gfx950 take the scale as a float of which they use
// the exponent: the byte shifted to its place.  Their results were compared with
// this definition for every code and every scale byte: exact in bf16 (subnormal
// where they are below 2^-126, infinite from 2^128 on, NaN for the byte 255).
#pragma once

#include "iq_fp4.h"
#include "layers_common.hpp"

namespace iqk {

constexpr int kGroup = IQ_GROUP;

__device__ __forceinline__ float group_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// The 8 codes of a word as bf16, in order.
__device__ __forceinline__ v8bf values_of(uint32_t codes, float scale)
{
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    const v2bf v[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0),
                       __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1),
                       __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2),
                       __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3)};
    return __builtin_bit_cast(v8bf, v);
}

// Codes whose values are infinite as that of 0: 4 and 6 times 2^126 (bits 2 and 1 of the
// code), from 2 times 2^127 on (bit 2).
constexpr uint32_t kInfinite = 253;

__device__ __forceinline__ uint32_t finite_codes(uint32_t codes, uint32_t byte)
{
    const uint32_t also = byte == kInfinite ? codes >> 1 : (byte > kInfinite ? ~0u : 0u);
    return codes & ~((codes >> 2 & also & 0x11111111u) * 15u);
}

// The same as fp16: exact for scale bytes kLowF16 .. kHighF16, where half of the lowest
// power is 2^-24 and 6 times the highest below 2^16.  Values of other bytes may not be
// representable, but for 0, which is 0 (NaN for the byte 255) with any of them.
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
constexpr uint32_t kLowF16 = 104, kHighF16 = 140;

__device__ __forceinline__ v8h half_values_of(uint32_t codes, float scale)
{
    typedef _Float16 v2h __attribute__((ext_vector_type(2)));
    const v2h v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 0),
                      __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 1),
                      __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 2),
                      __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 3)};
    return __builtin_bit_cast(v8h, v);
}

}  // namespace iqk
