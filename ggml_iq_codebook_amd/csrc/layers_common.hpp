// layers_common.hpp -- device helpers of the layer operators: values of the
// three storage types as fp32 and back, and vectors of them at any alignment.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"

namespace iqk {

// One storage type (iq_dtype_t): to fp32 exactly, from fp32 rounded to nearest
// even (the conversion instructions keep NaN and infinity).
template <int kDT>
struct Value;
template <>
struct Value<IQ_DTYPE_F32> {
    typedef uint32_t raw;
    __device__ __forceinline__ static float load(raw r) { return __uint_as_float(r); }
    __device__ __forceinline__ static raw store(float f) { return __float_as_uint(f); }
};
template <>
struct Value<IQ_DTYPE_BF16> {
    typedef uint16_t raw;
    __device__ __forceinline__ static float load(raw r) { return bf16_to_f32(r); }
    __device__ __forceinline__ static raw store(float f)
    {
        return __builtin_bit_cast(uint16_t, (__bf16)f);
    }
};
template <>
struct Value<IQ_DTYPE_F16> {
    typedef uint16_t raw;
    __device__ __forceinline__ static float load(raw r)
    {
        return (float)__builtin_bit_cast(_Float16, r);
    }
    __device__ __forceinline__ static raw store(float f)
    {
        return __builtin_bit_cast(uint16_t, (_Float16)f);
    }
};

// n consecutive values read or written as one or two instructions.  The
// addresses need the alignment of the value only: global memory instructions
// take any address, and the compiler is told so by going through memcpy.
template <class T, int kN>
struct Pack {
    T v[kN];
    __device__ __forceinline__ void load(const T* p) { __builtin_memcpy(v, p, sizeof(v)); }
    __device__ __forceinline__ void store(T* p) const { __builtin_memcpy(p, v, sizeof(v)); }
};

// Runs body(kDT constant) for a validated storage type.
template <int kV>
struct Int {
    static constexpr int value = kV;
};
template <class Body>
inline hipError_t with_dtype(int dtype, Body&& body)
{
    switch (dtype) {
    case IQ_DTYPE_F32: return body(Int<IQ_DTYPE_F32>());
    case IQ_DTYPE_BF16: return body(Int<IQ_DTYPE_BF16>());
    default: return body(Int<IQ_DTYPE_F16>());
    }
}

}  // namespace iqk
