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
        // Keeps a product from being rounded to fp16 in one step with its
        // conversion (v_fma_mixlo_f16), which the compiler does in some kernels
        // and not in others: every result is rounded to fp32 first.
        asm("" : "+v"(f));
        return __builtin_bit_cast(uint16_t, (_Float16)f);
    }
};

// 16 bytes of a row, read or written as one instruction.  The addresses need
// the alignment of a value only (global memory instructions take any address;
// memcpy tells the compiler).  The last vector of a row whose width is no
// multiple goes value by value, and values beyond the width read as 0.
template <int kDT>
struct Row {
    typedef typename Value<kDT>::raw raw;
    static constexpr int kN = 16 / (int)sizeof(raw);
    uint32_t u[4];
    __device__ __forceinline__ raw get(int i) const
    {
        return sizeof(raw) == 4 ? (raw)u[i] : (raw)(u[i / 2] >> (16 * (i % 2)));
    }
    __device__ __forceinline__ void load(const raw* row, int64_t at, int64_t width)
    {
        if (at + kN <= width) {
            __builtin_memcpy(u, row + at, 16);
        } else {
            zero();
#pragma unroll
            for (int i = 0; i < kN; ++i)
                if (at + i < width) put(i, row[at + i]);
        }
    }
    // A whole vector that is not read again soon.
    __device__ __forceinline__ void load_once(const raw* from)
    {
        typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(2)));
        const u4 v = __builtin_nontemporal_load(reinterpret_cast<const u4*>(from));
        u[0] = v.x; u[1] = v.y; u[2] = v.z; u[3] = v.w;
    }
    __device__ __forceinline__ void store(raw* row, int64_t at, int64_t width) const
    {
        if (at + kN <= width) {
            __builtin_memcpy(row + at, u, 16);
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i)
                if (at + i < width) row[at + i] = get(i);
        }
    }
    // kStreaming: a whole vector goes past the caches.
    template <bool kStreaming>
    __device__ __forceinline__ void store(raw* row, int64_t at, int64_t width) const
    {
        if (kStreaming && at + kN <= width) {
            typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(2)));
            const u4 v = {u[0], u[1], u[2], u[3]};
            __builtin_nontemporal_store(v, reinterpret_cast<u4*>(row + at));
        } else {
            store(row, at, width);
        }
    }
    __device__ __forceinline__ void zero() { u[0] = u[1] = u[2] = u[3] = 0u; }
    // Value i of a vector that held 0 there.
    __device__ __forceinline__ void put(int i, raw r)
    {
        if (sizeof(raw) == 4)
            u[i] = r;
        else
            u[i / 2] |= (uint32_t)r << (16 * (i % 2));
    }
    __device__ __forceinline__ float operator[](int i) const { return Value<kDT>::load(get(i)); }
    __device__ __forceinline__ void set(int i, float f) { put(i, Value<kDT>::store(f)); }
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
