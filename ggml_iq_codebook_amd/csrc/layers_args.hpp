// layers_args.hpp -- checks that the entry points of the layer operators share.
// Host code only.
#pragma once

#include <cstdint>

#include "iq_layers.h"

namespace iqk {

// Bytes per value, 0 for a type these calls do not take.
inline int value_bytes(iq_dtype_t t)
{
    return t == IQ_DTYPE_F32 ? 4 : (t == IQ_DTYPE_BF16 || t == IQ_DTYPE_F16 ? 2 : 0);
}

// Rows of `cols` values with stride ld: every offset stays below 2^61.
// Outputs may not have rows that overlap (ld >= cols); inputs may.
inline bool bad_rows(int64_t rows, int64_t cols, int64_t ld, bool output)
{
    if (rows < 0 || cols < 1 || ld < 0 || (output && rows > 1 && ld < cols)) return true;
    const int64_t most = INT64_C(1) << 61;
    return cols > most || (ld > 0 && rows > most / ld);
}

// Places are 32-bit.
inline bool bad_choices(int64_t tokens, int32_t top_k)
{
    return tokens < 0 || top_k < 1 || tokens > INT32_MAX / top_k;
}

inline int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

}  // namespace iqk
