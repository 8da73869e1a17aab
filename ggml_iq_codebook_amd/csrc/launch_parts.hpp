// launch_parts.hpp -- launches of any number of workgroups.
//
// A launch has fewer than 2^32 threads in x: beyond, the runtime takes the number
// modulo 2^32 and reports nothing, and the rest of the workgroups never run.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace iqk {

// launch(first, count) for each part of `wgs` workgroups, of at most 2^31 threads,
// until one fails.  Parts begin at multiples of 8 workgroups, so that workgroup
// first + i runs on XCD i % 8.
template <class Launch>
inline hipError_t in_parts(int64_t wgs, int threads, Launch&& launch)
{
    const int64_t most = (INT64_C(1) << 31) / threads;
    hipError_t e = hipSuccess;
    for (int64_t first = 0; first < wgs && e == hipSuccess; first += most)
        e = launch(first, dim3((unsigned)std::min(most, wgs - first)));
    return e;
}

}  // namespace iqk
