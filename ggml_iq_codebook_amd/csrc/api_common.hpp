// api_common.hpp -- host helpers shared by the C-ABI entry points: the device
// check, alignment, and running a launch with or without a caller's status
// word.  Defined in api.hip where they are not inline.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "iq_codec.h"

namespace iqk {

// IQ_OK if the current device is a gfx950 GPU; its compute units in *cus (when
// given): launches size their grids and tiles by it.
iq_status_t check_device(int* cus = nullptr);

inline bool aligned(const void* p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

inline iq_status_t from_hip(hipError_t e) { return e == hipSuccess ? IQ_OK : IQ_ERR_HIP; }

// launch(what, word) reporting into the device's own status word; waits for
// the stream and returns the word.
iq_status_t run_synced(hipStream_t stream, hipError_t (*launch)(void*, int32_t*), void* what);

// Runs launch(status) when the caller gave a status word, and otherwise
// run_synced's form of it.
template <class Launch>
iq_status_t run_with_status(int32_t* status, hipStream_t stream, Launch&& launch)
{
    if (status) return from_hip(launch(status));
    return run_synced(
        stream,
        [](void* what, int32_t* word) -> hipError_t {
            return (*static_cast<typename std::remove_reference<Launch>::type*>(what))(word);
        },
        &launch);
}

}  // namespace iqk
