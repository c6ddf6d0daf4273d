// Host-side helpers shared by the C entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq.h"

namespace mxq {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline mxq_status launch_status()
{
    hipError_t e = hipGetLastError();
    return e == hipSuccess ? MXQ_OK : MXQ_ERR_LAUNCH;
}

}  // namespace mxq
