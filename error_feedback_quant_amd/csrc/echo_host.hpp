// echo_host.hpp — host-side pieces that every entry point shares: the calling
// thread's last HIP error and the pointer checks.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "echo.h"

namespace echo {

inline thread_local int t_last_hip_error = 0;

inline int hip_fail(hipError_t e)
{
    t_last_hip_error = (int)e;
    return ECHO_EHIP;
}

inline int check_launch()
{
    hipError_t e = hipGetLastError();
    return e == hipSuccess ? ECHO_OK : hip_fail(e);
}

inline bool aligned_to(const void* p, size_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned_to(p, 16); }

}  // namespace echo
