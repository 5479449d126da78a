// echo_host.hpp — host-side pieces that every entry point shares: the calling
// thread's last HIP error and the checks of pointers, sizes and launches.
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

// ---- what the operators on matrices of rows check

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxLd = int64_t(1) << 32;        // row strides; offsets are 64-bit
constexpr int64_t kMaxGrid = int64_t(1) << 20;      // blocks of a launch; kernels stride over the rest

inline bool float_dtype(int d) { return d == ECHO_F32 || d == ECHO_BF16; }
inline size_t dtype_bytes(int d) { return d == ECHO_F32 ? 4 : (d == ECHO_BF16 ? 2 : 1); }
inline bool aligned_elem(const void* p, int dtype) { return aligned_to(p, dtype_bytes(dtype)); }

// rows of `cols` elements at a distance of ld (which a single row does not use)
inline bool bad_ld(int64_t ld, int64_t rows, int64_t cols) { return rows > 1 && (ld < cols || ld > kMaxLd); }
inline bool bad_dim(int64_t v, int64_t most) { return v < 0 || v > most; }

inline unsigned grid_of(int64_t items) { return (unsigned)(items < kMaxGrid ? items : kMaxGrid); }
// a launch's work-items are a 32-bit number
inline bool grid_fits(int64_t blocks, int64_t threads) { return blocks * threads < (int64_t(1) << 32); }

}  // namespace echo
