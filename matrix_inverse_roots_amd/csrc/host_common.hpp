// Host-side helpers shared by the library's translation units: the
// thread-local error message, launch checks and per-device properties.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>

#include "shampoo.h"

namespace shampoo {

// Records the calling thread's message and returns s.
shampoo_status fail(shampoo_status s, const char* fmt, ...);

#define HIP_TRY(expr)                                                                  \
  do {                                                                                 \
    hipError_t e_ = (expr);                                                            \
    if (e_ != hipSuccess) return fail(SHAMPOO_E_HIP, "%s: %s", #expr, hipGetErrorString(e_)); \
  } while (0)

#define LAUNCH_CHECK(what)                                                             \
  do {                                                                                 \
    hipError_t e_ = hipGetLastError();                                                 \
    if (e_ != hipSuccess) return fail(SHAMPOO_E_HIP, "%s launch: %s", what, hipGetErrorString(e_)); \
  } while (0)

#define HIP_TRY_ERR(expr)         \
  do {                            \
    hipError_t e_ = (expr);       \
    if (e_ != hipSuccess) return e_; \
  } while (0)

constexpr size_t ALIGN = 256;
inline size_t align_up(size_t x) { return (x + ALIGN - 1) / ALIGN * ALIGN; }

constexpr int MAX_DEVICES = 64;

// Compute units of the current device, queried once per device.
hipError_t cu_count(int* cus);

}  // namespace shampoo
