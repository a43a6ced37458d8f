/*
 * zs_host_common.h -- what every host source of libzeroshard's entry points
 * shares: the thread's last error, the launch check, and the overlap and
 * size tests of argument validation. Host code only.
 */
#ifndef ZS_HOST_COMMON_H
#define ZS_HOST_COMMON_H

#include <hip/hip_runtime.h>

#include <stdint.h>
#include <stdio.h>

#include "zeroshard.h"

namespace zs_host {

inline thread_local char g_err[512] = "";

inline int fail(int status, const char *fmt, const char *detail = "") {
  snprintf(g_err, sizeof g_err, fmt, detail);
  return status;
}

inline int launch_result() {
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(ZS_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  g_err[0] = 0;
  return ZS_OK;
}

/* Element counts and offsets above 2^48 are refused before any size
 * arithmetic (byte extents below are 4 * n and must not wrap). */
constexpr uint64_t kMaxElems = 1ull << 48;

inline bool too_big(uint64_t n) { return n > kMaxElems; }

inline bool overlaps(const void *a, uint64_t abytes, const void *b, uint64_t bbytes) {
  if (!a || !b || !abytes || !bbytes) return false;
  uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + bbytes && b0 < a0 + abytes;
}

}  // namespace zs_host
#endif  // ZS_HOST_COMMON_H
