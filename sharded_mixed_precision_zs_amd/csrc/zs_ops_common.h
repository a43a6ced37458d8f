/*
 * zs_ops_common.h -- what the host sides of the operators share: tests of
 * arguments, and the choice of a kernel's template arguments. Host code only.
 */
#ifndef ZS_OPS_COMMON_H
#define ZS_OPS_COMMON_H

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "zeroshard.h"

#include "zs_host_common.h"

namespace zs_ops {

using zs_host::fail;
using zs_host::launch_result;
using zs_host::overlaps;
using zs_host::too_big;

constexpr uint64_t kMaxVocab = 0x7fffffffull;   /* token ids are 31 bits */

/* Whether a launch may have so many blocks: its threads are counted in 32 bits. */
inline bool fits(uint64_t blocks, uint64_t threads) { return blocks <= 0xffffffffull / threads; }

inline bool valid16(int dt) { return dt == ZS_BF16 || dt == ZS_FP16; }
inline bool valid_any(int dt) { return valid16(dt) || dt == ZS_FP32; }
inline bool valid_format(int f) { return f == ZS_MX_E2M1 || f == ZS_MX_E4M3; }

inline uint64_t esize(int dt) { return dt == ZS_FP32 ? 4 : 2; }
inline uint64_t padded_of(uint64_t k) { return (k + ZS_MX_GROUP - 1) / ZS_MX_GROUP * ZS_MX_GROUP; }
inline uint64_t code_bytes(int format, uint64_t padded) { return format == ZS_MX_E2M1 ? padded / 2 : padded; }

inline bool aligned(const void *p, uint64_t bytes) { return (uintptr_t)p % bytes == 0; }

/* Bytes from the first to the last element of `rows` rows of `cols`, `ld` apart. */
inline uint64_t extent(uint64_t rows, uint64_t cols, uint64_t ld, uint64_t esz) {
  return rows ? ((rows - 1) * ld + cols) * esz : 0;
}

/* A matrix whose element counts stay below 2^48. */
inline bool matrix_too_big(uint64_t rows, uint64_t cols) {
  return too_big(rows) || too_big(cols) || (cols && rows > zs_host::kMaxElems / cols);
}

/* Calls f with std::integral_constant-like tags chosen at run time. */
template <int V>
struct Tag {
  static constexpr int value = V;
};

template <class F>
void with16(int dt, F f) {
  if (dt == ZS_BF16) f(Tag<ZS_BF16>{});
  else f(Tag<ZS_FP16>{});
}

template <class F>
void with_any(int dt, F f) {
  if (dt == ZS_FP32) f(Tag<ZS_FP32>{});
  else with16(dt, f);
}

template <class F>
void with_format(int fmt, F f) {
  if (fmt == ZS_MX_E2M1) f(Tag<ZS_MX_E2M1>{});
  else f(Tag<ZS_MX_E4M3>{});
}

template <class F>
void with_bool(bool b, F f) {
  if (b) f(Tag<1>{});
  else f(Tag<0>{});
}

/* CUs of the current device (256 if unknown). */
inline int cu_count() {
  static thread_local int cached_dev = -1, cached = 256;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 256;
  if (dev != cached_dev) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) n = 0;
    cached = n > 0 ? n : 256;
    cached_dev = dev;
  }
  return cached;
}

}  // namespace zs_ops
#endif  // ZS_OPS_COMMON_H
