/*
 * zs_norm_launch.h -- the norms' launch shapes. Host code only.
 */
#ifndef ZS_NORM_LAUNCH_H
#define ZS_NORM_LAUNCH_H

#include "zs_ops_common.h"

namespace zs_ops {

/* ------------------------------------------------------------------------
 * The norm's threads per row and vectors of eight per thread: a wave for
 * short rows, then a block that grows with the row, so that a thread has two
 * vectors and the backward pass's sums and next row fit its registers
 * (16384 x 4096 backward: 110 us with 256 threads of two vectors, 285 with
 * one wave of eight; up to 1024 elements one wave saves the barrier: 65536 x
 * 1024 forward in 87 us). That ends at 8192 elements: the backward pass of
 * 1024 threads, of 128 registers each, keeps 72 to 284 bytes a thread in
 * scratch memory up to 16384 and 1.5 to 2.1 KB above.
 * ---------------------------------------------------------------------- */
constexpr uint64_t kMaxNormCols = 65536;

template <class F>
void with_norm_shape(uint64_t padded, F f) {
  if (padded <= 512) f(Tag<64>{}, Tag<1>{});
  else if (padded <= 1024) f(Tag<64>{}, Tag<2>{});
  else if (padded <= 2048) f(Tag<256>{}, Tag<1>{});
  else if (padded <= 4096) f(Tag<256>{}, Tag<2>{});
  else if (padded <= 8192) f(Tag<512>{}, Tag<2>{});
  else if (padded <= 16384) f(Tag<1024>{}, Tag<2>{});
  else f(Tag<1024>{}, Tag<8>{});
}

/* Groups that share the rows of a backward pass: some four rows each, for
 * their sums of dg cost as much again as a row or two; 256 at least, a block
 * for every CU, and 1024 at most. */
inline uint32_t norm_parts(uint64_t rows) {
  const uint64_t want = rows / 4 < 256 ? 256 : rows / 4 > 1024 ? 1024 : rows / 4;
  return (uint32_t)(rows < want ? rows : want);
}

}  // namespace zs_ops
#endif  // ZS_NORM_LAUNCH_H
