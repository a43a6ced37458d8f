/*
 * zs_dropout_kernels.h -- dropout with the residual's addition (gfx950):
 *   out = R(residual + (kept ? x / (1 - p) : 0))
 * Bound by HBM: x and the residual in, out out, nothing else, by blocks that
 * live for one vector a thread, as a copy is fastest here (16384 x 4096 bf16 63
 * us, 6.4 TB/s).
 */
#ifndef ZS_DROPOUT_KERNELS_H
#define ZS_DROPOUT_KERNELS_H

#include "zs_philox.h"

namespace zs {

struct DropoutArgs {
  const void *x, *res;     /* res optional */
  void *out;
  uint64_t rows, cols;
  uint32_t vpr;            /* vectors of eight per row */
  uint32_t vecs;           /* in all */
  DropArgs drop;
};

/* A vector of eight elements of a row per thread. A dropped element is not
 * multiplied but replaced, so that an infinity or NaN in its place is gone. */
template <int DT, bool AL>
__global__ __launch_bounds__(kBlock) void dropout_kernel(DropoutArgs a) {
  const uint32_t id = blockIdx.x * kBlock + threadIdx.x;   /* a launch has below 2^32 */
  if (id >= a.vecs) return;
  constexpr uint64_t esz = DT == ZS_FP32 ? 4 : 2;
  const uint32_t row = id / a.vpr, v = id % a.vpr;
  const uint64_t at = (uint64_t)row * a.cols * esz;
  float x[8], r[8] = {};
  load8<DT, AL, true>(static_cast<const char *>(a.x) + at, (uint64_t)v * 8, a.cols, x);
  if (a.res) load8<DT, AL, true>(static_cast<const char *>(a.res) + at, (uint64_t)v * 8, a.cols, r);
  if (a.drop.threshold) {
    const RandomWords w = random_words(a.drop, drop_offset(a.drop), v, row);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = kept(w, j, a.drop.threshold) ? x[j] * a.drop.factor : 0.0f;
  }
  /* without a residual r is 0, and a sum of zeros is +0: -0 stays -0 */
  if (a.res) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = r[j] + x[j];
  }
  char *out = static_cast<char *>(a.out) + at;
  if constexpr (DT == ZS_FP32) store8f<AL, true>(reinterpret_cast<float *>(out), (uint64_t)v * 8, a.cols, x);
  else store8<DT, AL, true>(reinterpret_cast<uint16_t *>(out), (uint64_t)v * 8, a.cols, x);
}

}  // namespace zs
#endif  // ZS_DROPOUT_KERNELS_H
