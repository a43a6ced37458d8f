/*
 * zs_norm_rows.h -- what the norms share (gfx950): a row's scale, a value
 * rounded so that its 16 or 8 bits are right, and vectors of eight elements
 * asked for ahead.
 */
#ifndef ZS_NORM_ROWS_H
#define ZS_NORM_ROWS_H

#include "zs_mx.h"

namespace zs {

/* 1 / sqrt(ss * inv_cols + eps): the binary64 instruction's estimate, good to
 * more than a float, corrected by one step of Newton's. Binary64 throughout,
 * for a bf16 row's squares leave fp32's range. */
__device__ __forceinline__ double row_scale64(double ss, double inv_cols, float eps) {
  const double m = ss * inv_cols + (double)eps;
  const double r = __builtin_amdgcn_rsq(m);
  const double d = fma(0.5 * r, fma(-m * r, r, 1.0), r);
  /* beyond float, or not a number: as the estimate says */
  return r > 0.0 && (float)d <= 3.0e38f ? d : r;
}

/* The same as the sum of two floats. */
struct RowScale {
  float hi, lo;
};

__device__ __forceinline__ RowScale row_scale(double ss, double inv_cols, float eps) {
  const double d = row_scale64(ss, inv_cols, eps);
  RowScale s;
  s.hi = (float)d;
  s.lo = s.hi > 0.0f && s.hi <= 3.0e38f ? (float)(d - (double)s.hi) : 0.0f;
  return s;
}

/* hg (hi + lo), rounded to odd: where it is no float, to the neighbour whose
 * last bit is set. Rounded again to 16 or 8 bits this gives what the exact
 * value gives, for it is neither a tie nor a power of two that the exact value
 * is not. (Rounded to nearest first, one code in some millions fell to the
 * other side of a tie, and a block's scale with it at a power of two; it costs
 * 1.5 us of 16384 x 4096's 75.) */
__device__ __forceinline__ float times_odd(float hg, const RowScale &s) {
  const float small = hg * s.lo, y = fmaf(hg, s.hi, small);
  const float rest = fmaf(hg, s.hi, -y) + small;
  const int b = __float_as_int(y);
  /* towards 0, if the rest points there, and the last bit set */
  const int odd = (b + ((b ^ __float_as_int(rest)) >> 31)) | 1;
  constexpr int kFiniteNotZero = 0x198;   /* normal and subnormal, of either sign */
  return __int_as_float(__builtin_amdgcn_classf(rest, kFiniteNotZero) ? odd : b);
}

/* Eight elements of a row, asked for ahead: the last few of a row that is not
 * whole vectors come with what is before them, and are shifted down when they
 * are used, so that no load waits for another (8192 x 2047 bf16 backward: 42
 * us; one by one where they are asked for, 61). */
template <bool AL>
__device__ __forceinline__ Raw16<8> load8_ahead(const void *row, uint32_t col, uint32_t cols) {
  if (AL || cols < 8) return load8_raw<AL, true>(row, col, cols);
  Raw16<8> r = {};
  if (col < cols) {
    const uint32_t at = col + 8 <= cols ? col : cols - 8;
    const Loose16 v =
        *reinterpret_cast<const Loose16 *>(static_cast<const uint16_t *>(row) + at);
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[j] = v.w[j];
  }
  return r;
}

template <bool AL>
__device__ __forceinline__ void settle8(Raw16<8> &r, uint32_t col, uint32_t cols) {
  if (AL || cols < 8 || col >= cols || col + 8 <= cols) return;
  const uint32_t k = col + 8 - cols;   /* 1 .. 7 elements too early */
  if (k & 4) r.w[0] = r.w[2], r.w[1] = r.w[3], r.w[2] = r.w[3] = 0;
  if (k & 2) r.w[0] = r.w[1], r.w[1] = r.w[2], r.w[2] = r.w[3], r.w[3] = 0;
  if (k & 1) {
#pragma unroll
    for (int j = 0; j < 3; ++j) r.w[j] = r.w[j] >> 16 | r.w[j + 1] << 16;
    r.w[3] >>= 16;
  }
}

}  // namespace zs
#endif  // ZS_NORM_ROWS_H
