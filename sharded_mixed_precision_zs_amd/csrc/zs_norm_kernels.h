/*
 * zs_norm_kernels.h -- root-mean-square norm with the residual's addition
 * and an 8-bit microscaled output, forward and backward (gfx950).
 *
 *   h = R16(x + r);  rstd = 1 / sqrt(mean(h^2) + eps);  y = h * rstd * g
 *   dx = R16(dres + rstd * (g*dy - h * rstd^2 * mean(g*dy*h)))
 *   dg = sum over rows of dy * h * rstd
 *
 * Both are bound by HBM: every element is read once, kept in registers
 * between the row's sum and its use, and written once. Sums are binary64
 * forward and fp32 backward. The statistics are those of the rounded h, which
 * is what the backward pass reads, so both passes see the same row.
 */
#ifndef ZS_NORM_KERNELS_H
#define ZS_NORM_KERNELS_H

#include "zs_mx.h"

namespace zs {

struct NormArgs {
  const void *x, *res, *gain;
  uint16_t *h, *y;           /* optional outputs */
  float *rstd;               /* optional */
  uint8_t *codes, *scales;   /* both or neither */
  uint64_t rows;
  uint32_t cols, padded;     /* padded: cols rounded up to whole groups */
  float eps;
  double inv_cols;
};

/* 1 / sqrt(ss * inv_cols + eps) as the sum of two floats: the binary64
 * instruction's estimate, good to more than a float, corrected by one step of
 * Newton's. Binary64 throughout, for a bf16 row's squares leave fp32's range. */
struct RowScale {
  float hi, lo;
};

__device__ __forceinline__ RowScale row_scale(double ss, double inv_cols, float eps) {
  const double m = ss * inv_cols + (double)eps;
  const double r = __builtin_amdgcn_rsq(m);
  const double d = fma(0.5 * r, fma(-m * r, r, 1.0), r);
  RowScale s;
  s.hi = (float)d;
  s.lo = (float)(d - (double)s.hi);
  /* beyond float, or not a number: as the estimate says */
  if (!(r > 0.0 && s.hi <= 3.0e38f)) s = {(float)r, 0.0f};
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

/* One row per group of G threads (64: four rows per 256-thread block), ITEMS
 * vectors of eight elements per thread: x and the residual are asked for
 * whole before anything waits, and stay in registers until y. 16384 x 4096
 * bf16 with residual, h and codes: 75 us, 6.3 TB/s of the 472 MB that it has
 * to move, what a plain copy reaches; one row of 768 is a launch (2.9 us).
 * h is stored non-temporally: the next norm reads it, after a layer's
 * products (16384 x 4096: 82 us plain; eight norms each before two products
 * by 4096 x 4096: 5.11 ms plain, 5.00 so, equal up to 2048 rows). What the
 * next kernel reads, codes and y, stays in the caches.
 *
 * Precision: an element's product with the gain is exact in fp32 (8 or 11
 * significant bits each), the squares and their sum are binary64, the row's
 * scale two floats, and y keeps what its 16 or 8 bits are rounded by: both are
 * the 64-bit result's own but within some 2^-45 of a tie. */
template <int DT, bool AL, int G, int ITEMS>
__global__ __launch_bounds__(G < 256 ? 256 : G) void norm_kernel(NormArgs a) {
  constexpr int kRows = G < 256 ? 256 / G : 1;
  __shared__ double part[G / 64];
  const uint32_t t = threadIdx.x % G;
  const uint64_t row = (uint64_t)blockIdx.x * kRows + threadIdx.x / G;
  if (row >= a.rows) return;   /* a whole wave; blocks of one row never take it */
  const uint16_t *x = static_cast<const uint16_t *>(a.x) + row * a.cols;
  const uint16_t *r = a.res ? static_cast<const uint16_t *>(a.res) + row * a.cols : nullptr;
  Raw16<8> xr[ITEMS], rr[ITEMS];
  float h[ITEMS][8];
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) xr[i] = load8_ahead<AL>(x, (i * G + t) * 8, a.cols);
  if (r) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) rr[i] = load8_ahead<AL>(r, (i * G + t) * 8, a.cols);
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    settle8<AL>(xr[i], (i * G + t) * 8, a.cols);
    upcast<8, DT>(xr[i], h[i]);
  }
  if (r) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      float b[8];
      settle8<AL>(rr[i], (i * G + t) * 8, a.cols);
      upcast<8, DT>(rr[i], b);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const uint32_t w = pack2<DT>(h[i][j] + b[j], h[i][j + 1] + b[j + 1]);
        h[i][j] = up_lo<DT>(w);
        h[i][j + 1] = up_hi<DT>(w);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    if (a.h) store8<DT, AL, true>(a.h + row * a.cols, (uint64_t)(i * G + t) * 8, a.cols, h[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fma((double)h[i][j], (double)h[i][j], ss);
  }
  ss = group_sum<G>(ss, part);
  const RowScale rstd = row_scale(ss, a.inv_cols, a.eps);
  if (a.rstd && t == 0) a.rstd[row] = rstd.hi;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const uint32_t v = i * G + t;
    if (v * 8 >= a.padded) break;   /* whole quads: padded is a multiple of 128 */
    float g[8], y[8];
    load8<DT, AL>(a.gain, (uint64_t)v * 8, a.cols, g);
    uint32_t top = 0;
    /* zeros past the row's end: h and the gain are 0 there, but 0 * inf is not */
    const RowScale s = v * 8 < a.cols ? rstd : RowScale{0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[j] = times_odd(h[i][j] * g[j], s);
      top = umax(top, mag_bits(y[j]));
    }
    if (a.y) store8<DT, AL>(a.y + row * a.cols, (uint64_t)v * 8, a.cols, y);
    if (a.codes) {
      const uint32_t byte = mx_scale_byte<ZS_MX_E4M3>(quad_max(top));
      uint32_t code[2];
      mx_encode<ZS_MX_E4M3>(y, byte, code);
      *reinterpret_cast<u32x2 *>(a.codes + row * a.padded + v * 8) = u32x2{code[0], code[1]};
      if ((v & 3) == 0) a.scales[row * (a.padded / kMxBlock) + v / 4] = (uint8_t)byte;
    }
  }
}

struct NormGradArgs {
  const void *dy, *h, *gain, *dres;   /* dres optional */
  const float *rstd;
  uint16_t *dx;
  float *part;                        /* [parts][cols] */
  uint64_t rows;
  uint32_t cols, parts;
};

/* A row's share of one thread, as it lies in memory: the next row's is
 * fetched while this one is summed. */
template <int DT, bool AL, int ITEMS>
struct GradRow {
  Raw16<8> dy[ITEMS], h[ITEMS], dres[ITEMS];
  float rstd;
};

template <int DT, bool AL, int G, int ITEMS>
__device__ __forceinline__ void load_grad_row(const NormGradArgs &a, uint64_t row, uint32_t t,
                                              GradRow<DT, AL, ITEMS> &r) {
  const uint64_t at = row * a.cols;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const uint32_t c = (i * G + t) * 8;
    r.dy[i] = load8_ahead<AL>(static_cast<const uint16_t *>(a.dy) + at, c, a.cols);
    r.h[i] = load8_ahead<AL>(static_cast<const uint16_t *>(a.h) + at, c, a.cols);
    if (a.dres)
      r.dres[i] = load8_ahead<AL>(static_cast<const uint16_t *>(a.dres) + at, c, a.cols);
  }
  r.rstd = a.rstd[row];
}

/* Each of `parts` groups of G threads walks rows p, p + parts, ... and keeps
 * its share of dg in registers; norm_gain_kernel adds the shares in order,
 * so the result does not depend on scheduling (no atomics). One barrier a
 * row: the dot product's parts lie in two places in turn. 16384 x 4096 bf16
 * with dres: 102 us and 5 for the shares of dg, 5.3 TB/s of the 537 MB of
 * the rows; bound by HBM and, by 4 %, the second launch. */
template <int DT, bool AL, int G, int ITEMS>
__global__ __launch_bounds__(G < 256 ? 256 : G) void norm_grad_kernel(NormGradArgs a) {
  constexpr int kRows = G < 256 ? 256 / G : 1;
  __shared__ float sums[2][G / 64];
  const uint32_t t = threadIdx.x % G;
  const uint32_t p = blockIdx.x * kRows + threadIdx.x / G;
  if (p >= a.parts) return;
  float dg[ITEMS][8], g[ITEMS][8];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    load8<DT, AL>(a.gain, (uint64_t)(i * G + t) * 8, a.cols, g[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = 0.0f;
  }
  GradRow<DT, AL, ITEMS> r, next;
  load_grad_row<DT, AL, G>(a, p, t, r);
  int turn = 0;
  for (uint64_t row = p; row < a.rows; row += a.parts, turn ^= 1) {
    const bool more = row + a.parts < a.rows;
    if (more) load_grad_row<DT, AL, G>(a, row + a.parts, t, next);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      float h[8], d[8];
      settle8<AL>(r.dy[i], (i * G + t) * 8, a.cols);
      settle8<AL>(r.h[i], (i * G + t) * 8, a.cols);
      if (a.dres) settle8<AL>(r.dres[i], (i * G + t) * 8, a.cols);
      upcast<8, DT>(r.dy[i], d);
      upcast<8, DT>(r.h[i], h);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dg[i][j] = fmaf(d[j], h[j] * r.rstd, dg[i][j]);
        dot = fmaf(d[j] * g[i][j], h[j], dot);
      }
    }
    const float s = group_sum<G>(dot, sums[turn]) / (float)a.cols * r.rstd * r.rstd;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      float h[8], d[8], o[8] = {};
      upcast<8, DT>(r.dy[i], d);
      upcast<8, DT>(r.h[i], h);
      if (a.dres) upcast<8, DT>(r.dres[i], o);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        o[j] = fmaf(r.rstd, fmaf(-h[j], s, d[j] * g[i][j]), o[j]);
      store8<DT, AL>(a.dx + row * a.cols, (uint64_t)(i * G + t) * 8, a.cols, o);
    }
    if (more) r = next;
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t c = (i * G + t) * 8 + j;
      if (c < a.cols) a.part[(uint64_t)p * a.cols + c] = dg[i][j];
    }
}

/* dg[c] = sum of part[p][c] over p: 32 columns per block, 32 half waves that
 * take every 32nd share each (eight at a time, so that their latencies
 * overlap), joined in order. 1024 shares of 4096 columns: 5 us, the shares
 * still in the caches. */
constexpr int kGainCols = 32, kGainRuns = 32;

__global__ __launch_bounds__(kGainCols * kGainRuns) void norm_gain_kernel(const float *part,
                                                                          uint32_t parts,
                                                                          uint32_t cols,
                                                                          float *dgain) {
  __shared__ float sums[kGainRuns][kGainCols + 1];
  const uint32_t lane = threadIdx.x % kGainCols, run = threadIdx.x / kGainCols;
  const uint32_t c = blockIdx.x * kGainCols + lane;
  float s = 0.0f;
  if (c < cols) {
    const float *q = part + c;
    for (uint32_t p = run; p < parts; p += 8 * kGainRuns) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t at = p + k * kGainRuns;
        v[k] = at < parts ? q[(uint64_t)at * cols] : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[k];
    }
  }
  sums[run][lane] = s;
  __syncthreads();
  if (run == 0 && c < cols) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < kGainRuns; ++w) s += sums[w][lane];
    dgain[c] = s;
  }
}

}  // namespace zs
#endif  // ZS_NORM_KERNELS_H
