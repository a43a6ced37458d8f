/*
 * zs_epilogue.h -- what a product does with its fp32 sums before they are
 * stored, and activations (gfx950):
 *   pre = sum + bias;  c = R16(residual + act(pre))
 * pre is rounded only where it is stored; the activation sees its fp32. Bound
 * with the product by the matrix cores: 8192 x 16384 x 4096 of 8 x 4 bits with
 * bias, gelu and pre 960 us, with bias and residual 923, the product alone 970.
 *
 * gelu, the form with the hyperbolic tangent, 0.5 x (1 + tanh u), and silu are
 * both x times the logistic function of w: 2 u = 2 sqrt(2 / pi) (x + 0.044715
 * x^3), and x. So neither 1 + tanh nor a sum near it loses the small values.
 */
#ifndef ZS_EPILOGUE_H
#define ZS_EPILOGUE_H

#include "zs_mx.h"

namespace zs {

constexpr float kGeluCube = 0.044715f;
constexpr float kGeluLog2 = 2.30220819f;   /* 2 sqrt(2 / pi) log2(e) */
constexpr float kGelu = 1.59576912f;       /* 2 sqrt(2 / pi) */
constexpr float kLog2e = 1.44269504f;

/* The instruction's reciprocal is off by a unit in the last place, of 24 bits
 * where the result has 8 or 11. */
template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if constexpr (ACT == ZS_ACT_RELU) return x > 0.0f ? x : x == x ? 0.0f : x;
  if constexpr (ACT == ZS_ACT_GELU || ACT == ZS_ACT_SILU) {
    const float w = ACT == ZS_ACT_GELU ? kGeluLog2 * x * fmaf(kGeluCube * x, x, 1.0f) : kLog2e * x;
    return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-w));
  }
  return x;
}

/* d act / d x. With p the logistic function of w and q = 1 - p, formed without
 * the difference: p (1 + x q w'). Beyond 30 the slope is 0 or 1 in any type
 * here, and w' of such x would leave fp32. The exponential is 0 below 2^-126, and
 * so are slopes below some 2^-118 (gelu's left of -10). */
template <int ACT>
__device__ __forceinline__ float slope_of(float x) {
  if constexpr (ACT == ZS_ACT_RELU) return x > 0.0f ? 1.0f : x == x ? 0.0f : x;
  if constexpr (ACT == ZS_ACT_GELU || ACT == ZS_ACT_SILU) {
    constexpr float top = ACT == ZS_ACT_GELU ? 30.0f : 110.0f;
    const float c = __builtin_amdgcn_fmed3f(x, -top, top);
    float w = kLog2e * c, dw = 1.0f;
    if constexpr (ACT == ZS_ACT_GELU) {
      const float s = c * c;
      w = kGeluLog2 * c * fmaf(kGeluCube, s, 1.0f);
      dw = kGelu * fmaf(3.0f * kGeluCube, s, 1.0f);
    }
    const float t = __builtin_amdgcn_exp2f(-fabsf(w));
    const float big = __builtin_amdgcn_rcpf(1.0f + t), small = t * big;
    const float p = w >= 0.0f ? big : small, q = w >= 0.0f ? small : big;
    return x == x ? p * fmaf(c * q, dw, 1.0f) : x;
  }
  return 1.0f;
}

struct NoEpilogue {
  static constexpr bool kOn = false;
};

/* The activation is one of a launch's few: told apart at run time, once for
 * the values of a thread. */
struct Epilogue {
  static constexpr bool kOn = true;
  const void *bias, *res;   /* optional */
  uint16_t *pre;            /* optional, [m][n] */
  uint64_t ldr;
  int act;

  template <int N>
  __device__ __forceinline__ void apply(float (&x)[N]) const {
    if (act == ZS_ACT_GELU) {
#pragma unroll
      for (int j = 0; j < N; ++j) x[j] = activate<ZS_ACT_GELU>(x[j]);
    } else if (act == ZS_ACT_SILU) {
#pragma unroll
      for (int j = 0; j < N; ++j) x[j] = activate<ZS_ACT_SILU>(x[j]);
    } else if (act == ZS_ACT_RELU) {
#pragma unroll
      for (int j = 0; j < N; ++j) x[j] = activate<ZS_ACT_RELU>(x[j]);
    }
  }

  /* Eight neighbouring sums of a row, their bias and residual given, to memory. */
  template <int CDT>
  __device__ __forceinline__ void store(uint64_t row, uint32_t col, uint32_t n, float (&x)[8],
                                        const float (&b)[8], const Raw16<8> &residual, uint16_t *c,
                                        uint64_t ldc) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] += b[j];
    if (pre) store8<CDT, false>(pre + row * n, col, n, x);
    apply(x);
    if (res) {
      float r[8];
      upcast<8, CDT>(residual, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] += r[j];
    }
    store8<CDT, false>(c + row * ldc, col, n, x);
  }

  __device__ __forceinline__ Raw16<8> load(uint64_t row, uint32_t col, uint32_t n) const {
    return load8_raw<false>(static_cast<const uint16_t *>(res) + row * ldr, col, n);
  }

  /* One sum. */
  template <int CDT>
  __device__ __forceinline__ void store1(uint64_t row, uint32_t col, uint32_t n, float x,
                                         uint16_t *c, uint64_t ldc) const {
    if (col >= n) return;
    float v[1] = {x};
    if (bias) v[0] += up_lo<CDT>(static_cast<const uint16_t *>(bias)[col]);
    if (pre) pre[row * n + col] = pack1<CDT>(v[0]);
    apply(v);
    if (res) v[0] += up_lo<CDT>(static_cast<const uint16_t *>(res)[row * ldr + col]);
    c[row * ldc + col] = pack1<CDT>(v[0]);
  }
};

}  // namespace zs
#endif  // ZS_EPILOGUE_H
