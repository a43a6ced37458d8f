/*
 * zs_mx.h -- microscaled rows on the device (gfx950): the scale byte of a
 * block, conversion of eight values to E2M1 or E4M3 codes and back, and the
 * eight-element loads and stores the operators share.
 *
 * A block of 32 elements holds q_i * 2^(b - 127) with b = max(1, E - emax),
 * E the biased fp32 exponent of the largest magnitude in the block and
 * emax = 2 (E2M1, largest value 6 = 1.5 * 2^2) or 8 (E4M3, 448 = 1.75 * 2^8).
 * Dividing by a power of two is exact, so the only rounding is the one to
 * the element format: to nearest, ties to even, saturating. A block that
 * holds an infinity or NaN gets b = 255 and zero codes: all its values are
 * NaN, in the product too.
 *
 * Eight consecutive elements belong to one thread and four neighbouring
 * lanes share a block, so a block's maximum is two exchanges inside a quad
 * of lanes and needs no shared memory.
 */
#ifndef ZS_MX_H
#define ZS_MX_H

#include "zs_kernels.h"

namespace zs {

constexpr uint32_t kMxBlock = ZS_MX_BLOCK; /* elements that share a scale   */
constexpr uint32_t kMxGroup = ZS_MX_GROUP; /* rows are padded to whole groups */

template <int FMT>
constexpr int kMxEmax = FMT == ZS_MX_E2M1 ? 2 : 8;

/* Bytes of the codes of `n` elements. */
template <int FMT>
__host__ __device__ constexpr uint64_t mx_bytes(uint64_t n) {
  return FMT == ZS_MX_E2M1 ? n / 2 : n;
}

/* Magnitude bits: ordered like the magnitudes, with infinity and NaN on top. */
__device__ __forceinline__ uint32_t mag_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

/* Largest of the four lanes of a quad, on all four. */
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, true)); /* lane ^ 1 */
  v = umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, true)); /* lane ^ 2 */
  return v;
}

template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);
  const int b = e - kMxEmax<FMT>;
  return e == 255 ? 255u : (uint32_t)(b > 1 ? b : 1);
}

/* 2^(b - 127); infinity for the NaN byte */
__device__ __forceinline__ float mx_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

typedef short s16x2 __attribute__((ext_vector_type(2)));

/* Codes of eight values: one word (E2M1) or two (E4M3), element 0 lowest.
 * The converts divide by the scale, round to nearest even and, for E2M1,
 * saturate; E4M3 values are clamped to 448 first (beyond it the convert
 * gives NaN). */
template <int FMT>
__device__ __forceinline__ void mx_encode(const float (&x)[8], uint32_t byte, uint32_t (&code)[2]) {
  const float s = mx_scale(byte);
  if constexpr (FMT == ZS_MX_E2M1) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], s, 3);
    code[0] = byte == 255 ? 0u : w;
    code[1] = 0;
  } else {
    const float top = 448.0f * s;
    float c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = __builtin_amdgcn_fmed3f(x[j], -top, top);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s16x2 w = {0, 0};
      w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c[4 * h], c[4 * h + 1], s, false);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c[4 * h + 2], c[4 * h + 3], s, true);
      code[h] = byte == 255 ? 0u : __builtin_bit_cast(uint32_t, w);
    }
  }
}

/* The values that eight codes stand for. */
template <int FMT>
__device__ __forceinline__ void mx_decode(const uint32_t (&code)[2], uint32_t byte, float (&x)[8]) {
  const float s = byte == 255 ? __uint_as_float(0x7fc00000u) : mx_scale(byte);
  f32x2 p[4];
  if constexpr (FMT == ZS_MX_E2M1) {
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[0], 1.0f, 0);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[0], 1.0f, 1);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[0], 1.0f, 2);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[0], 1.0f, 3);
  } else {
    p[0] = __builtin_amdgcn_cvt_pk_f32_fp8((int)code[0], false);
    p[1] = __builtin_amdgcn_cvt_pk_f32_fp8((int)code[0], true);
    p[2] = __builtin_amdgcn_cvt_pk_f32_fp8((int)code[1], false);
    p[3] = __builtin_amdgcn_cvt_pk_f32_fp8((int)code[1], true);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = p[j].x * s;
    x[2 * j + 1] = p[j].y * s;
  }
}

/* ------------------------------------------------------------------------
 * Eight elements of a row of `cols`. ONCE: loaded non-temporally, where no
 * one reads them again soon (norm of 16384 x 4096: 84 us plain, 82; its
 * gradient 113 and 110; bf16 8191 x 4096 along the columns 37 and 33). AL: the row is 16-byte aligned and cols
 * is a multiple of 8, so the eight are all there or none. Otherwise the row
 * may start at any element: eight that are there still move at once (the
 * memory unit takes unaligned vectors), the last few one by one; zeros past
 * the end.
 * ---------------------------------------------------------------------- */
struct __attribute__((packed, aligned(2))) Loose16 { uint32_t w[4]; };   /* 8 16-bit elements */
struct __attribute__((packed, aligned(4))) Loose32 { float x[8]; };

template <bool AL, bool ONCE = false>
__device__ __forceinline__ Raw16<8> load8_raw(const void *row, uint64_t col, uint64_t cols) {
  Raw16<8> r = {};
  const uint16_t *p = static_cast<const uint16_t *>(row) + col;
  if constexpr (AL) {
    if (col < cols) r = ld16<8, ONCE>(p);
  } else if (col + 8 <= cols) {
    const Loose16 v = *reinterpret_cast<const Loose16 *>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[j] = v.w[j];
  } else if (col < cols) {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (col + j < cols) r.w[j / 2] |= (uint32_t)p[j] << (16 * (j & 1));
  }
  return r;
}

template <int DT, bool AL, bool ONCE = false>
__device__ __forceinline__ void load8(const void *row, uint64_t col, uint64_t cols, float (&x)[8]) {
  if constexpr (DT != ZS_FP32) {
    upcast<8, DT>(load8_raw<AL, ONCE>(row, col, cols), x);
  } else {
    const float *p = static_cast<const float *>(row) + col;
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    if constexpr (AL) {
      if (col < cols) ldf_p<8, ONCE>(p, x);
    } else if (col + 8 <= cols) {
      const Loose32 v = *reinterpret_cast<const Loose32 *>(p);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = v.x[j];
    } else if (col < cols) {
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (col + j < cols) x[j] = p[j];
    }
  }
}

/* Eight 16-bit elements of a row; LATER: stored non-temporally, past the
 * caches, which what is read next keeps then. */
template <bool AL, bool LATER = false>
__device__ __forceinline__ void store8_raw(uint16_t *row, uint64_t col, uint64_t cols,
                                           const u32x4 &w) {
  if constexpr (AL) {
    u32x4 *p = reinterpret_cast<u32x4 *>(row + col);
    if (col < cols) {
      if constexpr (LATER) __builtin_nontemporal_store(w, p);
      else *p = w;
    }
  } else if (col + 8 <= cols) {
    *reinterpret_cast<Loose16 *>(row + col) = Loose16{{w.x, w.y, w.z, w.w}};
  } else if (col < cols) {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (col + j < cols) row[col + j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
  }
}

/* The same, rounded to nearest even. */
template <int DT, bool AL, bool LATER = false>
__device__ __forceinline__ void store8(uint16_t *row, uint64_t col, uint64_t cols,
                                       const float (&x)[8]) {
  store8_raw<AL, LATER>(row, col, cols, u32x4{pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]),
                                              pack2<DT>(x[4], x[5]), pack2<DT>(x[6], x[7])});
}

/* Sum over the G threads of a row's group, on all of them; a fixed tree, so
 * the same inputs give the same bits. `part`: G / 64 values in LDS; the
 * caller uses another part of it, or waits, before the next call. */
template <int G, class T>
__device__ __forceinline__ T group_sum(T v, T *part) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
  if constexpr (G > 64) {
    const int wave = (int)(threadIdx.x >> 6);
    if ((threadIdx.x & 63) == 0) part[wave] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < G / 64; ++w) v += part[w];
  }
  return v;
}

}  // namespace zs
#endif  // ZS_MX_H
