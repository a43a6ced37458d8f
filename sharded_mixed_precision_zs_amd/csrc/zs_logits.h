/*
 * zs_logits.h -- what the losses over rows of logits share (gfx950): elements
 * and 16-byte vectors of a row at any alignment, reductions over a block, and
 * the terms of a softmax.
 */
#ifndef ZS_LOGITS_H
#define ZS_LOGITS_H

#include "zs_mx.h"

namespace zs {

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

template <int DT>
__device__ __forceinline__ float load1(const void *p, uint64_t i) {
  if constexpr (DT == ZS_FP32) return static_cast<const float *>(p)[i];
  else return up_lo<DT>(static_cast<const uint16_t *>(p)[i]);
}

/* An element as it lies in memory, and its value: apart, so that nothing
 * waits for the element before its value is used. */
template <int DT>
__device__ __forceinline__ uint32_t load_raw(const void *p, uint64_t i) {
  if constexpr (DT == ZS_FP32) return static_cast<const uint32_t *>(p)[i];
  else return static_cast<const uint16_t *>(p)[i];
}

template <int DT>
__device__ __forceinline__ float raw_value(uint32_t w) {
  if constexpr (DT == ZS_FP32) return __uint_as_float(w);
  else return up_lo<DT>(w);
}

/* A value that nothing writes while the kernel runs, by the scalar unit:
 * vector loads return in order, and this one must not wait for a row. */
__device__ __forceinline__ float load_scalar(const float *p, uint32_t i) {
  return reinterpret_cast<const __attribute__((address_space(4))) float *>(
      reinterpret_cast<uintptr_t>(p))[i];
}

template <int DT>
__device__ __forceinline__ void store1(void *p, uint64_t i, float x) {
  if constexpr (DT == ZS_FP32) static_cast<float *>(p)[i] = x;
  else static_cast<uint16_t *>(p)[i] = pack1<DT>(x);
}

/* Elements per 16-byte vector. */
template <int DT>
constexpr uint32_t kVecElems = DT == ZS_FP32 ? 4 : 8;

template <int DT>
__device__ __forceinline__ void unpack_vec(const u32x4 &w, float (&x)[kVecElems<DT>]) {
  if constexpr (DT == ZS_FP32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(w[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = up_lo<DT>(w[j]);
      x[2 * j + 1] = up_hi<DT>(w[j]);
    }
  }
}

template <int DT>
__device__ __forceinline__ u32x4 pack_vec(const float (&x)[kVecElems<DT>]) {
  u32x4 w;
  if constexpr (DT == ZS_FP32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(x[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack2<DT>(x[2 * j], x[2 * j + 1]);
  }
  return w;
}

/* A row as whole 16-byte vectors between a few single elements at either
 * end, whatever the row's alignment. */
struct RowShape {
  uint32_t head, vecs, tail;   /* elements, vectors, elements */
};

template <int DT>
__device__ __forceinline__ RowShape row_shape(const void *row, uint32_t n) {
  constexpr uint32_t esz = DT == ZS_FP32 ? 4 : 2, ve = kVecElems<DT>;
  RowShape s;
  s.head = (uint32_t)((16 - ((uintptr_t)row & 15)) & 15) / esz;
  if (s.head > n) s.head = n;
  s.vecs = (n - s.head) / ve;
  s.tail = n - s.head - s.vecs * ve;
  return s;
}

/* The single element that thread t has besides its vectors: the head's in
 * threads 0 .. 7, the tail's in threads 8 .. 15; vocab if none. */
template <int DT>
__device__ __forceinline__ uint32_t edge_index(const RowShape &s, uint32_t t, bool first,
                                               bool last, uint32_t vocab) {
  if (first && t < s.head) return t;
  if (last && t >= 8 && t - 8 < s.tail) return s.head + s.vecs * kVecElems<DT> + t - 8;
  return vocab;
}

/* ------------------------------------------------------------------------
 * Reductions over a block: within each wave, then over the waves' results by
 * every wave alike; a fixed tree, on all threads. `part`: NT / 64 values that
 * nothing else uses before the next barrier.
 * ---------------------------------------------------------------------- */
struct MaxOf {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct SumOf {
  template <class T>
  __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};

/* A value of another lane of the same 16, by the lane pattern CTRL. */
template <int CTRL>
__device__ __forceinline__ float lane_move(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ double lane_move(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, CTRL, 0xf, 0xf, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), CTRL, 0xf, 0xf,
                                                         true);
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

/* Within groups of `width` lanes: neighbours, pairs, then the mirrored half
 * of 8 and of 16 lanes (equal within each half by then), then across. */
template <class T, class Op>
__device__ __forceinline__ T wave_reduce(T v, Op op, int width) {
  v = op(v, lane_move<0xB1>(v));
  v = op(v, lane_move<0x4E>(v));
  if (width > 4) v = op(v, lane_move<0x141>(v));
  if (width > 8) v = op(v, lane_move<0x140>(v));
  if (width > 16) v = op(v, __shfl_xor(v, 16, 64));
  if (width > 32) v = op(v, __shfl_xor(v, 32, 64));
  return v;
}

/* Before the barrier: the wave's result; after it: the block's. */
template <class T, class Op>
__device__ __forceinline__ void reduce_put(T v, Op op, T *part) {
  v = wave_reduce(v, op, 64);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
}

template <int NT, class T, class Op>
__device__ __forceinline__ T reduce_get(Op op, const T *part) {
  if constexpr (NT == 64) return part[0];
  if constexpr (NT == 128) return op(part[0], part[1]);
  return wave_reduce(part[threadIdx.x & (NT / 64 - 1)], op, NT / 64);
}

/* ------------------------------------------------------------------------
 * Terms. A maximum of -inf (nothing but -inf) counts as 0, so that such
 * terms are 0 and a NaN stays one.
 *
 * From 2^24 exponent units on, reached by large logits or a small temperature,
 * fp32 has no whole number next to max c: they lie up to 2^(e - 24) apart, and
 * terms would be off by half of that in their exponents. Neighbouring 16-bit
 * values lie 2^12 units and more apart there, so that terms are 1 or 0 by any
 * c: one that is a power of two and makes max c a whole number of 24 bits
 * does. Of fp32's, whose neighbours may lie 1 apart, the difference is taken
 * off each exponent; from 2^32 on they too are 2^8 apart.
 * ---------------------------------------------------------------------- */
struct Shift {
  float max, c, whole;
  float frac;   /* of fp32's exponents, off each: max c - whole from 2^24 on, else 0 */
  float rest;   /* ln 2 * (max c - whole - frac) */
};

template <int DT>
__device__ __forceinline__ Shift shift_of(float max, float c) {
  constexpr float kWhole = 16777216.0f, kFar = DT == ZS_FP32 ? 4294967296.0f : kWhole;
  constexpr uint32_t kTop = DT == ZS_FP32 ? 32 : 23;   /* |max c| in [2^kTop, 2^(kTop + 1)) then */
  Shift s;
  s.max = max == -INFINITY ? 0.0f : max;
  s.c = c;
  s.frac = 0.0f;
  if (fabsf(s.max * c) < kFar) {
    s.whole = rintf(s.max * c);
    if (DT == ZS_FP32 && fabsf(s.whole) >= kWhole) s.frac = fmaf(s.max, c, -s.whole);
  } else {   /* c is below 2^127, so that a max of fp32 is above 2^-95; or it is no number */
    s.c = __uint_as_float((254 + kTop - (__float_as_uint(s.max) >> 23 & 255)) << 23);
    s.whole = s.max * s.c;
  }
  s.rest = (fmaf(s.max, s.c, -s.whole) - s.frac) * 0.69314718f;
  return s;
}

template <int DT>
__device__ __forceinline__ float term(float z, const Shift &s) {
  const float e = fmaf(z, s.c, -s.whole);
  return exp2_fast(DT == ZS_FP32 ? e - s.frac : e);
}

/* What turns a sum of terms by shift `own`, 2^lift too large, into one by shift
 * `to`: a power of two, but for a difference of fracs; 0 where the two have
 * another c, and so no terms in common, or lie too far apart. */
template <int DT>
__device__ __forceinline__ double shift_factor(const Shift &own, const Shift &to, float lift) {
  float by = own.whole - to.whole - lift, part = 0.0f;
  if constexpr (DT == ZS_FP32) {
    by += own.frac - to.frac;
    part = by;
    by = floorf(by);
    part -= by;
  }
  const double f = __hiloint2double(own.c == to.c && by > -900.0f ? (1023 + (int)by) << 20 : 0, 0);
  return DT == ZS_FP32 ? f * (double)exp2_fast(part) : f;
}

template <int DT>
__device__ __forceinline__ u32x4 empty_vec() {   /* -inf */
  const uint32_t w = DT == ZS_FP32 ? 0xff800000u : DT == ZS_BF16 ? 0xff80ff80u : 0xfc00fc00u;
  return u32x4{w, w, w, w};
}

/* A buffer that hardware checks the bounds of: reads past `bytes` give 0 and
 * writes there are dropped, without a branch in the code. Only the vector
 * offset is checked, so all of an offset goes there. The description is that
 * of plain 32-bit data. */
__device__ __forceinline__ __amdgpu_buffer_rsrc_t bounded(const void *p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, (int)bytes, 0x00027000);
}

/* Running maximum of whole vectors. Written in instructions for two reasons:
 * the compiler would quiet every operand first, and it would carry the
 * values unpacked here to the sums, at twice the registers. What a NaN does
 * to the row, its sum does anyway. */
template <int DT>
struct VecMax {
  uint32_t m = DT == ZS_FP16 ? 0xfc00fc00u : 0xff800000u;   /* -inf, two of them in fp16 */

  __device__ __forceinline__ void add(const u32x4 &x) {
    if constexpr (DT == ZS_FP16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) asm("v_pk_max_f16 %0, %0, %1" : "+v"(m) : "v"(x[j]));
    } else if constexpr (DT == ZS_FP32) {
#pragma unroll
      for (int j = 0; j < 4; j += 2)
        asm("v_max3_f32 %0, %0, %1, %2" : "+v"(m) : "v"(x[j]), "v"(x[j + 1]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t lo, hi;
        asm("v_lshlrev_b32 %0, 16, %1" : "=v"(lo) : "v"(x[j]));
        asm("v_and_b32 %0, 0xffff0000, %1" : "=v"(hi) : "v"(x[j]));
        asm("v_max3_f32 %0, %0, %1, %2" : "+v"(m) : "v"(lo), "v"(hi));
      }
    }
  }

  __device__ __forceinline__ float get() const {
    if constexpr (DT == ZS_FP16) return fmaxf(up_lo<DT>(m), up_hi<DT>(m));
    else return __uint_as_float(m);
  }
};

}  // namespace zs
#endif  // ZS_LOGITS_H
