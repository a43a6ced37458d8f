/*
 * zs_distill_kernels.h -- loss against a teacher's top logits and its
 * gradient (gfx950).
 *
 * With u = z / tau, q = softmax(u) and p the teacher's probabilities on its
 * slots, a row's gradient is a multiple of q - p: every logit gets its term
 * times one factor in one sweep, and the few slots are written again
 * afterwards by the threads that hold them. Slots of the same token add up:
 * each writes the same sum.
 *
 * A term is 2^(z c - I), c = log2(e) / tau and I the whole number next to
 * max(z) c: one multiply-add whose only rounding is of the exponent itself.
 *
 * With the teacher's logsumexp over its whole vocabulary, the mass that it
 * has off the slots, pr, meets the student's, qr, as one more outcome; off
 * the slots the gradient is then q * (1 - pr / qr). qr = (S - sum of the
 * slots' terms) / S: both sums are kept in binary64 over the same fp32 terms,
 * so what cancels cancels exactly, however little is left.
 *
 * Bound by HBM: logits in, gradient out, once each where a block's registers
 * hold the row (distill_row_kernel).
 */
#ifndef ZS_DISTILL_KERNELS_H
#define ZS_DISTILL_KERNELS_H

#include "zs_mx.h"

namespace zs {

constexpr uint32_t kMaxSlots = ZS_DISTILL_MAX_SLOTS;

/* Statistics of one part of a row: maximum and sum of terms. */
struct DistillPart {
  double sum;
  float max;
  float pad;
};

struct DistillArgs {
  const void *z;
  const int32_t *ids;
  const void *teacher;
  const float *lse, *weight;       /* optional */
  const zs_device_scaler *dev;     /* optional: its scale in place of `scale` */
  float *loss;
  void *grad;                      /* optional */
  DistillPart *ws;                 /* rows in parts: [rows][parts] */
  float *ws_z;                     /* and their slots' logits: [rows][slots] */
  uint64_t rows, ld, gld;
  uint32_t vocab, slots, parts, part_vecs;
  float tau, inv_tau, log2_scale, scale;   /* log2_scale = log2(e) / tau */
  int vec_store;                   /* gradient rows are aligned as the logits' */
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

template <int DT>
__device__ __forceinline__ float load1(const void *p, uint64_t i) {
  if constexpr (DT == ZS_FP32) return static_cast<const float *>(p)[i];
  else return up_lo<DT>(static_cast<const uint16_t *>(p)[i]);
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

template <class T, class Op>
__device__ __forceinline__ T wave_reduce(T v, Op op, int width) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1)
    if (m < width) v = op(v, __shfl_xor(v, m, 64));
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
  return wave_reduce(part[threadIdx.x & (NT / 64 - 1)], op, NT / 64);
}

/* ------------------------------------------------------------------------
 * Terms. A maximum of -inf (nothing but -inf) counts as 0, so that such
 * terms are 0 and a NaN stays one. Beyond 2^60 in exponent units, where
 * z c could overflow, neighbouring values lie so far apart that any c gives
 * terms of 1 and 0: 2^-4 does.
 * ---------------------------------------------------------------------- */
struct Shift {
  float max, c, whole;
  float rest;   /* ln 2 * (max c - whole) */
};

__device__ __forceinline__ Shift shift_of(float max, float c) {
  Shift s;
  s.max = max == -INFINITY ? 0.0f : max;
  s.c = fabsf(s.max * c) < 1.15292150e18f ? c : 0.0625f;
  s.whole = rintf(s.max * s.c);
  s.rest = fmaf(s.max, s.c, -s.whole) * 0.69314718f;
  return s;
}

__device__ __forceinline__ float term(float z, const Shift &s) {
  return exp2_fast(fmaf(z, s.c, -s.whole));
}

/* ------------------------------------------------------------------------
 * The slots of one row, by a whole block of NT threads: the teacher's
 * probabilities and what the loss sums over them.
 * ---------------------------------------------------------------------- */
template <int NT>
struct SlotLds {
  int32_t id[kMaxSlots];
  float w[kMaxSlots], z[kMaxSlots];
  float part[5][NT / 64];
  double dpart[2][NT / 64];
};

/* Ids and the teacher's logits over the temperature; returns their maximum
 * (+inf for a NaN) and whether a slot is filled. */
struct SlotTop {
  float top, any;
};

template <int DT, int NT>
__device__ __forceinline__ SlotTop slot_ids(const DistillArgs &a, uint64_t row, SlotLds<NT> &s) {
  SlotTop r{-INFINITY, 0.0f};
  for (uint32_t k = threadIdx.x; k < a.slots; k += NT) {
    const int32_t id = a.ids[row * a.slots + k];
    const bool ok = id >= 0 && (uint32_t)id < a.vocab;
    const float t = ok ? load1<DT>(a.teacher, row * a.slots + k) * a.inv_tau : -INFINITY;
    s.id[k] = ok ? id : -1;
    s.w[k] = t;
    if (ok) r.any = 1.0f;
    r.top = fmaxf(r.top, t != t ? INFINITY : t);
  }
  return r;
}

/* The slots' logits: from `saved` where that is given (the gradient may be
 * written over the logits, and another block may have begun to). */
template <int DT, int NT>
__device__ __forceinline__ void slot_logits(const DistillArgs &a, uint64_t row, const void *z,
                                            const float *saved, SlotLds<NT> &s) {
  for (uint32_t k = threadIdx.x; k < a.slots; k += NT) {
    const int32_t id = s.id[k];
    s.z[k] = id < 0 ? 0.0f : saved ? saved[row * a.slots + k] : load1<DT>(z, id);
  }
}

struct SlotSums {
  float mass;     /* sum of w */
  float cross;    /* sum of w * ((t - ref) - (u - max u)) */
  double terms;   /* sum of the distinct slots' terms */
};

/* This thread's share; weights w = exp(t - ref) take the logits' place.
 * All ids are in LDS before this. `term_of(token, logit)`: the token's term
 * with the very bits that it has in the row's sum. */
template <bool TAIL, int NT, class F>
__device__ __forceinline__ SlotSums slot_weights(const DistillArgs &a, float ref, const Shift &sh,
                                                 SlotLds<NT> &s, F term_of) {
  SlotSums r{0.0f, 0.0f, 0.0};
  for (uint32_t k = threadIdx.x; k < a.slots; k += NT) {
    const int32_t id = s.id[k];
    float w = 0.0f;
    if (id >= 0) {
      const float t = s.w[k], zk = s.z[k];
      w = exp2_fast((t - ref) * 1.44269504f);
      r.mass += w;
      if (!(w == 0.0f)) r.cross += w * ((t - ref) - (zk - sh.max) * a.inv_tau);
      if constexpr (TAIL) {
        bool seen = false;
        for (uint32_t j = 0; j < k; ++j) seen |= s.id[j] == id;
        if (!seen) r.terms += term_of((uint32_t)id, zk);
      }
    }
    s.w[k] = w;
  }
  return r;
}

/* The teacher's mass off its slots counts as none below 2^-20: its fp32
 * logsumexp does not say more, and against a student without such mass the
 * rounding's remainder would make the loss infinite. */
constexpr float kTailFloor = 9.5367431640625e-7f;

/* Loss of a row (without its weight and tau^2) and the factor of the
 * logits off the slots. */
struct RowResult {
  float loss, off;
};

template <bool TAIL>
__device__ __forceinline__ RowResult row_result(const SlotSums &s, const Shift &sh, double sum) {
  RowResult r;
  const float log_total = logf((float)sum) - sh.rest;   /* of the terms by the maximum */
  if constexpr (TAIL) {
    r.loss = s.cross + s.mass * log_total;
    float pr = 1.0f - s.mass;
    pr = pr >= kTailFloor ? pr : 0.0f;   /* NaN mass: the loss is NaN already */
    const double rest = sum - s.terms;
    const float qr = rest > 0.0 ? (float)(rest / sum) : 0.0f;
    if (pr > 0.0f) r.loss += pr * (logf(pr) - logf(qr));
    /* nothing off the slots: every such term is 0 whatever its factor */
    r.off = qr > 0.0f ? 1.0f - pr / qr : 1.0f;
  } else {
    r.loss = s.cross / s.mass - logf(s.mass) + log_total;
    r.off = 1.0f;
  }
  return r;
}

/* The slots' gradients, after the sweep over the row (and a barrier): this
 * block's share [first, last) of the vocabulary. */
template <int DT, bool TAIL, int NT>
__device__ __forceinline__ void store_slots(const DistillArgs &a, void *g, const SlotLds<NT> &s,
                                            const Shift &sh, float total, float mass, float coef,
                                            uint32_t first, uint32_t last) {
  for (uint32_t k = threadIdx.x; k < a.slots; k += NT) {
    const int32_t id = s.id[k];
    if (id < 0 || (uint32_t)id < first || (uint32_t)id >= last) continue;
    float w = 0.0f;
    for (uint32_t j = 0; j < a.slots; ++j) w += s.id[j] == id ? s.w[j] : 0.0f;
    const float p = TAIL ? w : w / mass;
    store1<DT>(g, id, (term(s.z[k], sh) / total - p) * coef);
  }
}

/* What a row's sweep multiplies by. */
struct RowFactors {
  float total, coef, factor;
  bool live;
};

/* From the joined sums: the row's loss (stored by the thread that `says`)
 * and its factors. */
template <bool TAIL>
__device__ __forceinline__ RowFactors finish_row(const DistillArgs &a, uint64_t row, float weight,
                                                 bool live, const SlotSums &s, const Shift &sh,
                                                 double sum, bool says) {
  const RowResult r = row_result<TAIL>(s, sh, sum);
  RowFactors f;
  f.live = live;
  f.total = (float)sum;
  f.coef = (a.dev ? a.dev->scale : a.scale) * a.tau * weight;
  f.factor = f.coef * r.off / f.total;
  if (says) a.loss[row] = live ? weight * a.tau * a.tau * r.loss : 0.0f;
  return f;
}

/* A vector of terms times the factor, or zeros. */
template <int DT>
__device__ __forceinline__ void store_grad(const DistillArgs &a, char *g, uint32_t head, uint32_t v,
                                           const float (&x)[kVecElems<DT>]) {
  constexpr uint32_t ve = kVecElems<DT>;
  constexpr uint32_t esz = DT == ZS_FP32 ? 4 : 2;
  if (a.vec_store) {
    *reinterpret_cast<u32x4 *>(g + (head + (uint64_t)v * ve) * esz) = pack_vec<DT>(x);
  } else {
#pragma unroll
    for (uint32_t j = 0; j < ve; ++j) store1<DT>(g, head + (uint64_t)v * ve + j, x[j]);
  }
}

/* Keeps the compiler from carrying unpacked values from one sweep over the
 * registers to the next, which would take twice the registers. */
template <int ITEMS>
__device__ __forceinline__ void unpack_again(u32x4 (&x)[ITEMS]) {
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) asm volatile("" : "+v"(x[i]));
}

/* A thread's sum of terms: binary64 where slots' terms are taken out of it. */
template <bool TAIL>
struct Sum { typedef float type; };
template <>
struct Sum<true> { typedef double type; };

/* ------------------------------------------------------------------------
 * A row per block, held in registers between its statistics and its
 * gradient: ITEMS 16-byte vectors per thread and, in a few threads, one
 * single element.
 * ---------------------------------------------------------------------- */
template <int DT>
__device__ __forceinline__ u32x4 empty_vec() {   /* -inf */
  const uint32_t w = DT == ZS_FP32 ? 0xff800000u : DT == ZS_BF16 ? 0xff80ff80u : 0xfc00fc00u;
  return u32x4{w, w, w, w};
}

template <int DT, bool TAIL, int NT, int ITEMS>
__global__ __launch_bounds__(NT) void distill_row_kernel(DistillArgs a) {
  constexpr uint32_t ve = kVecElems<DT>, esz = DT == ZS_FP32 ? 4 : 2;
  __shared__ SlotLds<NT> lds;
  const uint64_t row = blockIdx.x;
  const uint32_t t = threadIdx.x;
  const char *z = static_cast<const char *>(a.z) + row * a.ld * esz;
  char *g = a.grad ? static_cast<char *>(a.grad) + row * a.gld * esz : nullptr;
  const float weight = a.weight ? a.weight[row] : 1.0f;
  const RowShape sh = row_shape<DT>(z, a.vocab);
  const uint32_t edge = edge_index<DT>(sh, t, true, true, a.vocab);
  u32x4 x[ITEMS];
  float single = -INFINITY;
  RowFactors f{1.0f, 0.0f, 0.0f, false};
  SlotSums sums{};
  Shift shift{};
  if (weight != 0.0f) {   /* uniform over the block */
    const SlotTop top = slot_ids<DT, NT>(a, row, lds);
    const u32x4 *zv = reinterpret_cast<const u32x4 *>(z + sh.head * esz);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const uint32_t v = i * NT + t;
      x[i] = v < sh.vecs ? __builtin_nontemporal_load(zv + v) : empty_vec<DT>();
    }
    if (edge < a.vocab) single = load1<DT>(z, edge);
    slot_logits<DT, NT>(a, row, z, nullptr, lds);
    float max = single;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      float e[ve];
      unpack_vec<DT>(x[i], e);
#pragma unroll
      for (uint32_t j = 0; j < ve; j += 2) max = fmaxf(max, fmaxf(e[j], e[j + 1]));
    }
    unpack_again(x);
    reduce_put(max, MaxOf{}, lds.part[0]);
    reduce_put(top.top, MaxOf{}, lds.part[1]);
    reduce_put(top.any, MaxOf{}, lds.part[2]);
    __syncthreads();
    shift = shift_of(reduce_get<NT>(MaxOf{}, lds.part[0]), a.log2_scale);
    const float highest = reduce_get<NT>(MaxOf{}, lds.part[1]);
    const float ref = TAIL ? a.lse[row] : highest;
    const bool live = TAIL ? reduce_get<NT>(MaxOf{}, lds.part[2]) > 0.0f : highest > -INFINITY;
    typename Sum<TAIL>::type sum = edge < a.vocab ? term(single, shift) : 0.0f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      float e[ve];
      unpack_vec<DT>(x[i], e);
#pragma unroll
      for (uint32_t j = 0; j < ve; ++j) sum += term(e[j], shift);
    }
    unpack_again(x);
    sums = slot_weights<TAIL, NT>(a, ref, shift, lds, [&](uint32_t, float zk) {
      return (double)term(zk, shift);
    });
    reduce_put(sums.mass, SumOf{}, lds.part[3]);
    reduce_put(sums.cross, SumOf{}, lds.part[4]);
    reduce_put((double)sum, SumOf{}, lds.dpart[0]);
    if constexpr (TAIL) reduce_put(sums.terms, SumOf{}, lds.dpart[1]);
    __syncthreads();
    sums.mass = reduce_get<NT>(SumOf{}, lds.part[3]);
    sums.cross = reduce_get<NT>(SumOf{}, lds.part[4]);
    if constexpr (TAIL) sums.terms = reduce_get<NT>(SumOf{}, lds.dpart[1]);
    f = finish_row<TAIL>(a, row, weight, live, sums, shift, reduce_get<NT>(SumOf{}, lds.dpart[0]),
                         t == 0);
  } else if (t == 0) {
    a.loss[row] = 0.0f;
  }
  if (!g) return;
  if (edge < a.vocab) store1<DT>(g, edge, f.live ? term(single, shift) * f.factor : 0.0f);
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const uint32_t v = i * NT + t;
    if (v >= sh.vecs) break;
    float e[ve];
    if (f.live) {
      unpack_vec<DT>(x[i], e);
#pragma unroll
      for (uint32_t j = 0; j < ve; ++j) e[j] = term(e[j], shift) * f.factor;
    } else {
#pragma unroll
      for (uint32_t j = 0; j < ve; ++j) e[j] = 0.0f;
    }
    store_grad<DT>(a, g, sh.head, v, e);
  }
  __syncthreads();
  if (f.live)
    store_slots<DT, TAIL, NT>(a, g, lds, shift, f.total, sums.mass, f.coef, 0, a.vocab);
}

/* ------------------------------------------------------------------------
 * Rows in parts, where there are few rows or a row is longer than a block's
 * registers: a block per part forms its statistics, then a block per part
 * joins all of its row's and writes its share of the gradient.
 * ---------------------------------------------------------------------- */
template <int DT, int NT>
__global__ __launch_bounds__(NT) void distill_stats_kernel(DistillArgs a) {
  constexpr uint32_t ve = kVecElems<DT>;
  __shared__ float fpart[NT / 64];
  __shared__ double dpart[NT / 64];
  const uint64_t row = blockIdx.x / a.parts;
  const uint32_t part = blockIdx.x % a.parts;
  if (a.weight && a.weight[row] == 0.0f) return;
  constexpr uint64_t esz = DT == ZS_FP32 ? 4 : 2;
  const char *z = static_cast<const char *>(a.z) + row * a.ld * esz;
  const RowShape sh = row_shape<DT>(z, a.vocab);
  const u32x4 *zv = reinterpret_cast<const u32x4 *>(z + sh.head * esz);
  const uint32_t v0 = part * a.part_vecs;
  const uint32_t v1 = v0 + a.part_vecs < sh.vecs ? v0 + a.part_vecs : sh.vecs;
  const uint32_t edge = edge_index<DT>(sh, threadIdx.x, part == 0, part == a.parts - 1, a.vocab);
  float max = edge < a.vocab ? load1<DT>(z, edge) : -INFINITY;
  for (uint32_t v = v0 + threadIdx.x; v < v1; v += NT) {
    float x[ve];
    unpack_vec<DT>(zv[v], x);
#pragma unroll
    for (uint32_t j = 0; j < ve; ++j) max = fmaxf(max, x[j]);
  }
  reduce_put(max, MaxOf{}, fpart);
  __syncthreads();
  max = reduce_get<NT>(MaxOf{}, fpart);
  const Shift shift = shift_of(max, a.log2_scale);
  double sum = edge < a.vocab ? (double)term(load1<DT>(z, edge), shift) : 0.0;
  for (uint32_t v = v0 + threadIdx.x; v < v1; v += NT) {
    float x[ve];
    unpack_vec<DT>(zv[v], x);
#pragma unroll
    for (uint32_t j = 0; j < ve; ++j) sum += (double)term(x[j], shift);
  }
  reduce_put(sum, SumOf{}, dpart);
  __syncthreads();
  sum = reduce_get<NT>(SumOf{}, dpart);
  if (threadIdx.x == 0) a.ws[blockIdx.x] = {sum, max, 0.0f};
  if (part != 0) return;
  for (uint32_t k = threadIdx.x; k < a.slots; k += NT) {
    const int32_t id = a.ids[row * a.slots + k];
    if (id >= 0 && (uint32_t)id < a.vocab) a.ws_z[row * a.slots + k] = load1<DT>(z, id);
  }
}

/* What turns a part's terms into the row's. They are by its own whole
 * number, so the factor is a power of two and exact; where the two scale
 * differently (beyond 2^60) the part has no terms worth the name. A part of
 * nothing but -inf has the sum 0. */
__device__ __forceinline__ double part_factor(float max, const Shift &row, float c) {
  if (max == -INFINITY) return 1.0;
  const Shift own = shift_of(max, c);
  return (double)exp2_fast(own.c == row.c ? own.whole - row.whole : -INFINITY);
}

template <int DT, bool TAIL, int NT>
__global__ __launch_bounds__(NT) void distill_grad_kernel(DistillArgs a, uint32_t blocks) {
  constexpr uint32_t ve = kVecElems<DT>;
  __shared__ SlotLds<NT> lds;
  const uint64_t row = blockIdx.x / blocks;   /* blocks: parts, or 1 without a gradient */
  const uint32_t part = blockIdx.x % blocks;
  constexpr uint64_t esz = DT == ZS_FP32 ? 4 : 2;
  const char *z = static_cast<const char *>(a.z) + row * a.ld * esz;
  char *g = a.grad ? static_cast<char *>(a.grad) + row * a.gld * esz : nullptr;
  const float weight = a.weight ? a.weight[row] : 1.0f;
  const RowShape sh = row_shape<DT>(z, a.vocab);
  const uint32_t v0 = part * a.part_vecs;
  const uint32_t v1 = v0 + a.part_vecs < sh.vecs ? v0 + a.part_vecs : sh.vecs;
  const bool first = part == 0, last = part == a.parts - 1;
  const uint32_t edge = edge_index<DT>(sh, threadIdx.x, first, last, a.vocab);
  RowFactors f{1.0f, 0.0f, 0.0f, false};
  Shift shift{};
  SlotSums sums{};
  if (weight != 0.0f) {
    const DistillPart *w = a.ws + row * a.parts;
    float max = -INFINITY;
    for (uint32_t i = 0; i < a.parts; ++i) max = fmaxf(max, w[i].max);
    shift = shift_of(max, a.log2_scale);
    double sum = 0.0;
    for (uint32_t i = 0; i < a.parts; ++i)
      sum += w[i].sum * part_factor(w[i].max, shift, a.log2_scale);
    const SlotTop top = slot_ids<DT, NT>(a, row, lds);
    slot_logits<DT, NT>(a, row, z, a.ws_z, lds);
    reduce_put(top.top, MaxOf{}, lds.part[1]);
    reduce_put(top.any, MaxOf{}, lds.part[2]);
    __syncthreads();
    const float highest = reduce_get<NT>(MaxOf{}, lds.part[1]);
    const float ref = TAIL ? a.lse[row] : highest;
    const bool live = TAIL ? reduce_get<NT>(MaxOf{}, lds.part[2]) > 0.0f : highest > -INFINITY;
    sums = slot_weights<TAIL, NT>(a, ref, shift, lds, [&](uint32_t id, float zk) {
      uint32_t i = id < sh.head ? 0 : (id - sh.head) / ve / a.part_vecs;
      i = i < a.parts ? i : a.parts - 1;
      return (double)term(zk, shift_of(w[i].max, a.log2_scale)) *
             part_factor(w[i].max, shift, a.log2_scale);
    });
    reduce_put(sums.mass, SumOf{}, lds.part[3]);
    reduce_put(sums.cross, SumOf{}, lds.part[4]);
    if constexpr (TAIL) reduce_put(sums.terms, SumOf{}, lds.dpart[1]);
    __syncthreads();
    sums.mass = reduce_get<NT>(SumOf{}, lds.part[3]);
    sums.cross = reduce_get<NT>(SumOf{}, lds.part[4]);
    if constexpr (TAIL) sums.terms = reduce_get<NT>(SumOf{}, lds.dpart[1]);
    f = finish_row<TAIL>(a, row, weight, live, sums, shift, sum, first && threadIdx.x == 0);
  } else if (first && threadIdx.x == 0) {
    a.loss[row] = 0.0f;
  }
  if (!g) return;
  const u32x4 *zv = reinterpret_cast<const u32x4 *>(z + sh.head * esz);
  if (edge < a.vocab)
    store1<DT>(g, edge, f.live ? term(load1<DT>(z, edge), shift) * f.factor : 0.0f);
  for (uint32_t v = v0 + threadIdx.x; v < v1; v += NT) {
    float x[ve];
    if (f.live) {
      unpack_vec<DT>(zv[v], x);
#pragma unroll
      for (uint32_t j = 0; j < ve; ++j) x[j] = term(x[j], shift) * f.factor;
    } else {
#pragma unroll
      for (uint32_t j = 0; j < ve; ++j) x[j] = 0.0f;
    }
    store_grad<DT>(a, g, sh.head, v, x);
  }
  __syncthreads();
  if (f.live)
    store_slots<DT, TAIL, NT>(a, g, lds, shift, f.total, sums.mass, f.coef,
                              first ? 0 : sh.head + v0 * ve,
                              last ? a.vocab : sh.head + v1 * ve);
}

}  // namespace zs
#endif  // ZS_DISTILL_KERNELS_H
