/*
 * zs_distill_kernels.h -- loss against a teacher's top logits and its
 * gradient (gfx950).
 *
 * With u = z / tau, q = softmax(u), S = sum exp(u - max u) and p the
 * teacher's probabilities on its slots, a row's gradient is a multiple of
 * q - p: every logit gets exp(u - max u) * coef / S in one sweep, and the few
 * slots are written again afterwards by the threads that hold them. Slots of
 * the same token add up: each writes the same sum.
 *
 * With the teacher's logsumexp over its whole vocabulary, the mass that it
 * has off the slots, pr, meets the student's, qr, as one more outcome; off
 * the slots the gradient is then q * (1 - pr / qr). qr = (S - sum of the
 * slots' terms) / S: both sums are kept in binary64 over the same fp32 terms,
 * so what cancels cancels exactly, however little is left.
 *
 * Bound by HBM: logits in, gradient out.
 */
#ifndef ZS_DISTILL_KERNELS_H
#define ZS_DISTILL_KERNELS_H

#include "zs_mx.h"

namespace zs {

constexpr uint32_t kMaxSlots = ZS_DISTILL_MAX_SLOTS;

/* Statistics of one part of a row: maximum and sum of exp(u - max). */
struct DistillPart {
  double sum;
  float max;
  float unused;
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

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor(v, m, 64));
  return v;
}

template <class T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

/* Maximum and sum over the block's NT threads; `part`: NT / 64 values. */
template <int NT>
__device__ __forceinline__ float block_max(float v, float *part) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) v = fmaxf(v, part[w]);
  return v;
}

template <int NT, class T>
__device__ __forceinline__ T block_sum(T v, T *part) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) v += part[w];
  return v;
}

/* exp(u - max) as every kernel here forms it. A maximum of -inf (nothing
 * but -inf) counts as 0, so that such terms are 0 and a NaN stays one. */
__device__ __forceinline__ float shifted(float max) { return max == -INFINITY ? 0.0f : max; }

__device__ __forceinline__ float term(float z, float max, float log2_scale) {
  return exp2_fast((z - max) * log2_scale);
}

/* ------------------------------------------------------------------------
 * The slots of one row, by a whole block of NT threads: the teacher's
 * probabilities and what the loss sums over them.
 * ---------------------------------------------------------------------- */
struct SlotSums {
  float mass;     /* sum of w */
  float cross;    /* sum of w * ((t - ref) - (u - max u)) */
  double terms;   /* sum of the distinct slots' exp(u - max u) */
  float ref;
  bool live;      /* the row has a slot with mass */
};

template <int NT>
struct SlotLds {
  int32_t id[kMaxSlots];
  float w[kMaxSlots], z[kMaxSlots];
  float part[4][NT / 64];
  double dpart[NT / 64];
};

/* The slots' logits come from `slot_z` where that is given: the gradient may
 * be written over the logits, and another block may have begun to. */
template <int DT, bool TAIL, int NT>
__device__ __forceinline__ SlotSums slot_sums(const DistillArgs &a, uint64_t row, const void *z,
                                              const float *slot_z, float max, SlotLds<NT> &s) {
  SlotSums r;
  const float inv_tau = a.inv_tau;
  const uint64_t base = row * a.slots;
  float top = -INFINITY, any = 0.0f;
  for (uint32_t k = threadIdx.x; k < a.slots; k += NT) {
    const int32_t id = a.ids[base + k];
    const bool ok = id >= 0 && (uint32_t)id < a.vocab;
    const float t = ok ? load1<DT>(a.teacher, base + k) * inv_tau : -INFINITY;
    s.id[k] = ok ? id : -1;
    s.w[k] = t;
    s.z[k] = !ok ? 0.0f : slot_z ? slot_z[base + k] : load1<DT>(z, id);
    if (ok) any = 1.0f;
    top = fmaxf(top, t != t ? INFINITY : t);
  }
  top = block_max<NT>(top, s.part[0]);
  any = block_max<NT>(any, s.part[1]);
  if constexpr (TAIL) {
    r.ref = a.lse[row];
    r.live = any > 0.0f;
  } else {
    r.ref = top;
    r.live = top > -INFINITY;
  }
  float mass = 0.0f, cross = 0.0f;
  double terms = 0.0;
  for (uint32_t k = threadIdx.x; k < a.slots; k += NT) {
    const int32_t id = s.id[k];
    if (id < 0) {
      s.w[k] = 0.0f;
      continue;
    }
    const float t = s.w[k], zk = s.z[k];
    const float w = exp2_fast((t - r.ref) * 1.44269504f);
    mass += w;
    if (!(w == 0.0f)) cross += w * ((t - r.ref) - (zk - max) * inv_tau);
    if constexpr (TAIL) {
      bool seen = false;
      for (uint32_t j = 0; j < k; ++j) seen |= s.id[j] == id;
      if (!seen) terms += (double)term(zk, max, a.log2_scale);
    }
    s.w[k] = w;
  }
  r.mass = block_sum<NT>(mass, s.part[2]);
  r.cross = block_sum<NT>(cross, s.part[3]);
  r.terms = 0.0;
  if constexpr (TAIL) r.terms = block_sum<NT>(terms, s.dpart);
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
__device__ __forceinline__ RowResult row_result(const SlotSums &s, double sum) {
  RowResult r;
  const float total = (float)sum;
  if constexpr (TAIL) {
    r.loss = s.cross + s.mass * logf(total);
    float pr = 1.0f - s.mass;
    pr = pr >= kTailFloor ? pr : 0.0f;   /* NaN mass: the loss is NaN already */
    const double rest = sum - s.terms;
    const float qr = rest > 0.0 ? (float)(rest / sum) : 0.0f;
    if (pr > 0.0f) r.loss += pr * (logf(pr) - logf(qr));
    /* nothing off the slots: every such term is 0 whatever its factor */
    r.off = qr > 0.0f ? 1.0f - pr / qr : 1.0f;
  } else {
    r.loss = s.cross / s.mass - logf(s.mass) + logf(total);
    r.off = 1.0f;
  }
  return r;
}

/* The slots' gradients, after the sweep over the row (and a barrier): this
 * block's share [first, last) of the vocabulary. */
template <int DT, bool TAIL, int NT>
__device__ __forceinline__ void store_slots(const DistillArgs &a, void *g, const SlotLds<NT> &s,
                                            float max, float total, float mass, float coef,
                                            uint32_t first, uint32_t last) {
  for (uint32_t k = threadIdx.x; k < a.slots; k += NT) {
    const int32_t id = s.id[k];
    if (id < 0 || (uint32_t)id < first || (uint32_t)id >= last) continue;
    float w = 0.0f;
    for (uint32_t j = 0; j < a.slots; ++j) w += s.id[j] == id ? s.w[j] : 0.0f;
    const float p = TAIL ? w : w / mass;
    store1<DT>(g, id, (term(s.z[k], max, a.log2_scale) / total - p) * coef);
  }
}

/* ------------------------------------------------------------------------
 * Rows in parts: a block per part forms its statistics, then a block per
 * part joins all of its row's and writes its share of the gradient.
 * ---------------------------------------------------------------------- */
template <int DT, bool TAIL, int NT>
__global__ __launch_bounds__(NT) void distill_stats_kernel(DistillArgs a) {
  constexpr uint32_t ve = kVecElems<DT>;
  __shared__ float fpart[2][NT / 64];
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
  max = block_max<NT>(max, fpart[0]);
  const float m = shifted(max);
  double sum = edge < a.vocab ? (double)term(load1<DT>(z, edge), m, a.log2_scale) : 0.0;
  for (uint32_t v = v0 + threadIdx.x; v < v1; v += NT) {
    float x[ve];
    unpack_vec<DT>(zv[v], x);
#pragma unroll
    for (uint32_t j = 0; j < ve; ++j) sum += (double)term(x[j], m, a.log2_scale);
  }
  sum = block_sum<NT>(sum, dpart);
  if (threadIdx.x == 0) a.ws[blockIdx.x] = {sum, max, 0.0f};
  if (part != 0) return;
  for (uint32_t k = threadIdx.x; k < a.slots; k += NT) {
    const int32_t id = a.ids[row * a.slots + k];
    if (id >= 0 && (uint32_t)id < a.vocab) a.ws_z[row * a.slots + k] = load1<DT>(z, id);
  }
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
  bool live = weight != 0.0f;
  float max = -INFINITY, total = 1.0f, factor = 0.0f, coef = 0.0f;
  SlotSums s{};
  if (live) {
    const DistillPart *w = a.ws + row * a.parts;
    for (uint32_t i = 0; i < a.parts; ++i) max = fmaxf(max, w[i].max);
    max = shifted(max);
    double sum = 0.0;
    for (uint32_t i = 0; i < a.parts; ++i)
      sum += w[i].sum * (double)term(shifted(w[i].max), max, a.log2_scale);
    s = slot_sums<DT, TAIL, NT>(a, row, z, a.ws_z, max, lds);
    live = s.live;
    const RowResult r = row_result<TAIL>(s, sum);
    total = (float)sum;
    coef = (a.dev ? a.dev->scale : a.scale) * a.tau * weight;
    factor = coef * r.off / total;
    if (first && threadIdx.x == 0) a.loss[row] = live ? weight * a.tau * a.tau * r.loss : 0.0f;
  } else if (first && threadIdx.x == 0) {
    a.loss[row] = 0.0f;
  }
  if (!g) return;
  const u32x4 *zv = reinterpret_cast<const u32x4 *>(z + sh.head * esz);
  u32x4 *gv = reinterpret_cast<u32x4 *>(g + sh.head * esz);
  if (edge < a.vocab)
    store1<DT>(g, edge, live ? term(load1<DT>(z, edge), max, a.log2_scale) * factor : 0.0f);
  for (uint32_t v = v0 + threadIdx.x; v < v1; v += NT) {
    float x[ve];
    if (live) {
      unpack_vec<DT>(zv[v], x);
#pragma unroll
      for (uint32_t j = 0; j < ve; ++j) x[j] = term(x[j], max, a.log2_scale) * factor;
    } else {
#pragma unroll
      for (uint32_t j = 0; j < ve; ++j) x[j] = 0.0f;
    }
    if (a.vec_store) {
      gv[v] = pack_vec<DT>(x);
    } else {
#pragma unroll
      for (uint32_t j = 0; j < ve; ++j) store1<DT>(g, sh.head + v * ve + j, x[j]);
    }
  }
  __syncthreads();
  if (live)
    store_slots<DT, TAIL, NT>(a, g, lds, max, total, s.mass, coef,
                              first ? 0 : sh.head + v0 * ve,
                              last ? a.vocab : sh.head + v1 * ve);
}

}  // namespace zs
#endif  // ZS_DISTILL_KERNELS_H
