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
 * the slots the gradient is then q * (1 - pr / qr). However little qr is, its
 * sum leaves the slots' terms out as they come (taking them off the whole sum
 * would leave rounding): a bit for each element in LDS says whether it is a
 * slot's. Where the sum is below 2^-40, the terms off the slots are formed
 * 2^96 larger, and so reach down to 2^-222 of the row's largest; what is
 * smaller counts as none. Gradients off the slots come from terms that are
 * scaled by their sum's power of two: neither 1 / qr nor pr / qr overflows.
 *
 * Bound by HBM: logits in, gradient out, once each where a block's registers
 * hold the row (distill_row_kernel), the logits twice or three times in parts.
 */
#ifndef ZS_DISTILL_KERNELS_H
#define ZS_DISTILL_KERNELS_H

#include "zs_logits.h"

namespace zs {

constexpr uint32_t kMaxSlots = ZS_DISTILL_MAX_SLOTS;

/* Statistics of one part of a row: maximum, and sum of terms 2^lift too large
 * (the terms off the slots, with a teacher's tail). */
struct DistillPart {
  double sum;
  float max;
  float lift;
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
  float *ws_z;                     /* their slots' logits, [rows][slots], or NULL */
  uint64_t rows, ld, gld;
  uint32_t vocab, slots, parts, part_vecs;
  float tau, inv_tau, log2_scale, scale;   /* log2_scale = log2(e) / tau */
  double inv_tau64;
  int vec_store;                   /* gradient rows are aligned as the logits' */
};

/* The shift that makes terms 2^96 larger, where a sum of those off the slots
 * below 2^-40 asks for it; false if it does not or cannot be (beyond 2^24 whole
 * numbers are apart by more). Not for every row: a term near the largest would
 * have an exponent near 96, and six bits less. */
constexpr float kLift = 96.0f, kLittle = 9.09494702e-13f;   /* 2^-40 */

__device__ __forceinline__ bool lift(Shift &s, double sum) {
  const float low = s.whole - kLift;
  if (!(sum < (double)kLittle) || s.whole - low != kLift) return false;
  s.whole = low;
  return true;
}

/* ------------------------------------------------------------------------
 * The slots of one row, by a whole block of NT threads: the teacher's
 * probabilities and what the loss sums over them.
 * ---------------------------------------------------------------------- */
struct SlotLds {           /* as many slots as the call has, to a multiple of four */
  int32_t *id;
  float *w, *z;
};

/* Bytes of LDS for the slots of a row; the launch asks for them. */
__host__ __device__ inline uint32_t slot_bytes(uint32_t slots) { return (slots + 3) / 4 * 4 * 12; }

__device__ __forceinline__ SlotLds slot_lds(uint32_t slots) {
  extern __shared__ __align__(16) char lds[];
  const uint32_t n = (slots + 3) / 4 * 4;
  SlotLds s;
  s.id = reinterpret_cast<int32_t *>(lds);
  s.w = reinterpret_cast<float *>(lds + n * 4);
  s.z = reinterpret_cast<float *>(lds + n * 8);
  return s;
}

/* The slots that round their number up: empty. */
__device__ __forceinline__ void pad_slots(uint32_t slots, const SlotLds &s) {
  const uint32_t k = slots + threadIdx.x;
  if (k < (slots + 3) / 4 * 4) {
    s.id[k] = -1;
    s.w[k] = 0.0f;
  }
}

/* What the reductions over a block pass between its waves. A row's terms are
 * added in fp32 by each thread and joined in binary64. */
template <int NT>
struct ReduceLds {
  float part[5][NT / 64];
  double dpart[4][NT / 64];
};

template <int NT>
__device__ __forceinline__ void put_mass(float v, ReduceLds<NT> &l) {
  reduce_put(v, SumOf{}, l.part[4]);
}
template <int NT>
__device__ __forceinline__ void put_mass(double v, ReduceLds<NT> &l) {
  reduce_put(v, SumOf{}, l.dpart[0]);
}
template <int NT>
__device__ __forceinline__ void get_mass(float &v, const ReduceLds<NT> &l) {
  v = reduce_get<NT>(SumOf{}, l.part[4]);
}
template <int NT>
__device__ __forceinline__ void get_mass(double &v, const ReduceLds<NT> &l) {
  v = reduce_get<NT>(SumOf{}, l.dpart[0]);
}

/* Sum of the weights of token id's slots. */
__device__ __forceinline__ float slot_weight(const SlotLds &s, uint32_t slots, int32_t id) {
  float w = 0.0f;
  for (uint32_t j = 0; j < slots; j += 4) {
    const int4 o = *reinterpret_cast<const int4 *>(s.id + j);
    const float4 v = *reinterpret_cast<const float4 *>(s.w + j);
    w += o.x == id ? v.x : 0.0f;
    w += o.y == id ? v.y : 0.0f;
    w += o.z == id ? v.z : 0.0f;
    w += o.w == id ? v.w : 0.0f;
  }
  return w;
}

/* Whether an earlier slot holds slot k's token. */
__device__ __forceinline__ bool slot_seen(const SlotLds &s, uint32_t k, int32_t id) {
  bool seen = false;
  for (uint32_t j = 0; j < k; j += 4) {
    const int4 o = *reinterpret_cast<const int4 *>(s.id + j);
    seen |= o.x == id || (j + 1 < k && o.y == id) || (j + 2 < k && o.z == id) ||
            (j + 3 < k && o.w == id);
  }
  return seen;
}

/* From slot `first` on: ids and the teacher's logits; returns the logits'
 * maximum over the temperature (+inf for a NaN) and whether a slot is filled. */
struct SlotTop {
  float top, any;
};

template <int DT, int NT>
__device__ __forceinline__ SlotTop slot_ids(const DistillArgs &a, uint64_t row, uint32_t first,
                                            const SlotLds &s) {
  SlotTop r{-INFINITY, 0.0f};
  for (uint32_t k = first + threadIdx.x; k < a.slots; k += NT) {
    const int32_t id = a.ids[row * a.slots + k];
    const bool ok = id >= 0 && (uint32_t)id < a.vocab;
    const float t = ok ? load1<DT>(a.teacher, row * a.slots + k) : -INFINITY;
    s.id[k] = ok ? id : -1;
    s.w[k] = t;
    if (ok) r.any = 1.0f;
    r.top = fmaxf(r.top, t != t ? INFINITY : t * a.inv_tau);
  }
  return r;
}

/* The slots' logits: from `saved` where that is given (the gradient may be
 * written over the logits, and another block may have begun to). */
template <int DT, int NT>
__device__ __forceinline__ void slot_logits(const DistillArgs &a, uint64_t row, const void *z,
                                            const float *saved, uint32_t first, const SlotLds &s) {
  for (uint32_t k = first + threadIdx.x; k < a.slots; k += NT) {
    const int32_t id = s.id[k];
    s.z[k] = id < 0 ? 0.0f : saved ? saved[row * a.slots + k] : load1<DT>(z, id);
  }
}

/* The teacher's mass: binary64 where the rest of 1 counts. */
template <bool TAIL>
struct Exact { typedef float type; };
template <>
struct Exact<true> { typedef double type; };

template <bool TAIL>
struct SlotSums {
  typename Exact<TAIL>::type mass;   /* sum of w */
  float cross;    /* sum of w * ((t - ref) - (u - max u)) */
  double terms;   /* sum of the distinct slots' terms */
};

/* This thread's share; weights w = exp(t / tau - ref) take the logits' place.
 * All ids are in LDS before this. With a tail the exponent is formed in
 * binary64: what it is off by goes into 1 - mass whole. */
template <int DT, bool TAIL, int NT>
__device__ __forceinline__ SlotSums<TAIL> slot_weights(const DistillArgs &a, float ref,
                                                       const Shift &sh, const SlotLds &s) {
  SlotSums<TAIL> r{0, 0.0f, 0.0};
  for (uint32_t k = threadIdx.x; k < a.slots; k += NT) {
    const int32_t id = s.id[k];
    float w = 0.0f;
    if (id >= 0) {
      const float t = s.w[k], zk = s.z[k];
      float u;
      if constexpr (TAIL) {
        const double d = fma((double)t, a.inv_tau64, -(double)ref);
        u = (float)d;
        w = exp2_fast((float)(d * 1.4426950408889634));
      } else {
        u = t * a.inv_tau - ref;
        w = exp2_fast(u * 1.44269504f);
      }
      r.mass += w;
      if (!(w == 0.0f)) r.cross += w * (u - (zk - sh.max) * a.inv_tau);
      if constexpr (TAIL) {
        if (!slot_seen(s, k, id)) r.terms += (double)term<DT>(zk, sh);
      }
    }
    s.w[k] = w;
  }
  return r;
}

/* The teacher's mass off its slots counts as none below 2^-20 or 2^-22 of
 * |lse|, whichever is more: its fp32 logsumexp does not say more, and against
 * a student without such mass the rounding's remainder would make the loss
 * infinite. A logsumexp that is off by half a step, 2^-24 |lse|, changes the
 * mass by as much; one of fp32 logits by three times that; the terms' exp and
 * the rounding of its exponent add 2^-22 at most. */
__device__ __forceinline__ float tail_floor(float lse) {
  return fmaxf(9.53674316e-7f, 2.38418579e-7f * fabsf(lse));
}

/* Loss of a row (without its weight and tau^2), the sum of all terms, and
 * what makes gradients of the terms off the slots: term * up * share * coef. */
struct RowResult {
  float loss, total, up, share;
};

/* sum: of the terms off the slots with TAIL (2^96 too large if `lifted`), of
 * all terms without. */
template <bool TAIL>
__device__ __forceinline__ RowResult row_result(const SlotSums<TAIL> &s, const Shift &sh, float lse,
                                                double sum64, bool lifted) {
  RowResult r;
  const float mass = (float)s.mass, sum = (float)sum64;
  const float down = lifted ? 1.26217745e-29f : 1.0f;   /* 2^-96 */
  r.total = TAIL ? (float)(sum64 * (double)down + s.terms) : sum;
  r.up = 1.0f;
  r.share = 1.0f / r.total;
  const float log_sum = logf(r.total), log_total = log_sum - sh.rest;   /* by the maximum */
  if constexpr (TAIL) {
    r.loss = s.cross + mass * log_total;
    float pr = (float)(1.0 - (double)s.mass);
    pr = pr >= tail_floor(lse) ? pr : 0.0f;   /* NaN mass: the loss is NaN already */
    const float log_rest = logf(sum) - (lifted ? kLift * 0.69314718f : 0.0f);
    if (pr > 0.0f) r.loss += pr * (logf(pr) - (log_rest - log_sum));
    /* nothing off the slots: every such term is 0 whatever its factor */
    if (sum > 0.0f) {
      const uint32_t e = __float_as_uint(sum) >> 23;   /* of 2^(e - 127), at most 2^31 */
      r.up = __uint_as_float((254 - e) << 23);
      r.share = __uint_as_float(e << 23) * down / r.total - pr / (sum * r.up);
    }
  } else {
    r.loss = s.cross / mass - logf(mass) + log_total;
  }
  return r;
}

/* The slots' gradients, after the sweep over the row (and a barrier): this
 * block's share [first, last) of the vocabulary. */
template <int DT, bool TAIL, int NT>
__device__ __forceinline__ void store_slots(const DistillArgs &a, void *g, const SlotLds &s,
                                            const Shift &sh, float total, float mass, float coef,
                                            uint32_t first, uint32_t last) {
  for (uint32_t k = threadIdx.x; k < a.slots; k += NT) {
    const int32_t id = s.id[k];
    if (id < 0 || (uint32_t)id < first || (uint32_t)id >= last) continue;
    const float w = slot_weight(s, a.slots, id);
    const float p = TAIL ? w : w / mass;
    store1<DT>(g, id, (term<DT>(s.z[k], sh) / total - p) * coef);
  }
}

/* What a row's sweep multiplies by. */
struct RowFactors {
  float total, coef, up, factor;
  bool live;
};

/* The gradient of a logit off the slots, from its term. */
template <bool TAIL>
__device__ __forceinline__ float off_slots(float term, const RowFactors &f) {
  return (TAIL ? term * f.up : term) * f.factor;
}

/* From the joined sums: the row's loss (stored by the thread that `says`)
 * and its factors. */
template <bool TAIL>
__device__ __forceinline__ RowFactors finish_row(const DistillArgs &a, uint64_t row, float weight,
                                                 float lse, bool live, const SlotSums<TAIL> &s,
                                                 const Shift &sh, double sum, bool lifted,
                                                 bool says) {
  const RowResult r = row_result<TAIL>(s, sh, lse, sum, lifted);
  RowFactors f;
  f.live = live;
  f.total = r.total;
  f.coef = (a.dev ? a.dev->scale : a.scale) * a.tau * weight;
  f.up = r.up;
  f.factor = TAIL ? f.coef * r.share : f.coef / f.total;
  if (says) a.loss[row] = live ? weight * a.tau * a.tau * r.loss : 0.0f;
  return f;
}

/* The elements of a row that are slots': a bit for each of a vector's, a byte
 * for each vector, and a word for the single elements, by the threads that
 * hold them. */
template <int DT>
__device__ __forceinline__ void mark_slot(uint32_t *bits, uint32_t edges, const RowShape &s,
                                          int32_t id, bool on) {
  constexpr uint32_t ve = kVecElems<DT>;
  const uint32_t at = (uint32_t)id - s.head;   /* wraps for the head's */
  const bool inside = at < s.vecs * ve;
  const uint32_t v = at / ve;
  const uint32_t word = inside ? v / 4 : edges;
  const uint32_t bit = inside                 ? v % 4 * 8 + at % ve
                       : (uint32_t)id < s.head ? (uint32_t)id
                                               : 8 + (at - s.vecs * ve);
  if (on) atomicOr(bits + word, 1u << bit);
  else bits[word] = 0;
}

/* ------------------------------------------------------------------------
 * A row per block, held in registers between its statistics and its
 * gradient: ITEMS 16-byte vectors per thread and, in a few threads, one
 * single element. So each logit is read once: 8192 x 128000 bf16 in 879 us,
 * 4.8 TB/s (read twice, in parts, 1490), with a teacher's tail 970, the loss
 * alone 490; 8192 x 50257 375 us, 16384 x 32000 441 us, 13 x 50257 10 us.
 *
 * Rows of up to 16 vectors a thread leave room for two waves or more of other
 * rows on a SIMD; longer ones, with half of the register file each, have a CU
 * to themselves, and while such a block reduces its maximum and its sum
 * little is under way: that, not the arithmetic (cut to an eighth in a trial:
 * 6 % less), is what it stays below a copy by. Terms by a running maximum as
 * the vectors arrive, twice the threads with half of the vectors, or blocks
 * that start apart in time gained nothing or little.
 * ---------------------------------------------------------------------- */
/* The gradient is stored non-temporally but in one-wave blocks: their short
 * rows have a slot in many of their lines, and a line that has left the L2 by
 * then is read back for it (65536 x 4096: 272 us plain, 326 non-temporal;
 * 16384 x 32000: 469 and 441). */
constexpr int kNonTemporal = 2;

/* What a block knows of a row before it holds it. A row without weight is
 * not read: its buffer is empty. */
struct RowIn {
  const char *z;
  RowShape shape;
  uint32_t edge;
  float weight, lse;
};

template <int DT, bool TAIL>
__device__ __forceinline__ RowIn open_row(const DistillArgs &a, uint32_t row) {
  constexpr uint64_t esz = DT == ZS_FP32 ? 4 : 2;
  RowIn r;
  r.z = static_cast<const char *>(a.z) + (uint64_t)row * a.ld * esz;
  r.shape = row_shape<DT>(r.z, a.vocab);
  r.weight = a.weight ? load_scalar(a.weight, row) : 1.0f;
  r.lse = TAIL ? load_scalar(a.lse, row) : 0.0f;
  r.edge = r.weight != 0.0f ? edge_index<DT>(r.shape, threadIdx.x, true, true, a.vocab) : a.vocab;
  return r;
}

template <int DT>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const RowIn &r) {
  return bounded(r.z + r.shape.head * (DT == ZS_FP32 ? 4 : 2),
                 r.weight != 0.0f ? r.shape.vecs * 16 : 0);
}

/* The vector at byte `at`, or the row's last for a thread past it: one that
 * the maximum may count twice and the sum leaves out. */
template <int DT>
__device__ __forceinline__ u32x4 fetch_vec(__amdgpu_buffer_rsrc_t row, const RowIn &r, uint32_t at) {
  const uint32_t last = (r.shape.vecs - 1) * 16, mine = at + threadIdx.x * 16;
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                       row, (int)(mine < last ? mine : last), 0, 0));
}

template <int DT>
__device__ __forceinline__ uint32_t fetch_edge(const DistillArgs &a, const RowIn &r) {
  uint32_t w = empty_vec<DT>()[0];
  if (r.edge < a.vocab) w = load_raw<DT>(r.z, r.edge);
  return w;
}

/* Holds the first NT slots of a row in a register each, fetched ahead, as
 * they lie in memory. */
struct SlotAhead {
  int32_t id;
  uint32_t t, z;
};

/* A block walks rows blockIdx, + gridDim, ... While it writes a row's
 * gradient it fetches the next row into the registers that fall free. Loads
 * return in order, so what is wanted early is asked for early: the next row's
 * slots before its vectors, their logits after. */
template <int DT, bool TAIL, int NT, int ITEMS>
__global__ __launch_bounds__(NT, ITEMS <= 16 ? 4 : 2) void distill_row_kernel(DistillArgs a) {
  constexpr uint32_t ve = kVecElems<DT>, esz = DT == ZS_FP32 ? 4 : 2;
  __shared__ ReduceLds<NT> red;
  constexpr uint32_t kMarks = NT * ITEMS / 4;   /* words; one more for the edges */
  __shared__ uint32_t marks[TAIL ? kMarks + 1 : 1];
  const SlotLds lds = slot_lds(a.slots);
  pad_slots(a.slots, lds);
  const uint32_t t = threadIdx.x;
  if constexpr (TAIL) {   /* a row clears its own marks afterwards */
    for (uint32_t i = t; i <= kMarks; i += NT) marks[i] = 0;
    __syncthreads();
  }
  uint32_t row = blockIdx.x;
  RowIn in = open_row<DT, TAIL>(a, row);
  auto slots_ahead = [&](uint32_t r, const RowIn &q, SlotAhead &s) {
    s.id = -1;
    s.t = 0;
    if (t < a.slots && q.weight != 0.0f) {
      s.id = a.ids[(uint64_t)r * a.slots + t];
      s.t = load_raw<DT>(a.teacher, (uint64_t)r * a.slots + t);
    }
  };
  auto logits_ahead = [&](const RowIn &q, SlotAhead &s) {
    s.z = 0;
    if ((uint32_t)s.id < a.vocab) s.z = load_raw<DT>(q.z, s.id);
  };
  SlotAhead slot;
  slots_ahead(row, in, slot);
  u32x4 x[ITEMS];
  {
    const __amdgpu_buffer_rsrc_t buf = row_buffer<DT>(in);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) x[i] = fetch_vec<DT>(buf, in, i * (NT * 16));
  }
  uint32_t raw_single = fetch_edge<DT>(a, in);
  logits_ahead(in, slot);
  for (;;) {
    /* rows are told apart by a scalar that the compiler cannot follow: it would
     * keep a pointer of its own in vector registers for every use */
    asm volatile("" : "+s"(row));
    const uint32_t next = row + gridDim.x;
    const RowIn after = open_row<DT, TAIL>(a, next < a.rows ? next : row);
    RowFactors f{1.0f, 0.0f, 1.0f, 0.0f, false};
    SlotSums<TAIL> sums{};
    Shift shift{}, off{};   /* off: of the terms off the slots */
    float single = -INFINITY;
    if (in.weight != 0.0f) {   /* uniform over the block */
      VecMax<DT> max;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) max.add(x[i]);
      single = raw_value<DT>(raw_single);
      SlotTop top{-INFINITY, 0.0f};
      if (t < a.slots) {
        const bool ok = (uint32_t)slot.id < a.vocab;
        const float v = ok ? raw_value<DT>(slot.t) : -INFINITY;
        lds.id[t] = ok ? slot.id : -1;
        lds.w[t] = v;
        lds.z[t] = raw_value<DT>(slot.z);
        if (ok) top = {v != v ? INFINITY : v * a.inv_tau, 1.0f};
      }
      if (a.slots > NT) {   /* the others */
        const SlotTop more = slot_ids<DT, NT>(a, row, NT, lds);
        slot_logits<DT, NT>(a, row, in.z, nullptr, NT, lds);
        top = {fmaxf(top.top, more.top), fmaxf(top.any, more.any)};
      }
      if constexpr (TAIL) {
        for (uint32_t k = t; k < a.slots; k += NT)
          if (lds.id[k] >= 0) mark_slot<DT>(marks, kMarks, in.shape, lds.id[k], true);
      }
      reduce_put(fmaxf(max.get(), single), MaxOf{}, red.part[0]);
      reduce_put(top.top, MaxOf{}, red.part[1]);
      reduce_put(top.any, MaxOf{}, red.part[2]);
      __syncthreads();
      shift = shift_of<DT>(reduce_get<NT>(MaxOf{}, red.part[0]), a.log2_scale);
      const float highest = reduce_get<NT>(MaxOf{}, red.part[1]);
      const float ref = TAIL ? in.lse : highest;
      const bool live = TAIL ? reduce_get<NT>(MaxOf{}, red.part[2]) > 0.0f : highest > -INFINITY;
      off = shift;
      auto sum_terms = [&] {
        float sum = in.edge < a.vocab ? term<DT>(single, off) : 0.0f;
        if constexpr (TAIL) {
          if (in.edge < a.vocab && marks[kMarks] >> t & 1) sum = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          float e[ve];
          if constexpr (TAIL) asm volatile("" : "+v"(x[i]));   /* unpacked anew each time */
          unpack_vec<DT>(x[i], e);
          float some = 0.0f;
          if constexpr (TAIL) {
            const uint32_t m = reinterpret_cast<const uint8_t *>(marks)[i * NT + t];
            if (m) {
#pragma unroll
              for (uint32_t j = 0; j < ve; ++j) e[j] = m >> j & 1 ? -INFINITY : e[j];
            }
          }
#pragma unroll
          for (uint32_t j = 0; j < ve; ++j) some += term<DT>(e[j], off);
          sum += (int)t < (int)in.shape.vecs - i * NT ? some : 0;
          if constexpr (TAIL) asm volatile("" : "+v"(sum));   /* now, not behind the next branch */
          __builtin_amdgcn_sched_barrier(0);
        }
        return sum;
      };
      reduce_put((double)sum_terms(), SumOf{}, red.dpart[1]);
      sums = slot_weights<DT, TAIL, NT>(a, ref, shift, lds);
      put_mass<NT>(sums.mass, red);
      reduce_put(sums.cross, SumOf{}, red.part[3]);
      if constexpr (TAIL) reduce_put(sums.terms, SumOf{}, red.dpart[2]);
      __syncthreads();
      double sum = reduce_get<NT>(SumOf{}, red.dpart[1]);
      bool lifted = false;
      if constexpr (TAIL) {
        lifted = lift(off, sum);   /* uniform over the block */
        if (lifted) {
          reduce_put((double)sum_terms(), SumOf{}, red.dpart[3]);
          __syncthreads();
          sum = reduce_get<NT>(SumOf{}, red.dpart[3]);
        }
      }
      get_mass<NT>(sums.mass, red);
      sums.cross = reduce_get<NT>(SumOf{}, red.part[3]);
      if constexpr (TAIL) {
        sums.terms = reduce_get<NT>(SumOf{}, red.dpart[2]);
        for (uint32_t k = t; k < a.slots; k += NT)
          if (lds.id[k] >= 0) mark_slot<DT>(marks, kMarks, in.shape, lds.id[k], false);
      }
      f = finish_row<TAIL>(a, row, in.weight, in.lse, live, sums, shift, sum, lifted, t == 0);
    } else if (t == 0) {
      a.loss[row] = 0.0f;
    }
    if (!f.live) {   /* zeros: terms of -inf */
      off.c = 1.0f;
      off.whole = off.frac = f.factor = 0.0f;
      f.up = 1.0f;
      single = -INFINITY;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) x[i] = empty_vec<DT>();
    }
    char *g = static_cast<char *>(a.grad) + (uint64_t)row * a.gld * esz;
    const bool more = next < a.rows;
    const __amdgpu_buffer_rsrc_t to = bounded(g + in.shape.head * esz, in.shape.vecs * 16);
    const __amdgpu_buffer_rsrc_t from = row_buffer<DT>(after);
    if (more) slots_ahead(next, after, slot);
    const uint32_t edge = edge_index<DT>(in.shape, t, true, true, a.vocab);
    if (a.grad && edge < a.vocab) store1<DT>(g, edge, off_slots<TAIL>(term<DT>(single, off), f));
    if (more) raw_single = fetch_edge<DT>(a, after);
    if (!a.grad) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) x[i] = fetch_vec<DT>(from, after, i * (NT * 16));
    } else {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        float e[ve];
        asm volatile("" : "+v"(x[i]));   /* unpacked anew, not kept since the sum */
        unpack_vec<DT>(x[i], e);
#pragma unroll
        for (uint32_t j = 0; j < ve; ++j) e[j] = off_slots<TAIL>(term<DT>(e[j], off), f);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, pack_vec<DT>(e)), to,
                                               (int)(t * 16 + i * (NT * 16)), 0,
                                               NT > 64 ? kNonTemporal : 0);
        x[i] = fetch_vec<DT>(from, after, i * (NT * 16));   /* past the last row: not used */
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (more) logits_ahead(after, slot);
    __syncthreads();
    if (a.grad && f.live)
      store_slots<DT, TAIL, NT>(a, g, lds, shift, f.total, (float)sums.mass, f.coef, 0, a.vocab);
    if (!more) return;
    __syncthreads();   /* the slots in LDS are done with */
    row = next;
    in = after;
  }
}

/* ------------------------------------------------------------------------
 * Rows in parts, where a row is longer than a block's registers (or its
 * gradient is aligned another way): a block per part forms its statistics,
 * then a block per part joins all of its row's and writes its share of the
 * gradient. Two launches and no wait between blocks; a part, read up to three
 * times, is short enough for the caches where few rows make many parts.
 *
 * A part's sum leaves the slots out with TAIL: a bit of LDS for every vector,
 * its number counted modulo the bits there are, says which to look at closely.
 * ---------------------------------------------------------------------- */
constexpr uint32_t kFilterWords = 1024;

/* -inf in the place of the slots' among N elements from token `first` on. */
template <uint32_t N>
__device__ __forceinline__ void leave_slots_out(const SlotLds &s, uint32_t slots, uint32_t first,
                                                float (&x)[N]) {
  for (uint32_t k = 0; k < slots; k += 4) {
    const int4 o = *reinterpret_cast<const int4 *>(s.id + k);
    const uint32_t at[4] = {(uint32_t)o.x - first, (uint32_t)o.y - first, (uint32_t)o.z - first,
                            (uint32_t)o.w - first};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (at[i] >= N) continue;
#pragma unroll
      for (uint32_t j = 0; j < N; ++j) x[j] = at[i] == j ? -INFINITY : x[j];
    }
  }
}

template <int DT, bool TAIL, int NT>
__global__ __launch_bounds__(NT) void distill_stats_kernel(DistillArgs a) {
  constexpr uint32_t ve = kVecElems<DT>;
  __shared__ float fpart[NT / 64];
  __shared__ double dpart[2][NT / 64];
  __shared__ uint32_t filter[TAIL ? kFilterWords : 1];
  const SlotLds lds = slot_lds(a.slots);   /* ids, with TAIL */
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
  if constexpr (TAIL) {
    pad_slots(a.slots, lds);
    for (uint32_t i = threadIdx.x; i < kFilterWords; i += NT) filter[i] = 0;
    __syncthreads();
    for (uint32_t k = threadIdx.x; k < a.slots; k += NT) {
      const int32_t id = a.ids[row * a.slots + k];
      lds.id[k] = id;
      const uint32_t v = ((uint32_t)id - sh.head) / ve;   /* ids elsewhere only set a bit more */
      atomicOr(filter + v / 32 % kFilterWords, 1u << v % 32);
    }
  }
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
  float single[1] = {edge < a.vocab ? load1<DT>(z, edge) : -INFINITY};
  if constexpr (TAIL) {
    if (edge < a.vocab) leave_slots_out(lds, a.slots, edge, single);
  }
  Shift off = shift_of<DT>(max, a.log2_scale);
  double sum;
  bool lifted = false;
  for (;;) {
    sum = edge < a.vocab ? (double)term<DT>(single[0], off) : 0.0;
    for (uint32_t v = v0 + threadIdx.x; v < v1; v += NT) {
      float x[ve];
      unpack_vec<DT>(zv[v], x);
      if constexpr (TAIL) {
        if (filter[v / 32 % kFilterWords] >> v % 32 & 1)
          leave_slots_out(lds, a.slots, sh.head + v * ve, x);
      }
#pragma unroll
      for (uint32_t j = 0; j < ve; ++j) sum += (double)term<DT>(x[j], off);
    }
    reduce_put(sum, SumOf{}, dpart[lifted]);
    __syncthreads();
    sum = reduce_get<NT>(SumOf{}, dpart[lifted]);
    if (!TAIL || lifted) break;
    lifted = lift(off, sum);   /* uniform over the block */
    if (!lifted) break;
  }
  if (threadIdx.x == 0) a.ws[blockIdx.x] = {sum, max, lifted ? kLift : 0.0f};
  if (part != 0 || !a.ws_z) return;
  for (uint32_t k = threadIdx.x; k < a.slots; k += NT) {
    const int32_t id = a.ids[row * a.slots + k];
    if (id >= 0 && (uint32_t)id < a.vocab) a.ws_z[row * a.slots + k] = load1<DT>(z, id);
  }
}

/* What turns a part's terms into the row's. A part of nothing but -inf has the
 * sum 0, one with a NaN or +inf off the slots a NaN. */
template <int DT>
__device__ __forceinline__ double part_factor(const DistillPart &w, const Shift &row, float c) {
  return w.max == -INFINITY ? 0.0 : shift_factor<DT>(shift_of<DT>(w.max, c), row, w.lift);
}

template <int DT, bool TAIL, int NT>
__global__ __launch_bounds__(NT) void distill_grad_kernel(DistillArgs a, uint32_t blocks) {
  constexpr uint32_t ve = kVecElems<DT>;
  __shared__ ReduceLds<NT> red;
  const SlotLds lds = slot_lds(a.slots);
  pad_slots(a.slots, lds);
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
  RowFactors f{1.0f, 0.0f, 1.0f, 0.0f, false};
  Shift shift{}, off{};
  SlotSums<TAIL> sums{};
  if (weight != 0.0f) {
    const DistillPart *w = a.ws + row * a.parts;
    float max = -INFINITY;
    for (uint32_t i = 0; i < a.parts; ++i) max = fmaxf(max, w[i].max);
    shift = shift_of<DT>(max, a.log2_scale);
    double sum = 0.0;
    for (uint32_t i = 0; i < a.parts; ++i)
      sum += w[i].sum * part_factor<DT>(w[i], shift, a.log2_scale);
    off = shift;
    bool lifted = false;
    if constexpr (TAIL) {
      lifted = lift(off, sum);
      if (lifted) sum *= 7.9228162514264338e28;   /* 2^96 */
    }
    const SlotTop top = slot_ids<DT, NT>(a, row, 0, lds);
    slot_logits<DT, NT>(a, row, z, a.ws_z, 0, lds);
    reduce_put(top.top, MaxOf{}, red.part[1]);
    reduce_put(top.any, MaxOf{}, red.part[2]);
    __syncthreads();
    const float highest = reduce_get<NT>(MaxOf{}, red.part[1]);
    const float ref = TAIL ? a.lse[row] : highest;
    const bool live = TAIL ? reduce_get<NT>(MaxOf{}, red.part[2]) > 0.0f : highest > -INFINITY;
    sums = slot_weights<DT, TAIL, NT>(a, ref, shift, lds);
    put_mass<NT>(sums.mass, red);
    reduce_put(sums.cross, SumOf{}, red.part[3]);
    if constexpr (TAIL) reduce_put(sums.terms, SumOf{}, red.dpart[2]);
    __syncthreads();
    get_mass<NT>(sums.mass, red);
    sums.cross = reduce_get<NT>(SumOf{}, red.part[3]);
    if constexpr (TAIL) sums.terms = reduce_get<NT>(SumOf{}, red.dpart[2]);
    f = finish_row<TAIL>(a, row, weight, ref, live, sums, shift, sum, lifted,
                         first && threadIdx.x == 0);
  } else if (first && threadIdx.x == 0) {
    a.loss[row] = 0.0f;
  }
  if (!g) return;
  const u32x4 *zv = reinterpret_cast<const u32x4 *>(z + sh.head * esz);
  if (edge < a.vocab)
    store1<DT>(g, edge, f.live ? off_slots<TAIL>(term<DT>(load1<DT>(z, edge), off), f) : 0.0f);
  for (uint32_t v = v0 + threadIdx.x; v < v1; v += NT) {
    float x[ve];
    if (f.live) {
      unpack_vec<DT>(zv[v], x);
#pragma unroll
      for (uint32_t j = 0; j < ve; ++j) x[j] = off_slots<TAIL>(term<DT>(x[j], off), f);
    } else {
#pragma unroll
      for (uint32_t j = 0; j < ve; ++j) x[j] = 0.0f;
    }
    if (a.vec_store) {
      *reinterpret_cast<u32x4 *>(g + sh.head * esz + v * 16ull) = pack_vec<DT>(x);
    } else {
#pragma unroll
      for (uint32_t j = 0; j < ve; ++j) store1<DT>(g, sh.head + (uint64_t)v * ve + j, x[j]);
    }
  }
  __syncthreads();
  if (f.live)
    store_slots<DT, TAIL, NT>(a, g, lds, shift, f.total, (float)sums.mass, f.coef,
                              first ? 0 : sh.head + v0 * ve,
                              last ? a.vocab : sh.head + v1 * ve);
}

}  // namespace zs
#endif  // ZS_DISTILL_KERNELS_H
