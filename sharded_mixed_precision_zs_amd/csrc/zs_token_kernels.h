/*
 * zs_token_kernels.h -- log-probabilities of given tokens, the clipped policy
 * loss and the loss of paired sequences, and the logits' gradient of both
 * (gfx950).
 *
 * With u = z / tau, q = softmax(u), a row's token a and g the loss's slope in
 * log q[a], the gradient is g / tau (1[j = a] - q[j]) whatever the loss: one
 * factor for all terms of the softmax, and one element of its own. That one,
 * 1 - q[a], is the sum of the other terms, which leaves a's out as it comes:
 * where a student is sure of its token, taking q[a] from 1 would leave
 * rounding; log q[a] is then log1p of the same ratio.
 *
 * Terms are 2^(z c - I), c = log2(e) / tau and I the whole number next to the
 * token's own z c: no pass over the row has to find its maximum first, and a
 * term is added as its logit arrives. Where that lets the sum leave 2^60 (a
 * token that has less than e^-41 of the mass), or where the token's logit is
 * -inf and no place to count from, it is formed again by the row's maximum; so
 * a part that is counted from -inf holds nothing but -inf. The rounding of an
 * exponent is relative to its size, which is that of the log-probability.
 *
 * Bound by HBM: the policy loss reads a row once, into a block's registers,
 * the preference loss twice, for a row's gradient needs its whole pair.
 */
#ifndef ZS_TOKEN_KERNELS_H
#define ZS_TOKEN_KERNELS_H

#include "zs_logits.h"

namespace zs {

/* Statistics of one part of a row: the sum of its terms but the token's, and
 * the logit that their shift is from. */
struct TokenPart {
  double rest;
  float from, pad;
};

/* What a row's gradient is made of: term * factor, and `own` for token id. */
struct TokenPlan {
  float from, factor, own;
  int32_t id;      /* kNoToken: zeros, and the logits are not read; kOutside: not written */
};
constexpr int32_t kNoToken = -1, kOutside = -2;

struct TokenArgs {
  const void *z;
  const int32_t *ids;
  const float *weight;             /* per row, optional */
  const zs_device_scaler *dev;     /* optional: its scale in place of `scale` */
  /* policy */
  const float *advantage, *old_logp, *ref_logp;   /* the last two optional */
  float *logp, *loss;              /* per row; loss per pair with starts */
  float clip_low, clip_high, kl_weight;
  /* pairs */
  const int32_t *starts;           /* [2 * pairs + 1], or NULL */
  const float *ref_seq, *pair_weight;   /* optional */
  float *seq_logp;                 /* optional */
  float beta, smoothing;
  uint32_t pairs;
  int kind, mean, clear;           /* clear: zeros in gradient rows outside all sequences */

  void *grad;                      /* optional */
  TokenPart *ws;                   /* [rows][parts] */
  TokenPlan *plan;                 /* [rows]; of pairs first with the total and the rest
                                    * for `factor` and `own` */
  double *lp;                      /* [rows]: log-probabilities, of pairs */
  float *own;                      /* [rows]: the tokens' logits, of rows in parts */
  uint64_t ld, gld;
  uint32_t rows, vocab, parts, part_vecs;
  uint32_t row0, blocks;           /* gradient: a launch's first row, blocks of a row */
  float log2_scale, inv_tau, scale;   /* log2_scale = log2(e) / tau */
};

__device__ __forceinline__ int32_t load_scalar(const int32_t *p, uint32_t i) {
  return __float_as_int(load_scalar(reinterpret_cast<const float *>(p), i));
}

/* Rows of the sequences, first and one past the last. */
struct TokenSpan {
  uint32_t first, last;
};

__device__ __forceinline__ uint32_t row_of(int32_t start, uint32_t rows) {
  return start < 0 ? 0u : (uint32_t)start < rows ? (uint32_t)start : rows;
}

__device__ __forceinline__ TokenSpan token_span(const TokenArgs &a) {
  if (!a.starts) return {0, a.rows};
  return {row_of(load_scalar(a.starts, 0), a.rows),
          row_of(load_scalar(a.starts, 2 * a.pairs), a.rows)};
}

__device__ __forceinline__ bool token_live(const TokenArgs &a, uint32_t row, int32_t id) {
  return (uint32_t)id < a.vocab && (!a.weight || a.weight[row] != 0.0f);
}

/* ------------------------------------------------------------------------
 * A row's token: its share of the softmax and its log-probability. `rest` and
 * `own` are the sums of the other terms and its own.
 * ---------------------------------------------------------------------- */
struct TokenMass {
  double rest, total, logp;
};

constexpr float kTokenTop = 1.15292150e18f;   /* 2^60 */

/* Whether z's exponent does not give its log-probability: where the shift's
 * logit lies beyond the exponents' range, so that terms have another c than the
 * row's, or z itself does, so that its product could overflow. */
__device__ __forceinline__ bool token_far(float z, const Shift &s, float c) {
  return s.c != c || !(fabsf(z * c) < kTokenTop);
}

/* Then its distance from that logit does, whose term is 1, or as near to it as
 * a distance of 2^60 tells. */
__device__ __forceinline__ double far_log(float z, const Shift &s, float c) {
  return ((double)z - (double)s.max) * ((double)c * 0.69314718055994531);
}

template <int DT>
__device__ __forceinline__ TokenMass token_mass(double rest, float z, const Shift &s, float c) {
  TokenMass m;
  const double own = (double)term<DT>(z, s);
  m.rest = rest;
  m.total = rest + own;
  if (rest <= own && own > 0.0)
    m.logp = -log1p(rest / own);
  else   /* NaN: comes here */
    m.logp = (token_far(z, s, c)
                  ? far_log(z, s, c)
                  : (fma((double)z, (double)s.c, -(double)s.whole) - (double)s.frac) *
                        0.69314718055994531) -
             log(m.total);
  return m;
}

/* The same in fp32, where a row's logits hold the registers: the logarithm is
 * off by half a unit in its last place, as the result's own rounding is. */
struct TokenMass32 {
  float rest, total, logp;
};

template <int DT>
__device__ __forceinline__ TokenMass32 token_mass32(double rest, float z, const Shift &s,
                                                    float c) {
  TokenMass32 m;
  const float own = term<DT>(z, s);
  m.rest = (float)rest;
  m.total = (float)(rest + (double)own);
  if (m.rest <= own && own > 0.0f)
    m.logp = -log1pf(m.rest / own);
  else   /* NaN: comes here */
    m.logp = (token_far(z, s, c) ? (float)far_log(z, s, c)
                                 : (fmaf(z, s.c, -s.whole) - s.frac) * 0.69314718f) -
             logf(m.total);
  return m;
}

/* exp(d) - 1 - d, by its series near 0, where the difference would leave
 * rounding; and its slope exp(d) - 1, from the series too there, but not
 * elsewhere: of a d far below 0 the sum with d would leave nothing of the 1. */
struct ExpRest {
  float rest, slope;
};

__device__ __forceinline__ ExpRest exp_rest(float d) {
  if (!(fabsf(d) < 1.0f)) {
    const float e = expf(d) - 1.0f;
    return {d == INFINITY ? d : e - d, e};   /* not the difference of two infinities */
  }
  float s = 1.0f + d * (1.0f / 12.0f);
#pragma unroll
  for (int k = 11; k > 2; --k) s = fmaf(d * (1.0f / (float)k), s, 1.0f);
  const float rest = 0.5f * d * d * s;
  return {rest, d + rest};
}

struct Slope {
  float loss, slope;   /* slope: of the loss in the log-probability */
};

/* What a row's policy loss takes in, loaded ahead of its use. */
struct PolicyIn {
  float advantage, old_logp, ref_logp, weight;
};

__device__ __forceinline__ PolicyIn policy_in(const TokenArgs &a, uint32_t row) {
  PolicyIn p;
  p.advantage = load_scalar(a.advantage, row);
  p.old_logp = a.old_logp ? load_scalar(a.old_logp, row) : 0.0f;
  p.ref_logp = a.ref_logp ? load_scalar(a.ref_logp, row) : 0.0f;
  p.weight = a.weight ? load_scalar(a.weight, row) : 1.0f;
  return p;
}

template <class T>
__device__ __forceinline__ Slope policy_slope(const TokenArgs &a, const PolicyIn &in, T logp) {
  const float adv = in.advantage;
  const float r = a.old_logp ? expf((float)(logp - (T)in.old_logp)) : 1.0f;
  const float low = 1.0f - a.clip_low, high = 1.0f + a.clip_high;
  /* without an advantage r is clipped too: it may lie beyond fp32, times 0 */
  const bool above = adv >= 0.0f && r > high, below = adv < 0.0f && r < low;
  Slope s;
  s.loss = -(above ? high : below ? low : r) * adv;
  s.slope = above || below ? 0.0f : -r * adv;
  if (a.ref_logp) {
    const ExpRest k = exp_rest((float)((T)in.ref_logp - logp));
    s.loss = fmaf(a.kl_weight, k.rest, s.loss);
    s.slope = fmaf(-a.kl_weight, k.slope, s.slope);
  }
  s.loss *= in.weight;
  s.slope *= in.weight;
  return s;
}

/* Loss scale over the temperature. */
__device__ __forceinline__ float grad_scale(const TokenArgs &a) {
  return (a.dev ? load_scalar(&a.dev->scale, 0) : a.scale) * a.inv_tau;
}

/* A row's plan from its sums and the slope times loss scale and 1 / tau. */
__device__ __forceinline__ TokenPlan make_plan(double rest, double total, float from, float slope,
                                               int32_t id) {
  TokenPlan p;
  p.from = from;
  p.factor = (float)(-(double)slope / total);
  p.own = (float)((double)slope * (rest / total));
  p.id = slope == 0.0f ? kNoToken : id;
  return p;
}

/* ------------------------------------------------------------------------
 * Statistics: a block per part of a row, U vectors of a thread under way at a
 * time. A thread's sums of U vectors are fp32, what they are added to
 * binary64. 8192 x 128000 bf16 306 us, 6.9 TB/s; rows of 1000 are held up by
 * their one thread's binary64 logarithm (65536 of them 46 us, 2.8 TB/s).
 * ---------------------------------------------------------------------- */
template <int DT>
__device__ __forceinline__ void leave_out(const RowShape &s, int32_t id, uint32_t v,
                                          float (&e)[kVecElems<DT>]) {
  constexpr uint32_t ve = kVecElems<DT>;
  const uint32_t at = (uint32_t)id - s.head - v * ve;   /* wraps for what is before */
  if (at >= ve) return;
#pragma unroll
  for (uint32_t j = 0; j < ve; ++j) e[j] = at == j ? -INFINITY : e[j];
}

/* The row's results, where one thread knows all of it: log-probability,
 * policy loss and plan, as far as they are asked for. */
template <int DT>
__device__ __forceinline__ void finish_token(const TokenArgs &a, uint32_t row, double rest,
                                             float from, float z, int32_t id) {
  const TokenMass m = token_mass<DT>(rest, z, shift_of<DT>(from, a.log2_scale), a.log2_scale);
  if (a.logp) a.logp[row] = (float)m.logp;
  if (a.starts) {
    a.lp[row] = m.logp;
    a.plan[row] = {from, (float)m.total, (float)m.rest, id};   /* until its pair gives a slope */
    return;
  }
  if (!a.loss) return;
  const Slope s = policy_slope(a, policy_in(a, row), m.logp);
  a.loss[row] = s.loss;
  if (a.grad) a.plan[row] = make_plan(m.rest, m.total, from, s.slope * grad_scale(a), id);
}

/* A row without a token, or without weight. */
__device__ __forceinline__ void dead_token(const TokenArgs &a, uint32_t row) {
  if (a.logp) a.logp[row] = 0.0f;
  if (a.loss && !a.starts) a.loss[row] = 0.0f;
  if (a.plan) a.plan[row] = {0.0f, 0.0f, 0.0f, kNoToken};
}

template <int DT, int NT>
__global__ __launch_bounds__(NT) void token_stats_kernel(TokenArgs a) {
  constexpr uint32_t ve = kVecElems<DT>, esz = DT == ZS_FP32 ? 4 : 2;
  constexpr int U = 4;
  __shared__ float fpart[NT / 64];
  __shared__ double dpart[2][NT / 64];
  const uint32_t row = blockIdx.x / a.parts, part = blockIdx.x % a.parts, t = threadIdx.x;
  const TokenSpan span = token_span(a);
  if (row < span.first || row >= span.last) {
    if (part == 0 && t == 0) a.plan[row] = {0.0f, 0.0f, 0.0f, a.clear ? kNoToken : kOutside};
    return;
  }
  const int32_t id = load_scalar(a.ids, row);
  if (!token_live(a, row, id)) {
    if (part == 0 && t == 0) dead_token(a, row);
    return;
  }
  const char *z = static_cast<const char *>(a.z) + (uint64_t)row * a.ld * esz;
  const RowShape sh = row_shape<DT>(z, a.vocab);
  const u32x4 *zv = reinterpret_cast<const u32x4 *>(z + sh.head * esz);
  const uint32_t v0 = part * a.part_vecs;
  const uint32_t v1 = v0 + a.part_vecs < sh.vecs ? v0 + a.part_vecs : sh.vecs;
  const uint32_t edge = edge_index<DT>(sh, t, part == 0, part == a.parts - 1, a.vocab);
  const float own = load1<DT>(z, id);
  const float single = edge < a.vocab && edge != (uint32_t)id ? load1<DT>(z, edge) : -INFINITY;
  float from = own;
  double sum;
  for (bool again = false;; again = true) {
    const Shift shift = shift_of<DT>(from, a.log2_scale);
    sum = (double)term<DT>(single, shift);
    for (uint32_t v = v0 + t; v < v1; v += U * NT) {
      u32x4 x[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        x[i] = v + i * NT < v1 ? __builtin_nontemporal_load(zv + v + i * NT) : empty_vec<DT>();
      float some = 0.0f;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float e[ve];
        unpack_vec<DT>(x[i], e);
        leave_out<DT>(sh, id, v + i * NT, e);
#pragma unroll
        for (uint32_t j = 0; j < ve; ++j) some += term<DT>(e[j], shift);
      }
      sum += (double)some;
    }
    reduce_put(sum, SumOf{}, dpart[again]);
    __syncthreads();
    sum = reduce_get<NT>(SumOf{}, dpart[again]);
    /* the same for the whole block */
    if (again || (sum < (double)kTokenTop && own != -INFINITY)) break;
    float max = single;
    for (uint32_t v = v0 + t; v < v1; v += NT) {
      float e[ve];
      unpack_vec<DT>(zv[v], e);
#pragma unroll
      for (uint32_t j = 0; j < ve; ++j) max = fmaxf(max, e[j]);
    }
    reduce_put(max, MaxOf{}, fpart);
    __syncthreads();
    from = reduce_get<NT>(MaxOf{}, fpart);
  }
  if (t != 0) return;
  if (a.parts == 1) {
    finish_token<DT>(a, row, sum, from, own, id);
  } else {
    a.ws[(uint64_t)row * a.parts + part] = {sum, from, 0.0f};
    if (part == 0) a.own[row] = own;
  }
}

/* All of a row's parts, 64 at most, by a wave: in order of a fixed tree, by the
 * largest of the logits that their shifts are from. */
constexpr uint32_t kMaxParts = 64;

template <int DT>
__device__ __forceinline__ TokenPart join_parts(const TokenArgs &a, uint32_t row) {
  const uint32_t lane = threadIdx.x & 63;
  TokenPart p{0.0, -INFINITY, 0.0f};
  if (lane < a.parts) p = a.ws[(uint64_t)row * a.parts + lane];
  const float from = wave_reduce(p.from, MaxOf{}, 64);
  /* a part from -inf has nothing else */
  const double f = p.from == -INFINITY
                       ? 0.0
                       : shift_factor<DT>(shift_of<DT>(p.from, a.log2_scale),
                                          shift_of<DT>(from, a.log2_scale), 0.0f);
  return {wave_reduce(p.rest * f, SumOf{}, 64), from, 0.0f};
}

/* ------------------------------------------------------------------------
 * Pairs: a block per pair sums its sequences' log-probabilities, in binary64
 * and in a fixed order, forms the loss and gives every row its plan. Latency: 4
 * us for 131 rows of two pairs, 8 for 16384 of 16.
 * ---------------------------------------------------------------------- */
constexpr int kPairThreads = 1024;

struct PairSlope {
  double loss, slope;   /* slope: of the loss in the difference of log ratios */
};

__device__ __forceinline__ PairSlope pair_slope(const TokenArgs &a, double delta) {
  const double beta = a.beta, m = beta * delta;
  if (a.kind == ZS_PREFERENCE_SIGMOID) {
    const double eps = a.smoothing, small = log1p(exp(-fabs(m)));
    const double up = m > 0.0 ? m : 0.0, down = m > 0.0 ? 0.0 : -m;   /* NaN: small is one */
    /* a term of weight 0 is none, also of an infinite difference */
    const double yes = eps < 1.0 ? (1.0 - eps) * (small + down) : 0.0;
    const double no = eps > 0.0 ? eps * (small + up) : 0.0;
    return {yes + no, beta * (eps / (1.0 + exp(-m)) - (1.0 - eps) / (1.0 + exp(m)))};
  }
  if (a.kind == ZS_PREFERENCE_HINGE) {
    const double l = 1.0 - m;
    return {l <= 0.0 ? 0.0 : l, l <= 0.0 ? 0.0 : l > 0.0 ? -beta : l};
  }
  const double d = delta - 0.5 / beta;
  return {d * d, 2.0 * d};
}

__global__ __launch_bounds__(kPairThreads) void token_pair_kernel(TokenArgs a) {
  constexpr int NT = kPairThreads;
  __shared__ double part[4][NT / 64];
  const uint32_t pair = blockIdx.x;
  double sum[2] = {0.0, 0.0}, count[2] = {0.0, 0.0};
  TokenSpan seq[2];
#pragma unroll
  for (int k = 0; k < 2; ++k)
    seq[k] = {row_of(load_scalar(a.starts, 2 * pair + k), a.rows),
              row_of(load_scalar(a.starts, 2 * pair + k + 1), a.rows)};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    for (uint64_t row = (uint64_t)seq[k].first + threadIdx.x; row < seq[k].last; row += NT) {
      const int32_t id = a.ids[row];
      const double lp = a.lp[row];   /* not written where there is no token */
      if (!token_live(a, row, id)) continue;
      sum[k] += lp;
      count[k] += 1.0;
    }
    reduce_put(sum[k], SumOf{}, part[2 * k]);
    reduce_put(count[k], SumOf{}, part[2 * k + 1]);
  }
  __syncthreads();
  double each[2], ratio[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    sum[k] = reduce_get<NT>(SumOf{}, part[2 * k]);
    count[k] = reduce_get<NT>(SumOf{}, part[2 * k + 1]);
    each[k] = a.mean && count[k] > 0.0 ? 1.0 / count[k] : 1.0;
    sum[k] *= each[k];
    ratio[k] = sum[k] - (a.ref_seq ? (double)a.ref_seq[2 * pair + k] : 0.0);
  }
  const double weight = a.pair_weight ? (double)a.pair_weight[pair] : 1.0;
  PairSlope s = pair_slope(a, ratio[0] - ratio[1]);
  if (weight == 0.0) s = {0.0, 0.0};   /* whatever the logits */
  if (threadIdx.x == 0) {
    a.loss[pair] = (float)(weight * s.loss);
    if (a.seq_logp) {
      a.seq_logp[2 * pair] = (float)sum[0];
      a.seq_logp[2 * pair + 1] = (float)sum[1];
    }
  }
  if (!a.grad) return;
  const double up = weight * s.slope * (double)(a.dev ? a.dev->scale : a.scale) * (double)a.inv_tau;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float slope = (float)((k ? -up : up) * each[k]);
    for (uint64_t row = (uint64_t)seq[k].first + threadIdx.x; row < seq[k].last; row += NT) {
      const TokenPlan p = a.plan[row];
      if (p.id >= 0) a.plan[row] = make_plan(p.own, p.factor, p.from, slope, p.id);
    }
  }
}

/* ------------------------------------------------------------------------
 * The gradient from the rows' plans: a vector per thread and blocks that live
 * as long as that takes, the shape in which a copy is fastest here (16384 x
 * 32000 bf16, 6 % of the rows without a token: 310 to 330 us). Rows whose
 * gradient is zero are not read.
 * ---------------------------------------------------------------------- */
template <int DT>
struct __attribute__((packed, aligned(DT == ZS_FP32 ? 4 : 2))) LooseVec { uint32_t w[4]; };

/* By the scalar unit: the one thing that a block waits for before its logits. */
__device__ __forceinline__ TokenPlan load_plan(const TokenPlan *p, uint32_t row) {
  const float *f = reinterpret_cast<const float *>(p + row);
  return {load_scalar(f, 0), load_scalar(f, 1), load_scalar(f, 2),
          __float_as_int(load_scalar(f, 3))};
}

template <int DT, int NT, bool JOIN>
__global__ __launch_bounds__(NT) void token_grad_kernel(TokenArgs a) {
  constexpr uint32_t ve = kVecElems<DT>, esz = DT == ZS_FP32 ? 4 : 2;
  const uint32_t row = a.row0 + blockIdx.x / a.blocks, block = blockIdx.x % a.blocks;
  const char *z = static_cast<const char *>(a.z) + (uint64_t)row * a.ld * esz;
  char *g = static_cast<char *>(a.grad) + (uint64_t)row * a.gld * esz;
  const RowShape sh = row_shape<DT>(z, a.vocab);
  TokenPlan p;
  if constexpr (JOIN) {   /* few rows, whose parts every block joins for itself */
    const int32_t id = load_scalar(a.ids, row);
    p = {0.0f, 0.0f, 0.0f, kNoToken};
    if (token_live(a, row, id)) {
      const TokenPart w = join_parts<DT>(a, row);
      const TokenMass m = token_mass<DT>(w.rest, load_scalar(a.own, row),
                                     shift_of<DT>(w.from, a.log2_scale), a.log2_scale);
      const Slope k = policy_slope(a, policy_in(a, row), m.logp);
      p = make_plan(m.rest, m.total, w.from, k.slope * grad_scale(a), id);
      if (block == 0 && threadIdx.x == 0) {
        if (a.logp) a.logp[row] = (float)m.logp;
        a.loss[row] = k.loss;
      }
    }
  } else {
    p = load_plan(a.plan, row);
  }
  if (p.id == kOutside) return;
  const bool live = p.id >= 0;
  const Shift shift = shift_of<DT>(p.from, a.log2_scale);
  const uint32_t edge = block == 0 ? edge_index<DT>(sh, threadIdx.x, true, true, a.vocab) : a.vocab;
  if (edge < a.vocab) {
    float x = 0.0f;
    if (live) x = edge == (uint32_t)p.id ? p.own : term<DT>(load1<DT>(z, edge), shift) * p.factor;
    store1<DT>(g, edge, x);
  }
  const uint32_t v = block * NT + threadIdx.x;
  if (v >= sh.vecs) return;
  u32x4 w = {0, 0, 0, 0};
  if (live) {
    float e[ve];
    unpack_vec<DT>(__builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(z + sh.head * esz) + v), e);
#pragma unroll
    for (uint32_t j = 0; j < ve; ++j) e[j] = term<DT>(e[j], shift) * p.factor;
    const uint32_t at = (uint32_t)p.id - sh.head - v * ve;
    if (at < ve) {
#pragma unroll
      for (uint32_t j = 0; j < ve; ++j) e[j] = at == j ? p.own : e[j];
    }
    w = pack_vec<DT>(e);
  }
  char *to = g + sh.head * esz + (uint64_t)v * 16;
  if (((uintptr_t)(g + sh.head * esz) & 15) == 0)
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(to));
  else
    *reinterpret_cast<LooseVec<DT> *>(to) = LooseVec<DT>{{w.x, w.y, w.z, w.w}};
}

/* ------------------------------------------------------------------------
 * The policy loss of rows that a block's registers hold: ITEMS 16-byte vectors
 * per thread and, in a few threads, one single element. A block walks rows
 * blockIdx, + gridDim, ..., and while it writes a row's gradient it fetches
 * the next row into the registers that fall free; its terms are added as they
 * arrive, and one reduction parts the two sweeps. 8192 x 128000 bf16 823 us, 5.1
 * TB/s; 65536 x 4096 198 us, 5.4 (a block for each row and no walk: 964 and 205).
 * ---------------------------------------------------------------------- */
constexpr int kTokenStore = 2;   /* non-temporal: read by a later call, in whole lines */

struct TokenIn {
  const char *z;
  RowShape shape;
  uint32_t edge;
  int32_t id;
  PolicyIn policy;
  bool live;
};

template <int DT>
__device__ __forceinline__ TokenIn open_token(const TokenArgs &a, uint32_t row) {
  constexpr uint64_t esz = DT == ZS_FP32 ? 4 : 2;
  TokenIn r;
  r.z = static_cast<const char *>(a.z) + (uint64_t)row * a.ld * esz;
  r.shape = row_shape<DT>(r.z, a.vocab);
  r.id = load_scalar(a.ids, row);
  r.policy = policy_in(a, row);
  r.live = (uint32_t)r.id < a.vocab && r.policy.weight != 0.0f;
  r.edge = edge_index<DT>(r.shape, threadIdx.x, true, true, a.vocab);
  return r;
}

/* A row without a token is not read: its buffer is empty. */
template <int DT>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t token_buffer(const TokenIn &r) {
  return bounded(r.z + r.shape.head * (DT == ZS_FP32 ? 4 : 2), r.live ? r.shape.vecs * 16 : 0);
}

/* The vector at byte `at`, or the row's last for a thread past it, which the
 * sum leaves out. */
__device__ __forceinline__ u32x4 token_vec(__amdgpu_buffer_rsrc_t row, const TokenIn &r,
                                           uint32_t at) {
  const uint32_t last = (r.shape.vecs - 1) * 16, mine = at + threadIdx.x * 16;
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                       row, (int)(mine < last ? mine : last), 0, 0));
}

template <int DT>
__device__ __forceinline__ void token_singles(const TokenArgs &a, const TokenIn &r, uint32_t &own,
                                              uint32_t &single) {
  own = single = empty_vec<DT>()[0];
  if (!r.live) return;
  own = load_raw<DT>(r.z, r.id);
  if (r.edge < a.vocab && r.edge != (uint32_t)r.id) single = load_raw<DT>(r.z, r.edge);
}

/* Where a row's token lies among a block's vectors: the same for all threads,
 * so that one item of one thread is looked at, and not each for every element. */
struct TokenPlace {
  uint32_t item, thread, elem;   /* item: none of them if the token is a single element */
};

template <int DT, int NT>
__device__ __forceinline__ TokenPlace token_place(const TokenIn &r) {
  constexpr uint32_t ve = kVecElems<DT>;
  const uint32_t at = (uint32_t)r.id - r.shape.head, v = at / ve;   /* wraps for the head's */
  return {at < r.shape.vecs * ve ? v / NT : ~0u, v % NT, at % ve};
}

/* Element j of a vector in memory's form; j is the same for all threads. */
template <int DT>
__device__ __forceinline__ void set_element(u32x4 &x, uint32_t j, uint32_t bits) {
  if constexpr (DT == ZS_FP32) {
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) x[k] = j == k ? bits : x[k];
  } else {
    const uint32_t keep = j & 1 ? 0xffffu : 0xffff0000u, put = j & 1 ? bits << 16 : bits & 0xffffu;
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) x[k] = j / 2 == k ? (x[k] & keep) | put : x[k];
  }
}

template <int DT>
__device__ __forceinline__ uint32_t raw_bits(float x) {
  if constexpr (DT == ZS_FP32) return __float_as_uint(x);
  else return pack1<DT>(x);
}

template <int DT, int NT, int ITEMS>
__global__ __launch_bounds__(NT, ITEMS <= 16 ? 4 : 2) void policy_row_kernel(TokenArgs a) {
  constexpr uint32_t ve = kVecElems<DT>, esz = DT == ZS_FP32 ? 4 : 2;
  __shared__ double dpart[2][2][NT / 64];
  __shared__ float fpart[2][NT / 64];
  const uint32_t t = threadIdx.x;
  const float scale = grad_scale(a);
  uint32_t row = blockIdx.x, turn = 0;
  TokenIn in = open_token<DT>(a, row);
  uint32_t raw_own, raw_single;
  token_singles<DT>(a, in, raw_own, raw_single);
  u32x4 x[ITEMS];
  {
    const __amdgpu_buffer_rsrc_t buf = token_buffer<DT>(in);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) x[i] = token_vec(buf, in, i * (NT * 16));
  }
  for (;;) {
    /* rows are told apart by a scalar that the compiler cannot follow: it would
     * keep a pointer of its own in vector registers for every use */
    asm volatile("" : "+s"(row));
    const uint32_t next = row + gridDim.x;
    const bool more = next < a.rows;
    const TokenIn after = open_token<DT>(a, more ? next : row);
    TokenPlan plan{0.0f, 0.0f, 0.0f, kNoToken};
    const TokenPlace place = token_place<DT, NT>(in);
    float single = -INFINITY;
    if (in.live) {   /* uniform over the block */
      const float own = raw_value<DT>(raw_own);
      single = raw_value<DT>(raw_single);
      float from = own;
      double rest;
      /* the token's own term is left out of the sum, and its gradient put in below */
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
        if (place.item == (uint32_t)i && t == place.thread)
          set_element<DT>(x[i], place.elem, empty_vec<DT>()[0]);
      for (bool again = false;; again = true) {
        const Shift s = shift_of<DT>(from, a.log2_scale);
        float sum = term<DT>(single, s);
        double sum64 = 0.0;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          float e[ve];
          asm volatile("" : "+v"(x[i]));   /* unpacked anew each time */
          unpack_vec<DT>(x[i], e);
          float some = 0.0f;
#pragma unroll
          for (uint32_t j = 0; j < ve; ++j) some += term<DT>(e[j], s);
          sum += (int)t < (int)in.shape.vecs - i * NT ? some : 0;
          if (i % 4 == 3 || i == ITEMS - 1) {   /* a few of them in fp32, the rest in binary64 */
            sum64 += (double)sum;
            sum = 0.0f;
            asm volatile("" : "+v"(sum64));
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        reduce_put(sum64, SumOf{}, dpart[turn][again]);
        __syncthreads();
        rest = reduce_get<NT>(SumOf{}, dpart[turn][again]);
        /* uniform over the block */
        if (again || (rest < (double)kTokenTop && own != -INFINITY)) break;
        VecMax<DT> max;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) max.add(x[i]);
        reduce_put(fmaxf(max.get(), single), MaxOf{}, fpart[turn]);
        __syncthreads();
        from = reduce_get<NT>(MaxOf{}, fpart[turn]);
      }
      const TokenMass32 m =
          token_mass32<DT>(rest, own, shift_of<DT>(from, a.log2_scale), a.log2_scale);
      const Slope s = policy_slope(a, in.policy, m.logp);
      if (t == 0) {
        if (a.logp) a.logp[row] = m.logp;
        a.loss[row] = s.loss;
      }
      const float slope = s.slope * scale;
      plan = {from, -slope / m.total, slope * (m.rest / m.total),
              slope == 0.0f ? kNoToken : in.id};
    } else if (t == 0) {
      if (a.logp) a.logp[row] = 0.0f;
      a.loss[row] = 0.0f;
    }
    if (plan.id < 0) {   /* zeros: terms of -inf */
      plan = {0.0f, 0.0f, 0.0f, kNoToken};
      single = -INFINITY;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) x[i] = empty_vec<DT>();
    }
    const Shift shift = shift_of<DT>(plan.from, a.log2_scale);
    char *g = static_cast<char *>(a.grad) + (uint64_t)row * a.gld * esz;
    const __amdgpu_buffer_rsrc_t to = bounded(g + in.shape.head * esz, in.shape.vecs * 16);
    const __amdgpu_buffer_rsrc_t from_next = token_buffer<DT>(after);
    if (in.edge < a.vocab)
      store1<DT>(g, in.edge,
                 in.edge == (uint32_t)plan.id ? plan.own : term<DT>(single, shift) * plan.factor);
    if (more) token_singles<DT>(a, after, raw_own, raw_single);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      float e[ve];
      asm volatile("" : "+v"(x[i]));   /* unpacked anew, not kept since the sum */
      unpack_vec<DT>(x[i], e);
#pragma unroll
      for (uint32_t j = 0; j < ve; ++j) e[j] = term<DT>(e[j], shift) * plan.factor;
      u32x4 w = pack_vec<DT>(e);
      if (place.item == (uint32_t)i && t == place.thread)
        set_element<DT>(w, place.elem, raw_bits<DT>(plan.own));
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, w), to,
                                             (int)(t * 16 + i * (NT * 16)), 0, kTokenStore);
      x[i] = token_vec(from_next, after, i * (NT * 16));   /* past the last row: not used */
      __builtin_amdgcn_sched_barrier(0);
    }
    if (!more) return;
    /* A wave may still read a row's sums while another is at the next row: that
     * one has the other half of them, and no wave reaches the row after it before
     * all have passed its barrier. A row without a token has no barrier, and so
     * takes no half: the next one's would be the one that is still read. */
    if (in.live) turn ^= 1;
    row = next;
    in = after;
  }
}

}  // namespace zs
#endif  // ZS_TOKEN_KERNELS_H
