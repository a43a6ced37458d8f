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
 * Terms as in the distillation loss: 2^(z c - I), I whole.
 *
 * Bound by HBM.
 */
#ifndef ZS_TOKEN_KERNELS_H
#define ZS_TOKEN_KERNELS_H

#include "zs_logits.h"

namespace zs {

/* Statistics of one part of a row: its maximum, and the sum of its terms but
 * the token's. */
struct TokenPart {
  double rest;
  float max, pad;
};

/* What a row's gradient is made of: term * factor, and `own` for token id. */
struct TokenPlan {
  float max, factor, own;
  int32_t id;      /* < 0: zeros, and the logits are not read */
};

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
  TokenPlan *plan;                 /* [rows] */
  float *own;                      /* [rows]: the tokens' logits */
  uint64_t ld, gld;
  uint32_t rows, vocab, parts, part_vecs;
  float log2_scale, inv_tau, scale;   /* log2_scale = log2(e) / tau */
};

/* Rows of the sequences, first and one past the last. */
struct TokenSpan {
  uint32_t first, last;
};

__device__ __forceinline__ uint32_t row_of(int32_t start, uint32_t rows) {
  return start < 0 ? 0u : (uint32_t)start < rows ? (uint32_t)start : rows;
}

__device__ __forceinline__ TokenSpan token_span(const TokenArgs &a) {
  if (!a.starts) return {0, a.rows};
  return {row_of(a.starts[0], a.rows), row_of(a.starts[2 * a.pairs], a.rows)};
}

__device__ __forceinline__ bool token_live(const TokenArgs &a, uint32_t row, int32_t id) {
  return (uint32_t)id < a.vocab && (!a.weight || a.weight[row] != 0.0f);
}

/* What turns a sum of terms by shift `own` into one by shift `to`, a power of
 * two; 0 where the two scale differently or lie too far apart. */
__device__ __forceinline__ double shift_factor(float max, const Shift &own, const Shift &to) {
  const float by = own.whole - to.whole;
  const bool some = max != -INFINITY && own.c == to.c && by > -800.0f;
  return __hiloint2double(some ? (1023 + (int)by) << 20 : 0, 0);
}

/* ------------------------------------------------------------------------
 * A row's token: its share of the softmax and its log-probability. `rest` and
 * `own` are the sums of the other terms and its own.
 * ---------------------------------------------------------------------- */
struct TokenMass {
  double rest, total, logp;
};

__device__ __forceinline__ TokenMass token_mass(double rest, float z, const Shift &s) {
  TokenMass m;
  const double own = (double)term(z, s);
  m.rest = rest;
  m.total = rest + own;
  if (rest <= own && own > 0.0)
    m.logp = -log1p(rest / own);
  else   /* NaN: comes here */
    m.logp = fma((double)z, (double)s.c, -(double)s.whole) * 0.69314718055994531 - log(m.total);
  return m;
}

/* exp(d) - 1 - d, by its series near 0, where the difference would leave
 * rounding. */
__device__ __forceinline__ float exp_rest(float d) {
  if (d == INFINITY) return d;   /* not the difference of two infinities */
  if (!(fabsf(d) < 1.0f)) return expf(d) - 1.0f - d;
  float s = 1.0f + d * (1.0f / 12.0f);
#pragma unroll
  for (int k = 11; k > 2; --k) s = fmaf(d * (1.0f / (float)k), s, 1.0f);
  return 0.5f * d * d * s;
}

struct Slope {
  float loss, slope;   /* slope: of the loss in the log-probability */
};

__device__ __forceinline__ Slope policy_slope(const TokenArgs &a, uint32_t row, double logp,
                                              float weight) {
  const float adv = a.advantage[row];
  const float r = a.old_logp ? expf((float)(logp - (double)a.old_logp[row])) : 1.0f;
  const float low = 1.0f - a.clip_low, high = 1.0f + a.clip_high;
  const bool above = adv > 0.0f && r > high, below = adv < 0.0f && r < low;
  Slope s;
  s.loss = -(above ? high : below ? low : r) * adv;
  s.slope = above || below ? 0.0f : -r * adv;
  if (a.ref_logp) {
    const float d = (float)((double)a.ref_logp[row] - logp), rest = exp_rest(d);
    s.loss = fmaf(a.kl_weight, rest, s.loss);
    s.slope = fmaf(-a.kl_weight, d + rest, s.slope);
  }
  s.loss *= weight;
  s.slope *= weight;
  return s;
}

/* A row's plan from its mass and the slope times loss scale and 1 / tau. */
__device__ __forceinline__ TokenPlan make_plan(const TokenMass &m, float max, float slope,
                                               int32_t id) {
  TokenPlan p;
  p.max = max;
  p.factor = (float)(-(double)slope / m.total);
  p.own = (float)((double)slope * (m.rest / m.total));
  p.id = slope == 0.0f ? -1 : id;
  return p;
}

/* ------------------------------------------------------------------------
 * Statistics: a block per part of a row, each thread with a maximum and sum
 * of its own that follow the vectors as they come, U of them under way at a
 * time, so that each logit is read once; then joined. A thread's sums of
 * U vectors are fp32, what they are added to binary64.
 * ---------------------------------------------------------------------- */
constexpr int kTokenAhead = 4;

template <int DT>
__device__ __forceinline__ void leave_out(const RowShape &s, int32_t id, uint32_t v,
                                          float (&e)[kVecElems<DT>]) {
  constexpr uint32_t ve = kVecElems<DT>;
  const uint32_t at = (uint32_t)id - s.head - v * ve;   /* wraps for what is before */
  if (at >= ve) return;
#pragma unroll
  for (uint32_t j = 0; j < ve; ++j) e[j] = at == j ? -INFINITY : e[j];
}

/* The row's results, where one block has seen all of it: log-probability,
 * policy loss and plan, as far as they are asked for. One thread. */
__device__ __forceinline__ void finish_token(const TokenArgs &a, uint32_t row, double rest,
                                             float max, float z, int32_t id) {
  const TokenMass m = token_mass(rest, z, shift_of(max, a.log2_scale));
  if (a.logp) a.logp[row] = (float)m.logp;
  if (!a.loss) return;
  const Slope s = policy_slope(a, row, m.logp, a.weight ? a.weight[row] : 1.0f);
  a.loss[row] = s.loss;
  if (a.grad)
    a.plan[row] = make_plan(m, max, s.slope * (a.dev ? a.dev->scale : a.scale) * a.inv_tau, id);
}

template <int DT, int NT>
__global__ __launch_bounds__(NT) void token_stats_kernel(TokenArgs a) {
  constexpr uint32_t ve = kVecElems<DT>, esz = DT == ZS_FP32 ? 4 : 2;
  constexpr int U = kTokenAhead;
  __shared__ float fpart[NT / 64];
  __shared__ double dpart[NT / 64];
  const uint32_t row = blockIdx.x / a.parts, part = blockIdx.x % a.parts, t = threadIdx.x;
  const TokenSpan span = token_span(a);
  if (row < span.first || row >= span.last) return;
  const int32_t id = a.ids[row];
  const bool live = token_live(a, row, id), says = part == 0 && t == 0;
  if (says) {
    if (a.plan) a.plan[row] = {0.0f, 0.0f, 0.0f, -1};
    if (!live) {
      if (a.logp) a.logp[row] = 0.0f;
      if (a.loss && !a.starts) a.loss[row] = 0.0f;
    }
  }
  if (!live) return;
  const char *z = static_cast<const char *>(a.z) + (uint64_t)row * a.ld * esz;
  const RowShape sh = row_shape<DT>(z, a.vocab);
  const u32x4 *zv = reinterpret_cast<const u32x4 *>(z + sh.head * esz);
  const uint32_t v0 = part * a.part_vecs;
  const uint32_t v1 = v0 + a.part_vecs < sh.vecs ? v0 + a.part_vecs : sh.vecs;
  const uint32_t edge = edge_index<DT>(sh, t, part == 0, part == a.parts - 1, a.vocab);
  const float own = load1<DT>(z, id);
  float max = edge < a.vocab ? load1<DT>(z, edge) : -INFINITY;
  Shift shift = shift_of(max, a.log2_scale);
  double sum = edge < a.vocab && edge != (uint32_t)id ? (double)term(max, shift) : 0.0;
  for (uint32_t v = v0 + t; v < v1; v += U * NT) {
    u32x4 x[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      x[i] = v + i * NT < v1 ? zv[v + i * NT] : empty_vec<DT>();
    VecMax<DT> top;
#pragma unroll
    for (int i = 0; i < U; ++i) top.add(x[i]);
    if (top.get() > max) {
      const Shift to = shift_of(top.get(), a.log2_scale);
      sum *= shift_factor(max, shift, to);
      max = top.get();
      shift = to;
    }
    float some = 0.0f;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float e[ve];
      unpack_vec<DT>(x[i], e);
      leave_out<DT>(sh, id, v + i * NT, e);
#pragma unroll
      for (uint32_t j = 0; j < ve; ++j) some += term(e[j], shift);
    }
    sum += (double)some;
  }
  reduce_put(max, MaxOf{}, fpart);
  __syncthreads();
  const float top = reduce_get<NT>(MaxOf{}, fpart);
  sum *= shift_factor(max, shift, shift_of(top, a.log2_scale));
  reduce_put(sum, SumOf{}, dpart);
  __syncthreads();
  sum = reduce_get<NT>(SumOf{}, dpart);
  if (t != 0) return;
  if (part == 0 && a.own) a.own[row] = own;
  if (a.parts == 1 && !a.starts) finish_token(a, row, sum, top, own, id);
  else a.ws[(uint64_t)row * a.parts + part] = {sum, top, 0.0f};
}

/* All of a row's parts. */
__device__ __forceinline__ TokenPart join_parts(const TokenArgs &a, uint32_t row) {
  const TokenPart *w = a.ws + (uint64_t)row * a.parts;
  TokenPart r{0.0, -INFINITY, 0.0f};
  for (uint32_t i = 0; i < a.parts; ++i) r.max = fmaxf(r.max, w[i].max);
  const Shift to = shift_of(r.max, a.log2_scale);
  for (uint32_t i = 0; i < a.parts; ++i)
    r.rest += w[i].rest * shift_factor(w[i].max, shift_of(w[i].max, a.log2_scale), to);
  return r;
}

/* Rows in parts: a thread per row joins them. */
__global__ __launch_bounds__(64) void token_finish_kernel(TokenArgs a) {
  const uint32_t row = blockIdx.x * 64 + threadIdx.x;
  if (row >= a.rows) return;
  const int32_t id = a.ids[row];
  if (!token_live(a, row, id)) return;
  const TokenPart p = join_parts(a, row);
  finish_token(a, row, p.rest, p.max, a.own[row], id);
}

/* ------------------------------------------------------------------------
 * Pairs: a block per pair sums its sequences' log-probabilities, in binary64
 * and in a fixed order, forms the loss and gives every row its plan.
 * ---------------------------------------------------------------------- */
constexpr int kPairThreads = 256;

struct PairSlope {
  double loss, slope;   /* slope: of the loss in the difference of log ratios */
};

__device__ __forceinline__ PairSlope pair_slope(const TokenArgs &a, double delta) {
  const double beta = a.beta, m = beta * delta;
  if (a.kind == ZS_PREFERENCE_SIGMOID) {
    const double eps = a.smoothing, small = log1p(exp(-fabs(m)));
    const double up = m > 0.0 ? m : 0.0, down = m > 0.0 ? 0.0 : -m;   /* NaN: small is one */
    return {(1.0 - eps) * (small + down) + eps * (small + up),
            beta * (eps / (1.0 + exp(-m)) - (1.0 - eps) / (1.0 + exp(m)))};
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
  double sum[2], count[2];
  TokenSpan seq[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    seq[k] = {row_of(a.starts[2 * pair + k], a.rows), row_of(a.starts[2 * pair + k + 1], a.rows)};
    sum[k] = count[k] = 0.0;
    for (uint64_t row = (uint64_t)seq[k].first + threadIdx.x; row < seq[k].last; row += NT) {
      const int32_t id = a.ids[row];
      if (!token_live(a, row, id)) continue;
      const TokenPart p = join_parts(a, row);
      sum[k] += token_mass(p.rest, a.own[row], shift_of(p.max, a.log2_scale)).logp;
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
      const int32_t id = a.ids[row];
      if (!token_live(a, row, id)) continue;
      const TokenPart p = join_parts(a, row);
      const TokenMass m = token_mass(p.rest, a.own[row], shift_of(p.max, a.log2_scale));
      a.plan[row] = make_plan(m, p.max, slope, id);
    }
  }
}

/* ------------------------------------------------------------------------
 * The gradient of a part of a row, from its plan: read once, written once;
 * rows whose gradient is zero are not read.
 * ---------------------------------------------------------------------- */
template <int DT>
struct __attribute__((packed, aligned(DT == ZS_FP32 ? 4 : 2))) LooseVec { uint32_t w[4]; };

template <int DT, int NT>
__global__ __launch_bounds__(NT) void token_grad_kernel(TokenArgs a) {
  constexpr uint32_t ve = kVecElems<DT>, esz = DT == ZS_FP32 ? 4 : 2;
  constexpr int U = kTokenAhead;
  const uint32_t row = blockIdx.x / a.parts, part = blockIdx.x % a.parts, t = threadIdx.x;
  const TokenSpan span = token_span(a);
  const bool inside = row >= span.first && row < span.last;
  if (!inside && !a.clear) return;
  const TokenPlan p = inside ? a.plan[row] : TokenPlan{0.0f, 0.0f, 0.0f, -1};
  const char *z = static_cast<const char *>(a.z) + (uint64_t)row * a.ld * esz;
  char *g = static_cast<char *>(a.grad) + (uint64_t)row * a.gld * esz;
  const RowShape sh = row_shape<DT>(z, a.vocab);
  const u32x4 *zv = reinterpret_cast<const u32x4 *>(z + sh.head * esz);
  const uint32_t v0 = part * a.part_vecs;
  const uint32_t v1 = v0 + a.part_vecs < sh.vecs ? v0 + a.part_vecs : sh.vecs;
  const uint32_t edge = edge_index<DT>(sh, t, part == 0, part == a.parts - 1, a.vocab);
  const bool live = p.id >= 0, vec = ((uintptr_t)(g + sh.head * esz) & 15) == 0;
  const Shift shift = shift_of(p.max, a.log2_scale);
  if (edge < a.vocab) {
    float x = 0.0f;
    if (live) x = edge == (uint32_t)p.id ? p.own : term(load1<DT>(z, edge), shift) * p.factor;
    store1<DT>(g, edge, x);
  }
  auto put = [&](uint32_t v, const u32x4 &w) {
    char *to = g + sh.head * esz + (uint64_t)v * 16;
    if (vec) __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(to));
    else *reinterpret_cast<LooseVec<DT> *>(to) = LooseVec<DT>{{w.x, w.y, w.z, w.w}};
  };
  if (!live) {
    for (uint32_t v = v0 + t; v < v1; v += NT) put(v, u32x4{0, 0, 0, 0});
    return;
  }
  for (uint32_t v = v0 + t; v < v1; v += U * NT) {
    u32x4 x[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      x[i] = v + i * NT < v1 ? zv[v + i * NT] : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (v + i * NT >= v1) break;
      float e[ve];
      unpack_vec<DT>(x[i], e);
#pragma unroll
      for (uint32_t j = 0; j < ve; ++j) e[j] = term(e[j], shift) * p.factor;
      const uint32_t at = (uint32_t)p.id - sh.head - (v + i * NT) * ve;
      if (at < ve) {
#pragma unroll
        for (uint32_t j = 0; j < ve; ++j) e[j] = at == j ? p.own : e[j];
      }
      put(v + i * NT, pack_vec<DT>(e));
    }
  }
}

}  // namespace zs
#endif  // ZS_TOKEN_KERNELS_H
