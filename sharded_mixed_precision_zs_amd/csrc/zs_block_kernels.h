/*
 * zs_block_kernels.h -- a block's end (gfx950): its output normed, gated,
 * dropped out, scaled and added to the scaled residual stream, and the next
 * block's norm of the sum; forward and backward.
 *
 *   n = x r1 g1 gate,  r1 = 1 / sqrt(mean(x^2) + eps)
 *   h = R16(l res + a k n)       k: 0, or 1 / (1 - p)
 *   y = h r2 g2,       r2 = 1 / sqrt(mean(h^2) + eps)
 *
 *   dh = dres + r2 (g2 dy - h r2^2 mean(g2 dy h))
 *   t = a k dh;  u = sum over rows of t x r1;  dgate = g1 u;  dg1 = gate u
 *   dx = r1 (q - x r1^2 mean(q x)),  q = t g1 gate
 *   dres' = l dh;  dg2 = sum over rows of dy h r2
 *
 * The gate is one vector for all rows, so that its gradient and that of the
 * first gain are one sum u, times the other. Without the first norm r1 and g1
 * are 1 and dx = q.
 *
 * Bound by HBM, the forward pass nearly as much by its instructions: every
 * element is read once, stays in registers over both sums of its row, and is
 * written once (16384 x 4096 bf16 with dropout and an 8-bit y: 92 us, 5.1 TB/s,
 * without dropout 83 to 90; the gradient 147 us, 5.4 TB/s, and 5 us for the sums
 * over rows).
 */
#ifndef ZS_BLOCK_KERNELS_H
#define ZS_BLOCK_KERNELS_H

#include "zs_logits.h"
#include "zs_norm_rows.h"
#include "zs_philox.h"

namespace zs {

struct BlockArgs {
  const void *x, *res, *post_gain, *gate, *gain;   /* post_gain, gate optional */
  uint16_t *h, *y;                                 /* y optional */
  float *post_rstd, *rstd;                         /* optional */
  uint8_t *codes, *scales;                         /* both or neither */
  uint64_t rows;
  uint32_t cols, padded;
  float eps;
  double inv_cols, residual_scale, branch_scale;
  float near_dropped;   /* 2^-100 where residual_scale times 16 bits is exact, else 2^-22 */
  DropArgs drop;
};

/* v rounded to odd in fp32: where it is no float, to the neighbour whose last
 * bit is set. Rounded again to 16 bits this gives what v gives. */
__device__ __forceinline__ float odd_float(double v) {
  const float y = (float)v;
  const float rest = (float)(v - (double)y);
  const int b = __float_as_int(y);
  const int odd = (b + ((b ^ __float_as_int(rest)) >> 31)) | 1;
  constexpr int kFiniteNotZero = 0x198;   /* normal and subnormal, of either sign */
  return __int_as_float(__builtin_amdgcn_classf(rest, kFiniteNotZero) ? odd : b);
}

/* Eight sums l r + c p rounded once to 16 bits. In fp32 a sum is off by at most
 * kNear times |l r| + |sum|: c p by 2^-24 for c's rounding, and as much for p's
 * in fp16, l r, the sum and its ends by 2^-24 each; or by nothing where p is 0
 * and l r exact, and `near` so small that both ends are the sum (0 would make
 * NaN of an infinite size, at both ends alike). Where both ends of that have the
 * same 16 bits, those are the exact sum's. Where they differ, in some 2^-12 of
 * bf16 sums and 2^-9 of fp16's, the two of a word are formed in binary64. (Short
 * scales without a first norm make ties, and go that way more often. Where a sum
 * is below fp32's normal range, 2^-150 more may be off, 2^-17 of bf16's step
 * there.) */
template <int DT>
constexpr float kNear = DT == ZS_FP16 ? 0x1p-22f : 0x1.8p-23f;

template <int DT>
__device__ __forceinline__ u32x4 sums16(const float (&p)[8], const float (&low)[8],
                                        const float (&r)[8], const float (&near)[8], double c,
                                        double l, const RandomWords &words, uint32_t threshold) {
  const float cf = (float)c, lf = (float)l;
  /* a scale that is no number reaches what is kept alone; and one below fp32's
   * normal range is off by more than 2^-24 */
  const uint32_t always =
      c == 0.0 || (fabsf(cf) >= 0x1p-126f && fabsf(cf) < INFINITY) ? 0 : 1;
  u32x4 w;
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    float up[2], down[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float lr = lf * r[j + k], sum = fmaf(cf, p[j + k], lr), size = fabsf(lr) + fabsf(sum);
      up[k] = fmaf(size, near[j + k], sum);
      down[k] = fmaf(size, -near[j + k], sum);
    }
    w[j / 2] = pack2<DT>(up[0], up[1]);
    if ((w[j / 2] ^ pack2<DT>(down[0], down[1])) | always) {
      float o[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const double lr = l * (double)r[j + k];   /* exact: 35 bits */
        double whole = p[j + k];
        if constexpr (DT == ZS_FP16) whole += (double)low[j + k];
        const double sum = fma(c, whole, lr);
        o[k] = odd_float(!threshold || kept(words, j + k, threshold) ? sum : lr);
      }
      w[j / 2] = pack2<DT>(o[0], o[1]);
    }
  }
  return w;
}

/* Eight products hg (hi + lo), so that their 16 or 8 bits are the exact ones'.
 * To nearest in fp32 does, but where that makes a tie of what is none (or a
 * power of two, a block's scale): then its low 12 bits are 0, in one of 4096,
 * and the eight are rounded to odd. */
__device__ __forceinline__ void times8(const float (&hg)[8], const RowScale &s, float (&y)[8]) {
  uint32_t low = ~0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    y[j] = fmaf(hg[j], s.hi, hg[j] * s.lo);
    const uint32_t b = __float_as_uint(y[j]) & 0xfffu;
    low = low < b ? low : b;
  }
  if (low == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = times_odd(hg[j], s);
  }
}

/* Sum over the G threads of a row's group, on all of them, in a fixed tree: by
 * lane moves within 16 lanes, which cost no LDS. `part`: G / 64 values in LDS
 * that nothing else uses before the next barrier. */
template <int G, class T>
__device__ __forceinline__ T row_sum(T v, T *part) {
  v = wave_reduce(v, SumOf{}, 64);
  if constexpr (G > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x / 64 % (G / 64)] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < G / 64; ++w) v += part[w];
  }
  return v;
}

/* As norm_kernel: a row per group of G threads, ITEMS vectors of eight each.
 * The sum that becomes h is rounded once, so that h is the 64-bit result's
 * own, and with it what the second norm and its codes see. */
template <int DT, bool AL, int G, int ITEMS>
__global__ __launch_bounds__(G < 128 ? 256 : G) void block_kernel(BlockArgs a) {
  constexpr int kRows = G < 128 ? 256 / G : 1;
  __shared__ double part[2][G / 64];
  const uint32_t t = threadIdx.x % G;
  const uint64_t row = (uint64_t)blockIdx.x * kRows + threadIdx.x / G;
  if (row >= a.rows) return;   /* a whole wave; blocks of one row never take it */
  const uint16_t *x = static_cast<const uint16_t *>(a.x) + row * a.cols;
  const uint16_t *res = static_cast<const uint16_t *>(a.res) + row * a.cols;
  Raw16<8> xr[ITEMS], rr[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) xr[i] = load8_ahead<AL>(x, (i * G + t) * 8, a.cols);
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) rr[i] = load8_ahead<AL>(res, (i * G + t) * 8, a.cols);
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    settle8<AL>(xr[i], (i * G + t) * 8, a.cols);
    settle8<AL>(rr[i], (i * G + t) * 8, a.cols);
  }
  /* the vectors too, before anything waits: they come from the caches */
  Raw16<8> gr[ITEMS], tr[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    if (a.post_gain) gr[i] = load8_raw<AL>(a.post_gain, (uint64_t)(i * G + t) * 8, a.cols);
    if (a.gate) tr[i] = load8_raw<AL>(a.gate, (uint64_t)(i * G + t) * 8, a.cols);
  }
  double scale = a.branch_scale;
  if (a.post_gain) {
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      float e[8];
      upcast<8, DT>(xr[i], e);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fma((double)e[j], (double)e[j], ss);
    }
    const double r1 = row_scale64(row_sum<G>(ss, part[0]), a.inv_cols, a.eps);
    if (a.post_rstd && t == 0) a.post_rstd[row] = (float)r1;
    scale *= r1;
  }
  const uint64_t offset = a.drop.threshold ? drop_offset(a.drop) : 0;
  if (a.drop.threshold) scale *= a.drop.factor64;
  float h[ITEMS][8];
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const uint32_t v = i * G + t;
    float p[8], low[8] = {}, r[8], g[8];
    upcast<8, DT>(xr[i], p);
    upcast<8, DT>(rr[i], r);
    if (a.post_gain) {
      upcast<8, DT>(gr[i], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] *= g[j];   /* exact: 22 bits at most */
    }
    if (a.gate) {
      upcast<8, DT>(tr[i], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float q = p[j] * g[j];   /* exact in bf16, 33 bits in fp16 */
        if constexpr (DT == ZS_FP16) low[j] = fmaf(p[j], g[j], -q);
        p[j] = q;
      }
    }
    RandomWords words{};
    float near[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) near[j] = kNear<DT>;
    if (a.drop.threshold) {
      words = random_words(a.drop, offset, v, (uint32_t)row);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool stays = kept(words, j, a.drop.threshold);
        p[j] = stays ? p[j] : 0.0f;
        near[j] = stays ? kNear<DT> : a.near_dropped;
        if constexpr (DT == ZS_FP16) low[j] = stays ? low[j] : 0.0f;
      }
    }
    u32x4 w = sums16<DT>(p, low, r, near, scale, a.residual_scale, words,
                         a.drop.threshold);
    if (!AL || v * 8 >= a.cols) {
      /* past the row's end x and res are 0, and so is h, but 0 * inf is not */
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (v * 8 + 2 * j >= a.cols) w[j] = 0;
        else if (v * 8 + 2 * j + 1 >= a.cols) w[j] &= 0xffffu;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[i][2 * j] = up_lo<DT>(w[j]);
      h[i][2 * j + 1] = up_hi<DT>(w[j]);
    }
    store8_raw<AL, true>(a.h + row * a.cols, (uint64_t)v * 8, a.cols, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fma((double)h[i][j], (double)h[i][j], ss);
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) gr[i] = load8_raw<AL>(a.gain, (uint64_t)(i * G + t) * 8, a.cols);
  ss = row_sum<G>(ss, part[1]);
  const RowScale rstd = row_scale(ss, a.inv_cols, a.eps);
  if (a.rstd && t == 0) a.rstd[row] = rstd.hi;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const uint32_t v = i * G + t;
    if (v * 8 >= a.padded) break;   /* whole quads: padded is a multiple of 128 */
    float g[8], y[8];
    upcast<8, DT>(gr[i], g);
    uint32_t top = 0;
    const RowScale s = v * 8 < a.cols ? rstd : RowScale{0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] *= h[i][j];
    times8(g, s, y);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = umax(top, mag_bits(y[j]));
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

struct BlockGradArgs {
  const void *dy, *h, *gain, *dres, *x, *post_gain, *gate;   /* dres, x, post_gain, gate optional */
  const float *rstd, *post_rstd;
  uint16_t *dx, *dresidual;
  float *part;                   /* [parts][2][cols]: shares of dg2, and of u */
  uint64_t rows;
  uint32_t cols, parts;
  float residual_scale, branch_scale;
  DropArgs drop;
};

/* A thread's vectors of a row. */
template <bool AL, int G, int ITEMS>
__device__ __forceinline__ void load_grad(const void *m, uint64_t at, uint32_t t, uint32_t cols,
                                          Raw16<8> (&r)[ITEMS]) {
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
    r[i] = load8_ahead<AL>(static_cast<const uint16_t *>(m) + at, (i * G + t) * 8, cols);
}

/* As norm_grad_kernel: `parts` groups walk the rows and keep their shares of
 * both sums over rows in registers; block_gain_kernel adds the shares in
 * order. Two barriers a row, one for each of its two dot products. What the
 * first needs of the next row is fetched as soon as its registers are free,
 * the rest while the row's own first sum is joined: in registers for no more
 * than a row, two blocks share a CU's. */
template <int DT, bool AL, int G, int ITEMS>
__global__ __launch_bounds__(G < 128 ? 256 : G, 4) void block_grad_kernel(BlockGradArgs a) {
  constexpr int kRows = G < 128 ? 256 / G : 1;   /* several only without barriers */
  __shared__ float sums[2][2][G / 64];
  const uint32_t t = threadIdx.x % G;
  /* the same for a whole wave: its rows' addresses are scalars */
  const uint32_t p =
      (uint32_t)__builtin_amdgcn_readfirstlane((int)(blockIdx.x * kRows + threadIdx.x / G));
  if (p >= a.parts) return;
  /* both sums' shares: in registers, or where a block of 1024 threads has two
   * vectors each, in LDS, a word of its own for each of a thread's */
  constexpr bool kInLds = G == 1024 && ITEMS == 2;
  __shared__ float acc[kInLds ? ITEMS * 16 * G : 1];
  float shares[kInLds ? 1 : ITEMS][2][8];
  auto share = [&](int i, int which, int j) -> float & {
    if constexpr (kInLds) return acc[((i * 2 + which) * 8 + j) * G + t];
    else return shares[i][which][j];
  };
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) share(i, 0, j) = share(i, 1, j) = 0.0f;
  /* gain, and g1 gate (exact): held where a thread has one vector, else from
   * the caches for every row */
  float g0[8], q0[8];
  auto vectors = [&](int i, float (&g)[8], float (&q)[8]) {
    load8<DT, AL>(a.gain, (uint64_t)(i * G + t) * 8, a.cols, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = 1.0f;
    if (a.post_gain) load8<DT, AL>(a.post_gain, (uint64_t)(i * G + t) * 8, a.cols, q);
    if (a.gate) {
      float gate[8];
      load8<DT, AL>(a.gate, (uint64_t)(i * G + t) * 8, a.cols, gate);
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] *= gate[j];
    }
  };
  vectors(0, g0, q0);
  const uint64_t offset = a.drop.threshold ? drop_offset(a.drop) : 0;
  const float scale = a.drop.threshold ? a.branch_scale * a.drop.factor : a.branch_scale;
  const float inv_cols = 1.0f / (float)a.cols;
  Raw16<8> rdy[ITEMS], rh[ITEMS], rdres[ITEMS], rx[ITEMS];
  load_grad<AL, G>(a.dy, (uint64_t)p * a.cols, t, a.cols, rdy);
  load_grad<AL, G>(a.h, (uint64_t)p * a.cols, t, a.cols, rh);
  int turn = 0;
  for (uint64_t row = p; row < a.rows; row += a.parts, turn ^= 1) {
    const uint64_t at = row * a.cols;
    if (a.dres) load_grad<AL, G>(a.dres, at, t, a.cols, rdres);
    if (a.x) load_grad<AL, G>(a.x, at, t, a.cols, rx);
    const float rstd = a.rstd[row], post_rstd = a.post_rstd ? a.post_rstd[row] : 1.0f;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      float h[8], d[8];
      settle8<AL>(rdy[i], (i * G + t) * 8, a.cols);
      settle8<AL>(rh[i], (i * G + t) * 8, a.cols);
      upcast<8, DT>(rdy[i], d);
      upcast<8, DT>(rh[i], h);
      if constexpr (ITEMS > 1) load8<DT, AL>(a.gain, (uint64_t)(i * G + t) * 8, a.cols, g0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        share(i, 0, j) = fmaf(d[j], h[j] * rstd, share(i, 0, j));
        dot = fmaf(d[j] * g0[j], h[j], dot);
      }
    }
    const float s = row_sum<G>(dot, sums[turn][0]) * inv_cols * rstd * rstd;
    float dn[ITEMS][8];
    dot = 0.0f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      float h[8], d[8], o[8] = {}, x[8] = {};
      asm volatile("" : "+v"(rdy[i].w[0]), "+v"(rh[i].w[0]));   /* unpacked anew, not kept */
      if (a.dres) settle8<AL>(rdres[i], (i * G + t) * 8, a.cols);
      if (a.x) settle8<AL>(rx[i], (i * G + t) * 8, a.cols);
      upcast<8, DT>(rdy[i], d);
      upcast<8, DT>(rh[i], h);
      if (a.dres) upcast<8, DT>(rdres[i], o);
      if constexpr (ITEMS > 1) vectors(i, g0, q0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o[j] = fmaf(rstd, fmaf(-h[j], s, d[j] * g0[j]), o[j]);   /* dh */
        d[j] = o[j] * a.residual_scale;
        o[j] *= scale;
      }
      store8<DT, AL, true>(a.dresidual + at, (uint64_t)(i * G + t) * 8, a.cols, d);
      if (a.x) upcast<8, DT>(rx[i], x);
      if (a.drop.threshold) {
        const RandomWords w = random_words(a.drop, offset, i * G + t, (uint32_t)row);
#pragma unroll
        for (int j = 0; j < 8; ++j) {   /* x too: 0 times what was replaced could be NaN */
          const bool stays = kept(w, j, a.drop.threshold);
          o[j] = stays ? o[j] : 0.0f;
          x[j] = stays ? x[j] : 0.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        share(i, 1, j) = fmaf(o[j], x[j] * post_rstd, share(i, 1, j));
        dn[i][j] = o[j] * q0[j];
        dot = fmaf(dn[i][j], x[j], dot);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (row + a.parts < a.rows) {
      load_grad<AL, G>(a.dy, at + (uint64_t)a.parts * a.cols, t, a.cols, rdy);
      load_grad<AL, G>(a.h, at + (uint64_t)a.parts * a.cols, t, a.cols, rh);
    }
    float s1 = 0.0f;
    if (a.post_gain) s1 = row_sum<G>(dot, sums[turn][1]) * inv_cols * post_rstd * post_rstd;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (a.post_gain) {
        float x[8];
        upcast<8, DT>(rx[i], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) dn[i][j] = post_rstd * fmaf(-x[j], s1, dn[i][j]);
      }
      store8<DT, AL, true>(a.dx + at, (uint64_t)(i * G + t) * 8, a.cols, dn[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t c = (i * G + t) * 8 + j;
      if (c < a.cols) {
        a.part[(uint64_t)p * 2 * a.cols + c] = share(i, 0, j);
        if (a.x) a.part[((uint64_t)p * 2 + 1) * a.cols + c] = share(i, 1, j);
      }
    }
}

/* A thread's eight elements of a row, from memory. */
template <int DT, bool AL>
struct BlockGradVec {
  float d[8], h[8], g[8], e[8], x[8], q[8];   /* e: dres + r2 g2 dy; q: g1 gate */
  bool kept[8];

  __device__ __forceinline__ BlockGradVec(const BlockGradArgs &a, uint64_t row, uint32_t v,
                                          float rstd, uint64_t offset) {
    const uint64_t at = row * a.cols, c = (uint64_t)v * 8;
    load8<DT, AL>(static_cast<const uint16_t *>(a.dy) + at, c, a.cols, d);
    load8<DT, AL>(static_cast<const uint16_t *>(a.h) + at, c, a.cols, h);
    load8<DT, AL>(a.gain, c, a.cols, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = x[j] = 0.0f, q[j] = 1.0f, kept[j] = true;
    if (a.dres) load8<DT, AL>(static_cast<const uint16_t *>(a.dres) + at, c, a.cols, e);
    if (a.x) load8<DT, AL>(static_cast<const uint16_t *>(a.x) + at, c, a.cols, x);
    if (a.post_gain) load8<DT, AL>(a.post_gain, c, a.cols, q);
    if (a.gate) {
      float gate[8];
      load8<DT, AL>(a.gate, c, a.cols, gate);
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] *= gate[j];
    }
    if (a.drop.threshold) {
      const RandomWords w = random_words(a.drop, offset, v, (uint32_t)row);
#pragma unroll
      for (int j = 0; j < 8; ++j) kept[j] = zs::kept(w, j, a.drop.threshold);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = fmaf(rstd, d[j] * g[j], e[j]);
  }
};

/* Rows whose vectors and shares a block's registers and LDS do not hold: read
 * twice, and their shares added to in memory, a word of its own for each of a
 * thread's (2048 x 32768 bf16 400 us; held as above, for the most part in
 * scratch memory, 1262). One reduction a row: with n = h r2 and dh = e - n c,
 * mean(q x) = (sum(q k e x) - c sum(q k n x)) a / cols. With n in place of h
 * c has dh's size: h's c is r2 times that, and its sum 1 / r2 times, which leave
 * fp32 for bf16 rows beyond 1e19 or below 1e-19. */
template <int DT, bool AL>
__global__ __launch_bounds__(1024) void block_grad_wide_kernel(BlockGradArgs a) {
  constexpr int G = 1024;
  __shared__ float sums[2][3][G / 64];
  const uint32_t t = threadIdx.x, p = blockIdx.x, vecs = (a.cols + 7) / 8;
  const uint64_t offset = a.drop.threshold ? drop_offset(a.drop) : 0;
  const float scale = a.drop.threshold ? a.branch_scale * a.drop.factor : a.branch_scale;
  const float inv_cols = 1.0f / (float)a.cols;
  float *own = a.part + (uint64_t)p * 2 * a.cols;
  int turn = 0;
  for (uint64_t row = p; row < a.rows; row += a.parts, turn ^= 1) {
    const float rstd = a.rstd[row], post_rstd = a.post_rstd ? a.post_rstd[row] : 1.0f;
    float dot = 0.0f, dot_e = 0.0f, dot_h = 0.0f;
    for (uint32_t v = t; v < vecs; v += G) {
      const BlockGradVec<DT, AL> m(a, row, v, rstd, offset);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = m.h[j] * rstd;
        dot = fmaf(m.d[j] * m.g[j], n, dot);
        if (m.kept[j]) {   /* else x may be no number */
          dot_e = fmaf(scale * m.e[j] * m.q[j], m.x[j], dot_e);
          dot_h = fmaf(scale * n * m.q[j], m.x[j], dot_h);
        }
      }
    }
    const float c = row_sum<G>(dot, sums[turn][0]) * inv_cols * rstd;
    float s1 = 0.0f;
    if (a.post_gain) {
      dot_e = row_sum<G>(dot_e, sums[turn][1]);
      dot_h = row_sum<G>(dot_h, sums[turn][2]);
      s1 = fmaf(-c, dot_h, dot_e) * inv_cols * post_rstd * post_rstd;
    }
    for (uint32_t v = t; v < vecs; v += G) {
      const BlockGradVec<DT, AL> m(a, row, v, rstd, offset);
      const uint64_t at = row * a.cols;
      const bool first = row == p;
      float r[8], dn[8], sg[8] = {}, su[8] = {};
      if (!first) {
        load8<ZS_FP32, false>(own, (uint64_t)v * 8, a.cols, sg);
        if (a.x) load8<ZS_FP32, false>(own + a.cols, (uint64_t)v * 8, a.cols, su);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = m.h[j] * rstd, dh = fmaf(-n, c, m.e[j]), o = m.kept[j] ? scale * dh : 0.0f;
        r[j] = dh * a.residual_scale;
        dn[j] = o * m.q[j];
        if (a.post_gain) dn[j] = post_rstd * fmaf(-m.x[j], s1, dn[j]);
        sg[j] = fmaf(m.d[j], n, sg[j]);
        su[j] = fmaf(o, m.kept[j] ? m.x[j] * post_rstd : 0.0f, su[j]);
      }
      store8f<false, false>(own, (uint64_t)v * 8, a.cols, sg);
      if (a.x) store8f<false, false>(own + a.cols, (uint64_t)v * 8, a.cols, su);
      store8<DT, AL, true>(a.dresidual + at, (uint64_t)v * 8, a.cols, r);
      store8<DT, AL, true>(a.dx + at, (uint64_t)v * 8, a.cols, dn);
    }
  }
}

/* The shares joined in order, as norm_gain_kernel does: blockIdx.y 0 for dg2,
 * 1 for u, which the other vector makes dg1 and dgate. */
constexpr int kBlockGainCols = 32, kBlockGainRuns = 32;

struct BlockGainArgs {
  const float *part;
  const void *post_gain, *gate;
  float *dgain, *dpost_gain, *dgate;
  uint32_t parts, cols;
};

template <int DT>
__global__ __launch_bounds__(kBlockGainCols * kBlockGainRuns) void block_gain_kernel(
    BlockGainArgs a) {
  __shared__ float sums[kBlockGainRuns][kBlockGainCols + 1];
  const uint32_t lane = threadIdx.x % kBlockGainCols, run = threadIdx.x / kBlockGainCols;
  const uint32_t c = blockIdx.x * kBlockGainCols + lane;
  float s = 0.0f;
  if (c < a.cols) {
    const float *q = a.part + (uint64_t)blockIdx.y * a.cols + c;
    for (uint32_t p = run; p < a.parts; p += 8 * kBlockGainRuns) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t at = p + k * kBlockGainRuns;
        v[k] = at < a.parts ? q[(uint64_t)at * 2 * a.cols] : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[k];
    }
  }
  sums[run][lane] = s;
  __syncthreads();
  if (run != 0 || c >= a.cols) return;
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < kBlockGainRuns; ++w) s += sums[w][lane];
  if (blockIdx.y == 0) {
    a.dgain[c] = s;
    return;
  }
  const auto at = [&](const void *v) {
    return v ? up_lo<DT>(static_cast<const uint16_t *>(v)[c]) : 1.0f;
  };
  if (a.dpost_gain) a.dpost_gain[c] = s * at(a.gate);
  if (a.dgate) a.dgate[c] = s * at(a.post_gain);
}

}  // namespace zs
#endif  // ZS_BLOCK_KERNELS_H
