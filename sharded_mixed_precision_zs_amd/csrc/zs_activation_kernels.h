/*
 * zs_activation_kernels.h -- the gradient of a product's epilogue (gfx950):
 * dpre = dc act'(pre), and dpre's sum over the rows. Bound by HBM: 8192 x 16384
 * bf16 with gelu 143 us, 5.6 TB/s of dc, pre and dpre.
 */
#ifndef ZS_ACTIVATION_KERNELS_H
#define ZS_ACTIVATION_KERNELS_H

#include "zs_epilogue.h"
#include "zs_norm_rows.h"

namespace zs {

constexpr int kActThreads = 512, kActRows = 4;

struct ActGradArgs {
  const void *dc, *pre;   /* pre optional: no activation */
  uint16_t *dpre;         /* optional */
  float *part;            /* [parts][cols], optional */
  uint64_t rows, each;    /* each: rows of a part */
  uint32_t cols, vecs;
  uint32_t across, down;  /* vectors of a row, and rows at a time, to a block */
};

/* A block takes `across` vectors of eight columns by `down` rows by kActRows at
 * a time, all of a thread's loads under way at once, and mostly no more than
 * that: short-lived blocks that sweep the rows side by side (the same with
 * blocks that walk the rows, the next one's loads under way: 158 us). Two rows
 * are 138 us, but twice the shares: sums alone 59 us, with four 49. A thread
 * keeps its columns' sums, unrounded, in registers, a block joins its threads'
 * in LDS, and the blocks' shares are joined in order. */
template <int DT, bool AL, int ACT>
__global__ __launch_bounds__(kActThreads) void act_grad_kernel(ActGradArgs a) {
  __shared__ float sums[kActThreads * 9];   /* eight of a thread, and one of room */
  const uint32_t t = threadIdx.x, across = t % a.across, down = t / a.across;
  const uint32_t first = blockIdx.x * a.across, v = first + across, col = v * 8;
  const uint64_t row0 = blockIdx.y * a.each;
  const uint64_t end = row0 + a.each < a.rows ? row0 + a.each : a.rows;
  const uint16_t *dc = static_cast<const uint16_t *>(a.dc);
  const uint16_t *pre = static_cast<const uint16_t *>(a.pre);
  float sum[8] = {};
  if (down < a.down && v < a.vecs) {
    for (uint64_t row = row0 + down; row < end; row += kActRows * a.down) {
      Raw16<8> d[kActRows], s[kActRows];
#pragma unroll
      for (int k = 0; k < kActRows; ++k) {
        const uint64_t at = row + k * a.down;
        d[k] = s[k] = {};
        if (at < end) {
          d[k] = load8_ahead<AL>(dc + at * a.cols, col, a.cols);
          if constexpr (ACT != ZS_ACT_NONE) s[k] = load8_ahead<AL>(pre + at * a.cols, col, a.cols);
        }
      }
#pragma unroll
      for (int k = 0; k < kActRows; ++k) {
        const uint64_t at = row + k * a.down;
        if (at >= end) break;
        float x[8], y[8];
        settle8<AL>(d[k], col, a.cols);
        upcast<8, DT>(d[k], x);
        if constexpr (ACT != ZS_ACT_NONE) {
          settle8<AL>(s[k], col, a.cols);
          upcast<8, DT>(s[k], y);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] *= slope_of<ACT>(y[j]);
        }
        if (a.dpre) store8<DT, AL>(a.dpre + at * a.cols, col, a.cols, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += x[j];
      }
    }
  }
  if (!a.part) return;   /* the same for a whole launch */
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[t * 9 + j] = sum[j];
  for (uint32_t n = a.down; n > 1;) {   /* the upper half of the rows to the lower */
    const uint32_t half = (n + 1) / 2;
    __syncthreads();
    if (down + half < n) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        sums[t * 9 + j] = sum[j] += sums[(t + half * a.across) * 9 + j];
    }
    n = half;
  }
  __syncthreads();
  for (uint32_t c = t; c < a.across * 8 && first * 8 + c < a.cols; c += kActThreads)
    a.part[(uint64_t)blockIdx.y * a.cols + first * 8 + c] = sums[c / 8 * 9 + c % 8];
}

/* The shares of dbias, added in order: 32 columns a block, 32 runs that take
 * every 32nd share each, eight at a time, so that their latencies overlap. */
constexpr int kBiasCols = 32, kBiasRuns = 32;

__global__ __launch_bounds__(kBiasCols * kBiasRuns) void bias_grad_kernel(const float *part,
                                                                          uint32_t parts,
                                                                          uint32_t cols,
                                                                          float *dbias) {
  __shared__ float sums[kBiasRuns][kBiasCols + 1];
  const uint32_t lane = threadIdx.x % kBiasCols, run = threadIdx.x / kBiasCols;
  const uint32_t c = blockIdx.x * kBiasCols + lane;
  float s = 0.0f;
  if (c < cols) {
    for (uint32_t p = run; p < parts; p += 8 * kBiasRuns) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t at = p + k * kBiasRuns;
        v[k] = at < parts ? part[(uint64_t)at * cols + c] : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[k];
    }
  }
  sums[run][lane] = s;
  __syncthreads();
  if (run != 0 || c >= cols) return;
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < kBiasRuns; ++w) s += sums[w][lane];
  dbias[c] = s;
}

}  // namespace zs
#endif  // ZS_ACTIVATION_KERNELS_H
