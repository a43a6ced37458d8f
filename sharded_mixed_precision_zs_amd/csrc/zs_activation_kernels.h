/*
 * zs_activation_kernels.h -- the gradient of a product's epilogue (gfx950):
 * dpre = dc act'(pre), and dpre's sum over the rows. Bound by HBM: 8192 x 16384
 * bf16 with gelu 135 us, 6.0 TB/s of dc, pre and dpre.
 */
#ifndef ZS_ACTIVATION_KERNELS_H
#define ZS_ACTIVATION_KERNELS_H

#include "zs_epilogue.h"
#include "zs_norm_rows.h"

namespace zs {

struct ActGradArgs {
  const void *dc, *pre;   /* pre optional: no activation */
  uint16_t *dpre;         /* optional */
  float *part;            /* [parts][cols], optional */
  uint64_t rows;
  uint32_t cols, vecs, parts;   /* parts: blocks that share the rows */
  uint32_t across, down;        /* vectors of a row, and rows at a time, to a block */
};

/* A block takes `across` vectors of eight columns by `down` rows at a time and
 * walks a share of the rows, the next row's vectors on their way; a thread
 * keeps its columns' sums, unrounded, in registers, a block joins its threads'
 * in LDS, and the blocks' shares are joined in order. */
template <int DT, bool AL, int ACT>
__global__ __launch_bounds__(kBlock) void act_grad_kernel(ActGradArgs a) {
  __shared__ float sums[8][kBlock];
  const uint32_t t = threadIdx.x, across = t % a.across, down = t / a.across;
  const uint32_t v = blockIdx.x * a.across + across, col = v * 8;
  const uint64_t groups = (uint64_t)a.parts * a.down;
  const uint16_t *dc = static_cast<const uint16_t *>(a.dc);
  const uint16_t *pre = static_cast<const uint16_t *>(a.pre);
  float sum[8] = {};
  if (down < a.down && v < a.vecs) {
    uint64_t row = (uint64_t)blockIdx.y * a.down + down;
    Raw16<8> d = {}, s = {};
    if (row < a.rows) {
      d = load8_ahead<AL>(dc + row * a.cols, col, a.cols);
      if constexpr (ACT != ZS_ACT_NONE) s = load8_ahead<AL>(pre + row * a.cols, col, a.cols);
    }
    for (; row < a.rows; row += groups) {
      const uint64_t next = row + groups;
      Raw16<8> d1 = {}, s1 = {};
      if (next < a.rows) {
        d1 = load8_ahead<AL>(dc + next * a.cols, col, a.cols);
        if constexpr (ACT != ZS_ACT_NONE) s1 = load8_ahead<AL>(pre + next * a.cols, col, a.cols);
      }
      float x[8], y[8];
      settle8<AL>(d, col, a.cols);
      upcast<8, DT>(d, x);
      if constexpr (ACT != ZS_ACT_NONE) {
        settle8<AL>(s, col, a.cols);
        upcast<8, DT>(s, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= slope_of<ACT>(y[j]);
      }
      if (a.dpre) store8<DT, AL>(a.dpre + row * a.cols, col, a.cols, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += x[j];
      d = d1;
      s = s1;
    }
  }
  if (!a.part) return;   /* the same for a whole launch */
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[j][t] = sum[j];
  __syncthreads();
  if (down != 0 || v >= a.vecs) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    for (uint32_t r = 1; r < a.down; ++r) sum[j] += sums[j][r * a.across + across];
    if (col + j < a.cols) a.part[(uint64_t)blockIdx.y * a.cols + col + j] = sum[j];
  }
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
