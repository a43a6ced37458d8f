/*
 * zs_block.hip -- libzeroshard's operators of a block's end (gfx950): dropout,
 * and the norms before and after the residual's addition fused with gate,
 * dropout and scales. Host side: argument validation and launches. The device
 * code is in zs_dropout_kernels.h and zs_block_kernels.h, over zs_philox.h.
 */
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>
#include <string.h>

#include "zeroshard.h"

#include "zs_block_kernels.h"
#include "zs_dropout_kernels.h"
#include "zs_norm_launch.h"
#include "zs_ops_common.h"

namespace {

using namespace zs;
using namespace zs_ops;

/* p as a number of 65536ths, and what a rule's pointer must be. */
int drop_args(const zs_dropout_rule *rule, DropArgs &d, const char *bad_p, const char *bad_offset) {
  d = {};
  d.factor = 1.0f;
  d.factor64 = 1.0;
  if (!rule) return ZS_OK;
  if (!(rule->p >= 0.0f && rule->p <= 1.0f)) return fail(ZS_ERR_INVALID_ARG, bad_p);
  if (!aligned(rule->dev_offset, 8)) return fail(ZS_ERR_UNSUPPORTED, bad_offset);
  d.dev_offset = rule->dev_offset;
  d.offset = rule->offset;
  d.key[0] = (uint32_t)rule->seed;
  d.key[1] = (uint32_t)(rule->seed >> 32);
  d.threshold = (uint32_t)floor((double)rule->p * 65536.0 + 0.5);
  d.factor64 = d.threshold < 65536 ? 65536.0 / (65536 - d.threshold) : 0.0;
  d.factor = (float)d.factor64;
  return ZS_OK;
}

/* Whether a float has at most 13 significant bits, and is no extreme one whose
 * products with 16-bit numbers could leave fp32's normal range unseen. */
bool short_float(float x) {
  uint32_t b;
  memcpy(&b, &x, sizeof b);
  return (b & 0x7ff) == 0 && (x == 0.0f || (fabsf(x) >= 0x1p-10f && fabsf(x) <= 0x1p10f));
}

/* The forward pass's threads per row and vectors of eight per thread: up to
 * 2048 elements half as many threads as the norm's, for there are two sums a
 * row to join (32768 x 2048: 90 us, with 256 threads 102; 4096 x 12288: 89 with
 * 512 of four vectors, 123 with 1024 of two; 16384 x 4096 91 with 256, 94 with
 * 128). Above 32768, eight vectors a thread, 204 to 420 bytes of them are in
 * scratch memory. */
template <class F>
void with_block_shape(uint64_t padded, F f) {
  if (padded <= 512) f(Tag<64>{}, Tag<1>{});
  else if (padded <= 1024) f(Tag<64>{}, Tag<2>{});
  else if (padded <= 2048) f(Tag<128>{}, Tag<2>{});
  else if (padded <= 4096) f(Tag<256>{}, Tag<2>{});
  else if (padded <= 8192) f(Tag<256>{}, Tag<4>{});
  else if (padded <= 16384) f(Tag<512>{}, Tag<4>{});
  else if (padded <= 32768) f(Tag<1024>{}, Tag<4>{});
  else f(Tag<1024>{}, Tag<8>{});
}

/* The gradient's: one vector per thread as far as a block goes, for a thread
 * holds four tensors' and the sums (16384 x 4096: 151 us with 512 threads of one,
 * 203 with 256 of two). Beyond 16384 elements it reads a row twice. 1024 threads
 * of two vectors keep 120 to 156 bytes each in scratch memory; threads of rows
 * that are not whole vectors 20 to 132 with one vector and up to 308 with two. */
constexpr uint64_t kHeldGrad = 16384;

template <class F>
void with_block_grad_shape(uint64_t padded, F f) {
  if (padded <= 512) f(Tag<64>{}, Tag<1>{});
  else if (padded <= 1024) f(Tag<128>{}, Tag<1>{});
  else if (padded <= 2048) f(Tag<256>{}, Tag<1>{});
  else if (padded <= 4096) f(Tag<512>{}, Tag<1>{});
  else if (padded <= 8192) f(Tag<1024>{}, Tag<1>{});
  else f(Tag<1024>{}, Tag<2>{});
}

/* Groups that share the rows: as many as are resident at a time, but some four
 * rows each, for their sums cost as much again as a row or two. */
uint32_t block_parts(uint64_t rows, uint64_t cols) {
  const uint64_t fit = cols <= 2048 ? 1024 : cols <= 4096 ? 512 : 256;
  const uint64_t want = rows / 4 < 256 ? 256 : rows / 4 > fit ? fit : rows / 4;
  return (uint32_t)(rows < want ? rows : want);
}

constexpr uint64_t kMaxDropRows = 1ull << 32;   /* a counter's word */

}  // namespace

extern "C" {

int zs_dropout(const void *x, const void *residual, int dtype, uint64_t rows, uint64_t cols,
               const zs_dropout_rule *rule, void *out, void *stream) {
  if (!valid_any(dtype)) return fail(ZS_ERR_INVALID_ARG, "zs_dropout: bad dtype%s");
  if (!rule) return fail(ZS_ERR_INVALID_ARG, "zs_dropout: null rule%s");
  DropoutArgs a{};
  if (int rc = drop_args(rule, a.drop, "zs_dropout: p must lie in [0, 1]%s",
                         "zs_dropout: dev_offset not aligned%s"))
    return rc;
  if (matrix_too_big(rows, cols))
    return fail(ZS_ERR_UNSUPPORTED, "zs_dropout: more than 2^48 elements%s");
  if (rows == 0 || cols == 0) return ZS_OK;
  if (!x || !out) return fail(ZS_ERR_INVALID_ARG, "zs_dropout: null x or out%s");
  const uint64_t vpr = (cols + 7) / 8;
  if (rows >= kMaxDropRows || vpr >> 32 || !fits((rows * vpr + kBlock - 1) / kBlock, kBlock))
    return fail(ZS_ERR_UNSUPPORTED, "zs_dropout: too large for one launch%s");
  const uint64_t esz = esize(dtype), bytes = rows * cols * esz;
  if (!aligned(x, esz) || !aligned(residual, esz) || !aligned(out, esz))
    return fail(ZS_ERR_UNSUPPORTED, "zs_dropout: an operand is not aligned%s");
  /* out may take the place of x or of the residual */
  if ((overlaps(out, bytes, x, bytes) && out != x) ||
      (overlaps(out, bytes, residual, bytes) && out != residual) ||
      overlaps(out, bytes, rule->dev_offset, 8))
    return fail(ZS_ERR_ALIAS, "zs_dropout: the output overlaps an input%s");
  a.x = x;
  a.res = residual;
  a.out = out;
  a.rows = rows;
  a.cols = cols;
  a.vpr = (uint32_t)vpr;
  a.vecs = (uint32_t)(rows * vpr);
  const bool al = cols % 8 == 0 && aligned(x, 16) && aligned(residual, 16) && aligned(out, 16);
  hipStream_t s = static_cast<hipStream_t>(stream);
  with_any(dtype, [&](auto dt) {
    with_bool(al, [&](auto v) {
      hipLaunchKernelGGL((dropout_kernel<decltype(dt)::value, decltype(v)::value>),
                         dim3((a.vecs + kBlock - 1) / kBlock), dim3(kBlock), 0, s, a);
    });
  });
  return launch_result();
}

int zs_block_norm_forward(const void *x, const void *residual, const void *post_gain,
                          const void *gate, const void *gain, int dtype, uint64_t rows,
                          uint64_t cols, float eps, float residual_scale, float branch_scale,
                          const zs_dropout_rule *dropout, void *h, float *post_rstd, float *rstd,
                          uint8_t *codes, uint8_t *scales, void *y, void *stream) {
  if (!valid16(dtype)) return fail(ZS_ERR_INVALID_ARG, "zs_block_norm_forward: bad dtype%s");
  if (!(eps >= 0.0f) || !isfinite(eps))
    return fail(ZS_ERR_INVALID_ARG, "zs_block_norm_forward: eps must be finite and >= 0%s");
  if (!isfinite(residual_scale) || !isfinite(branch_scale))
    return fail(ZS_ERR_INVALID_ARG, "zs_block_norm_forward: scales must be finite%s");
  if (!codes != !scales)
    return fail(ZS_ERR_INVALID_ARG, "zs_block_norm_forward: codes and scales go together%s");
  if (!codes && !y)
    return fail(ZS_ERR_INVALID_ARG, "zs_block_norm_forward: no output asked for%s");
  if (post_rstd && !post_gain)
    return fail(ZS_ERR_INVALID_ARG, "zs_block_norm_forward: post_rstd needs post_gain%s");
  BlockArgs a{};
  if (int rc = drop_args(dropout, a.drop, "zs_block_norm_forward: p must lie in [0, 1]%s",
                         "zs_block_norm_forward: dev_offset not aligned%s"))
    return rc;
  if (matrix_too_big(rows, cols))
    return fail(ZS_ERR_UNSUPPORTED, "zs_block_norm_forward: more than 2^48 elements%s");
  if (cols > kMaxNormCols)
    return fail(ZS_ERR_UNSUPPORTED, "zs_block_norm_forward: rows of more than 65536 elements%s");
  if (rows == 0 || cols == 0) return ZS_OK;
  if (!x || !residual || !gain || !h)
    return fail(ZS_ERR_INVALID_ARG, "zs_block_norm_forward: null x, residual, gain or h%s");
  if ((codes && (!aligned(codes, 16) || !aligned(scales, 4))) || !aligned(x, 2) ||
      !aligned(residual, 2) || !aligned(post_gain, 2) || !aligned(gate, 2) || !aligned(gain, 2) ||
      !aligned(h, 2) || !aligned(y, 2) || !aligned(post_rstd, 4) || !aligned(rstd, 4))
    return fail(ZS_ERR_UNSUPPORTED, "zs_block_norm_forward: an operand is not aligned%s");
  const uint64_t padded = padded_of(cols), bytes = rows * cols * 2;
  const void *outs[] = {h, y, codes, scales, rstd, post_rstd};
  const uint64_t out_bytes[] = {bytes, bytes, rows * padded, rows * padded / ZS_MX_BLOCK,
                                rows * 4, rows * 4};
  const void *ins[] = {x, residual, post_gain, gate, gain, a.drop.dev_offset};
  const uint64_t in_bytes[] = {bytes, bytes, cols * 2, cols * 2, cols * 2, 8};
  for (int i = 0; i < 6; ++i) {
    /* h may take the place of x or of the residual */
    for (int j = 0; j < 6; ++j)
      if (overlaps(outs[i], out_bytes[i], ins[j], in_bytes[j]) &&
          !(i == 0 && j < 2 && h == ins[j]))
        return fail(ZS_ERR_ALIAS, "zs_block_norm_forward: an output overlaps an input%s");
    for (int j = i + 1; j < 6; ++j)
      if (overlaps(outs[i], out_bytes[i], outs[j], out_bytes[j]))
        return fail(ZS_ERR_ALIAS, "zs_block_norm_forward: two outputs overlap%s");
  }
  a.x = x;
  a.res = residual;
  a.post_gain = post_gain;
  a.gate = gate;
  a.gain = gain;
  a.h = static_cast<uint16_t *>(h);
  a.y = static_cast<uint16_t *>(y);
  a.post_rstd = post_rstd;
  a.rstd = rstd;
  a.codes = codes;
  a.scales = scales;
  a.rows = rows;
  a.cols = (uint32_t)cols;
  a.padded = (uint32_t)padded;
  a.eps = eps;
  a.inv_cols = 1.0 / (double)cols;
  a.residual_scale = residual_scale;
  a.branch_scale = branch_scale;
  /* 13 bits of it times 11 of the residual's are 24 */
  a.near_dropped = short_float(residual_scale) ? 0x1p-100f : 0x1p-22f;
  const bool al = cols % 8 == 0 && aligned(x, 16) && aligned(residual, 16) &&
                  aligned(post_gain, 16) && aligned(gate, 16) && aligned(gain, 16) &&
                  aligned(h, 16) && aligned(y, 16);
  hipStream_t s = static_cast<hipStream_t>(stream);
  int rc = ZS_OK;
  with16(dtype, [&](auto dt) {
    with_bool(al, [&](auto v) {
      with_block_shape(padded, [&](auto g, auto items) {
        constexpr int G = decltype(g)::value, block = G < 128 ? 256 : G, per = block / G;
        const uint64_t blocks = (rows + per - 1) / per;
        if (!fits(blocks, block)) {
          rc = fail(ZS_ERR_UNSUPPORTED, "zs_block_norm_forward: too many rows for one launch%s");
          return;
        }
        hipLaunchKernelGGL((block_kernel<decltype(dt)::value, decltype(v)::value, G,
                                         decltype(items)::value>),
                           dim3((unsigned)blocks), dim3(block), 0, s, a);
        rc = launch_result();
      });
    });
  });
  return rc;
}

uint64_t zs_block_norm_backward_workspace(uint64_t rows, uint64_t cols) {
  return cols > kMaxNormCols ? 0 : (uint64_t)block_parts(rows, cols) * cols * 8;
}

int zs_block_norm_backward(const void *dy, const void *h, const float *rstd, const void *gain,
                           const void *dres, const void *x, const float *post_rstd,
                           const void *post_gain, const void *gate, int dtype, uint64_t rows,
                           uint64_t cols, float residual_scale, float branch_scale,
                           const zs_dropout_rule *dropout, void *dx, void *dresidual,
                           float *dgain, float *dpost_gain, float *dgate, void *workspace,
                           uint64_t workspace_bytes, void *stream) {
  if (!valid16(dtype)) return fail(ZS_ERR_INVALID_ARG, "zs_block_norm_backward: bad dtype%s");
  if (!isfinite(residual_scale) || !isfinite(branch_scale))
    return fail(ZS_ERR_INVALID_ARG, "zs_block_norm_backward: scales must be finite%s");
  if (!post_gain != !dpost_gain || !gate != !dgate)
    return fail(ZS_ERR_INVALID_ARG,
                "zs_block_norm_backward: post_gain and gate go with their gradients%s");
  BlockGradArgs a{};
  if (int rc = drop_args(dropout, a.drop, "zs_block_norm_backward: p must lie in [0, 1]%s",
                         "zs_block_norm_backward: dev_offset not aligned%s"))
    return rc;
  if (matrix_too_big(rows, cols))
    return fail(ZS_ERR_UNSUPPORTED, "zs_block_norm_backward: more than 2^48 elements%s");
  if (cols > kMaxNormCols)
    return fail(ZS_ERR_UNSUPPORTED, "zs_block_norm_backward: rows of more than 65536 elements%s");
  if (rows >= kMaxDropRows)
    return fail(ZS_ERR_UNSUPPORTED, "zs_block_norm_backward: too many rows%s");
  if (cols == 0) return ZS_OK;
  if (!dgain) return fail(ZS_ERR_INVALID_ARG, "zs_block_norm_backward: null dgain%s");
  if (!aligned(dgain, 4) || !aligned(dpost_gain, 4) || !aligned(dgate, 4) ||
      !aligned(post_gain, 2) || !aligned(gate, 2))
    return fail(ZS_ERR_UNSUPPORTED, "zs_block_norm_backward: an operand is not aligned%s");
  const bool need_x = post_gain || gate;
  const uint64_t bytes = rows * cols * 2, need = zs_block_norm_backward_workspace(rows, cols);
  if (rows) {
    if (!dy || !h || !rstd || !gain || !dx || !dresidual || (need_x && !x) ||
        (post_gain && !post_rstd))
      return fail(ZS_ERR_INVALID_ARG, "zs_block_norm_backward: null pointer%s");
    if (!workspace || workspace_bytes < need)
      return fail(ZS_ERR_INVALID_ARG, "zs_block_norm_backward: workspace too small%s");
    if (!aligned(workspace, 4) || !aligned(dy, 2) || !aligned(h, 2) || !aligned(gain, 2) ||
        !aligned(dres, 2) || !aligned(x, 2) || !aligned(dx, 2) || !aligned(dresidual, 2) ||
        !aligned(rstd, 4) || !aligned(post_rstd, 4))
      return fail(ZS_ERR_UNSUPPORTED, "zs_block_norm_backward: an operand is not aligned%s");
  }
  {
    const void *outs[] = {dx, dresidual, dgain, dpost_gain, dgate, rows ? workspace : nullptr};
    const uint64_t out_bytes[] = {bytes, bytes, cols * 4, cols * 4, cols * 4, need};
    const void *ins[] = {dy, h, dres, x, rstd, post_rstd, gain, post_gain, gate,
                         a.drop.dev_offset};
    const uint64_t in_bytes[] = {bytes, bytes, bytes, need_x ? bytes : 0, rows * 4,
                                 post_gain ? rows * 4 : 0, cols * 2, cols * 2, cols * 2, 8};
    for (int i = 0; i < 6; ++i) {
      /* dx and dresidual may take the place of dy, h, dres or x */
      for (int j = 0; j < 10; ++j)
        if (overlaps(outs[i], out_bytes[i], ins[j], in_bytes[j]) &&
            !(i < 2 && j < 4 && outs[i] == ins[j]))
          return fail(ZS_ERR_ALIAS, "zs_block_norm_backward: an output overlaps an input%s");
      for (int j = i + 1; j < 6; ++j)
        if (overlaps(outs[i], out_bytes[i], outs[j], out_bytes[j]))
          return fail(ZS_ERR_ALIAS, "zs_block_norm_backward: two outputs overlap%s");
    }
  }
  const uint32_t parts = block_parts(rows, cols);
  a.dy = dy;
  a.h = h;
  a.gain = gain;
  a.dres = dres;
  a.x = need_x ? x : nullptr;
  a.post_gain = post_gain;
  a.gate = gate;
  a.rstd = rstd;
  a.post_rstd = post_gain ? post_rstd : nullptr;
  a.dx = static_cast<uint16_t *>(dx);
  a.dresidual = static_cast<uint16_t *>(dresidual);
  a.part = static_cast<float *>(workspace);
  a.rows = rows;
  a.cols = (uint32_t)cols;
  a.parts = parts;
  a.residual_scale = residual_scale;
  a.branch_scale = branch_scale;
  const bool al = cols % 8 == 0 && aligned(dy, 16) && aligned(h, 16) && aligned(gain, 16) &&
                  aligned(dres, 16) && aligned(a.x, 16) && aligned(post_gain, 16) &&
                  aligned(gate, 16) && aligned(dx, 16) && aligned(dresidual, 16);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows) {
    with16(dtype, [&](auto dt) {
      with_bool(al, [&](auto v) {
        if (padded_of(cols) > kHeldGrad) {
          hipLaunchKernelGGL((block_grad_wide_kernel<decltype(dt)::value, decltype(v)::value>),
                             dim3(parts), dim3(1024), 0, s, a);
          return;
        }
        with_block_grad_shape(padded_of(cols), [&](auto g, auto items) {
          constexpr int G = decltype(g)::value, block = G < 128 ? 256 : G, per = block / G;
          hipLaunchKernelGGL((block_grad_kernel<decltype(dt)::value, decltype(v)::value, G,
                                                decltype(items)::value>),
                             dim3((parts + per - 1) / per), dim3(block), 0, s, a);
        });
      });
    });
    if (int rc = launch_result()) return rc;
  }
  const BlockGainArgs b{a.part, post_gain, gate, dgain, dpost_gain, dgate, parts, (uint32_t)cols};
  const dim3 grid((unsigned)((cols + kBlockGainCols - 1) / kBlockGainCols), need_x ? 2 : 1);
  with16(dtype, [&](auto dt) {
    hipLaunchKernelGGL((block_gain_kernel<decltype(dt)::value>), grid,
                       dim3(kBlockGainCols * kBlockGainRuns), 0, s, b);
  });
  return launch_result();
}

}  /* extern "C" */
