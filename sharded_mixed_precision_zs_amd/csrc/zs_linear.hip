/*
 * zs_linear.hip -- libzeroshard's product of microscaled operands with bias,
 * activation and residual in its epilogue, and the gradient of that epilogue
 * (gfx950). Host side: argument validation and launches. The device code is in
 * zs_matmul_kernels.h over zs_epilogue.h, and in zs_activation_kernels.h.
 */
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "zeroshard.h"

#include "zs_activation_kernels.h"
#include "zs_matmul_launch.h"
#include "zs_ops_common.h"

namespace {

using namespace zs;
using namespace zs_ops;

bool valid_act(int a) {
  return a == ZS_ACT_NONE || a == ZS_ACT_RELU || a == ZS_ACT_GELU || a == ZS_ACT_SILU;
}

template <class F>
void with_act(int act, F f) {
  if (act == ZS_ACT_RELU) f(Tag<ZS_ACT_RELU>{});
  else if (act == ZS_ACT_GELU) f(Tag<ZS_ACT_GELU>{});
  else if (act == ZS_ACT_SILU) f(Tag<ZS_ACT_SILU>{});
  else f(Tag<ZS_ACT_NONE>{});
}

/* A block's vectors of a row, 512 bytes of it or all, and its rows at a time
 * (32768 x 1600 with gelu 62 us, with 1024 bytes 67; rows that are no whole
 * vectors straddle lines at both ends of that: 16384 x 4095 97 us with 1024
 * bytes, 107 with 512). Parts of the rows: what a block takes at once, but 1024
 * at most. */
struct ActShape {
  uint32_t vecs, across, down, stripes, parts;
  uint64_t each;
};

ActShape act_shape(uint64_t rows, uint64_t cols) {
  ActShape s;
  s.vecs = (uint32_t)((cols + 7) / 8);
  const uint32_t most_across = cols % 8 ? 64 : 32;
  s.across = s.vecs < most_across ? s.vecs : most_across;
  s.down = kActThreads / s.across;
  s.stripes = (s.vecs + s.across - 1) / s.across;
  const uint64_t once = (uint64_t)kActRows * s.down, most = (rows + once - 1) / once;
  s.each = (most + 1023) / 1024 * once;
  s.parts = (uint32_t)((rows + s.each - 1) / s.each);
  return s;
}

constexpr uint64_t kMaxActCols = 1ull << 31;   /* columns are counted in 32 bits */

}  // namespace

extern "C" {

int zs_mx_linear(const uint8_t *a_codes, const uint8_t *a_scales, int a_format,
                 const uint8_t *b_codes, const uint8_t *b_scales, uint64_t m, uint64_t n,
                 uint64_t k, const void *bias, int activation, const void *residual, uint64_t ldr,
                 void *pre, void *c, int c_dtype, uint64_t ldc, void *workspace,
                 uint64_t workspace_bytes, void *stream) {
  if (!valid_format(a_format)) return fail(ZS_ERR_INVALID_ARG, "zs_mx_linear: bad format%s");
  if (!valid16(c_dtype)) return fail(ZS_ERR_INVALID_ARG, "zs_mx_linear: bad dtype%s");
  if (!valid_act(activation)) return fail(ZS_ERR_INVALID_ARG, "zs_mx_linear: bad activation%s");
  if (ldc < n || (residual && ldr < n))
    return fail(ZS_ERR_INVALID_ARG, "zs_mx_linear: ldc or ldr below n%s");
  constexpr uint64_t kMaxDim = 1ull << 30;
  if (m > kMaxDim || n > kMaxDim || k > kMaxMatmulK || matrix_too_big(m, ldc) ||
      (residual && matrix_too_big(m, ldr)))
    return fail(ZS_ERR_UNSUPPORTED, "zs_mx_linear: m or n above 2^30, or k above 2^22%s");
  if (m == 0 || n == 0) return ZS_OK;
  if (!c || (k && (!a_codes || !a_scales || !b_codes || !b_scales)))
    return fail(ZS_ERR_INVALID_ARG, "zs_mx_linear: null pointer%s");
  if (!aligned(a_codes, 16) || !aligned(b_codes, 16) || !aligned(a_scales, 4) ||
      !aligned(b_scales, 4) || !aligned(bias, 2) || !aligned(residual, 2) || !aligned(pre, 2) ||
      !aligned(c, 2) || !aligned(workspace, 16))
    return fail(ZS_ERR_UNSUPPORTED, "zs_mx_linear: an operand is not aligned%s");
  const uint64_t padded = padded_of(k);
  const void *outs[] = {c, pre, workspace};
  const uint64_t out_bytes[] = {extent(m, n, ldc, 2), m * n * 2, workspace_bytes};
  const void *ins[] = {residual, a_codes, a_scales, b_codes, b_scales, bias};
  const uint64_t in_bytes[] = {extent(m, n, ldr, 2), m * code_bytes(a_format, padded),
                               m * padded / ZS_MX_BLOCK, n * padded / 2, n * padded / ZS_MX_BLOCK,
                               n * 2};
  for (int i = 0; i < 3; ++i) {
    /* c may take the residual's place */
    for (int j = 0; j < 6; ++j)
      if (overlaps(outs[i], out_bytes[i], ins[j], in_bytes[j]) &&
          !(i == 0 && j == 0 && c == residual && ldc == ldr))
        return fail(ZS_ERR_ALIAS, "zs_mx_linear: an output overlaps an input%s");
    for (int j = i + 1; j < 3; ++j)
      if (overlaps(outs[i], out_bytes[i], outs[j], out_bytes[j]))
        return fail(ZS_ERR_ALIAS, "zs_mx_linear: two outputs overlap%s");
  }
  const MatmulArgs a{a_codes, a_scales, b_codes, b_scales, c, ldc,
                     (uint32_t)m, (uint32_t)n, (uint32_t)padded, nullptr, 0};
  Epilogue e{};
  e.bias = bias;
  e.res = residual;
  e.pre = static_cast<uint16_t *>(pre);
  e.ldr = ldr;
  e.act = activation;
  hipStream_t s = static_cast<hipStream_t>(stream);
  int rc = ZS_OK;
  with_format(a_format, [&](auto f) {
    with16(c_dtype, [&](auto dt) {
      rc = launch_matmul<decltype(f)::value, decltype(dt)::value>(
          a, e, static_cast<float *>(workspace), workspace ? workspace_bytes : 0, s);
    });
  });
  return rc;
}

uint64_t zs_activation_backward_workspace(uint64_t rows, uint64_t cols) {
  return !rows || !cols || cols >= kMaxActCols ? 0 : (uint64_t)act_shape(rows, cols).parts * cols * 4;
}

int zs_activation_backward(const void *dc, const void *pre, int activation, int dtype,
                           uint64_t rows, uint64_t cols, void *dpre, float *dbias,
                           void *workspace, uint64_t workspace_bytes, void *stream) {
  if (!valid16(dtype)) return fail(ZS_ERR_INVALID_ARG, "zs_activation_backward: bad dtype%s");
  if (!valid_act(activation))
    return fail(ZS_ERR_INVALID_ARG, "zs_activation_backward: bad activation%s");
  if (!dpre && !dbias)
    return fail(ZS_ERR_INVALID_ARG, "zs_activation_backward: no output asked for%s");
  if (matrix_too_big(rows, cols) || cols >= kMaxActCols)
    return fail(ZS_ERR_UNSUPPORTED,
                "zs_activation_backward: more than 2^48 elements, or 2^31 columns%s");
  if (cols == 0 || (rows == 0 && !dbias)) return ZS_OK;
  const bool need_pre = activation != ZS_ACT_NONE;
  const uint64_t bytes = rows * cols * 2, need = zs_activation_backward_workspace(rows, cols);
  if (rows && (!dc || (need_pre && !pre)))
    return fail(ZS_ERR_INVALID_ARG, "zs_activation_backward: null pointer%s");
  if (rows && dbias && (!workspace || workspace_bytes < need))
    return fail(ZS_ERR_INVALID_ARG, "zs_activation_backward: workspace too small%s");
  if (!aligned(dc, 2) || !aligned(pre, 2) || !aligned(dpre, 2) || !aligned(dbias, 4) ||
      !aligned(workspace, 4))
    return fail(ZS_ERR_UNSUPPORTED, "zs_activation_backward: an operand is not aligned%s");
  const void *outs[] = {dpre, dbias, workspace};
  const uint64_t out_bytes[] = {bytes, cols * 4, dbias ? need : 0};
  const void *ins[] = {dc, pre};
  const uint64_t in_bytes[] = {bytes, need_pre ? bytes : 0};
  for (int i = 0; i < 3; ++i) {
    /* dpre may take the place of dc or pre */
    for (int j = 0; j < 2; ++j)
      if (overlaps(outs[i], out_bytes[i], ins[j], in_bytes[j]) && !(i == 0 && dpre == ins[j]))
        return fail(ZS_ERR_ALIAS, "zs_activation_backward: an output overlaps an input%s");
    for (int j = i + 1; j < 3; ++j)
      if (overlaps(outs[i], out_bytes[i], outs[j], out_bytes[j]))
        return fail(ZS_ERR_ALIAS, "zs_activation_backward: two outputs overlap%s");
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint32_t parts = 0;
  if (rows) {
    const ActShape sh = act_shape(rows, cols);
    parts = sh.parts;
    const ActGradArgs a{dc, need_pre ? pre : nullptr, static_cast<uint16_t *>(dpre),
                        dbias ? static_cast<float *>(workspace) : nullptr, rows, sh.each,
                        (uint32_t)cols, sh.vecs, sh.across, sh.down};
    const bool al = cols % 8 == 0 && aligned(dc, 16) && aligned(a.pre, 16) && aligned(dpre, 16);
    if (!fits(sh.stripes, kActThreads))
      return fail(ZS_ERR_UNSUPPORTED, "zs_activation_backward: too many columns for one launch%s");
    const dim3 grid(sh.stripes, parts);
    with16(dtype, [&](auto dt) {
      with_bool(al, [&](auto v) {
        with_act(activation, [&](auto act) {
          hipLaunchKernelGGL((act_grad_kernel<decltype(dt)::value, decltype(v)::value,
                                              decltype(act)::value>),
                             grid, dim3(kActThreads), 0, s, a);
        });
      });
    });
    if (int rc = launch_result()) return rc;
  }
  if (!dbias) return ZS_OK;
  hipLaunchKernelGGL(bias_grad_kernel, dim3((unsigned)((cols + kBiasCols - 1) / kBiasCols)),
                     dim3(kBiasCols * kBiasRuns), 0, s, static_cast<const float *>(workspace),
                     parts, (uint32_t)cols, dbias);
  return launch_result();
}

}  /* extern "C" */
