/*
 * zs_ops.hip -- libzeroshard's operators for the output end of a model
 * trained in low precision (gfx950): the norm, the microscaled formats'
 * quantisation and product, and the distillation loss. Host side: argument
 * validation, choice of the kernel variant, launches. The device code is in
 * zs_norm_kernels.h, zs_quantize_kernels.h, zs_matmul_kernels.h and
 * zs_distill_kernels.h, over zs_mx.h.
 */
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "zeroshard.h"

#include "zs_distill_kernels.h"
#include "zs_matmul_launch.h"
#include "zs_norm_kernels.h"
#include "zs_norm_launch.h"
#include "zs_ops_common.h"
#include "zs_quantize_kernels.h"

namespace {

using namespace zs;
using namespace zs_ops;

}  // namespace

extern "C" {

int zs_rmsnorm_forward(const void *x, const void *residual, const void *gain, int dtype,
                       uint64_t rows, uint64_t cols, float eps, void *h, float *rstd,
                       uint8_t *codes, uint8_t *scales, void *y, void *stream) {
  if (!valid16(dtype)) return fail(ZS_ERR_INVALID_ARG, "zs_rmsnorm_forward: bad dtype%s");
  if (!(eps >= 0.0f) || !isfinite(eps))
    return fail(ZS_ERR_INVALID_ARG, "zs_rmsnorm_forward: eps must be finite and >= 0%s");
  if (!codes != !scales)
    return fail(ZS_ERR_INVALID_ARG, "zs_rmsnorm_forward: codes and scales go together%s");
  if (!codes && !y) return fail(ZS_ERR_INVALID_ARG, "zs_rmsnorm_forward: no output asked for%s");
  if (!h && residual)
    return fail(ZS_ERR_INVALID_ARG, "zs_rmsnorm_forward: a residual needs h%s");
  if (matrix_too_big(rows, cols))
    return fail(ZS_ERR_UNSUPPORTED, "zs_rmsnorm_forward: more than 2^48 elements%s");
  if (cols > kMaxNormCols)
    return fail(ZS_ERR_UNSUPPORTED, "zs_rmsnorm_forward: rows of more than 65536 elements%s");
  if (rows == 0 || cols == 0) return ZS_OK;
  if (!x || !gain) return fail(ZS_ERR_INVALID_ARG, "zs_rmsnorm_forward: null x or gain%s");
  if ((codes && (!aligned(codes, 16) || !aligned(scales, 4))) || !aligned(x, 2) ||
      !aligned(residual, 2) || !aligned(gain, 2) || !aligned(h, 2) || !aligned(y, 2) ||
      !aligned(rstd, 4))
    return fail(ZS_ERR_UNSUPPORTED, "zs_rmsnorm_forward: an operand is not aligned%s");
  const uint64_t padded = padded_of(cols), bytes = rows * cols * 2;
  const void *outs[] = {h, y, codes, scales, rstd};
  const uint64_t out_bytes[] = {bytes, bytes, rows * padded, rows * padded / ZS_MX_BLOCK, rows * 4};
  for (int i = 0; i < 5; ++i) {
    /* h may take the place of x or of the residual */
    if ((overlaps(outs[i], out_bytes[i], x, bytes) && !(i == 0 && h == x)) ||
        (overlaps(outs[i], out_bytes[i], residual, bytes) && !(i == 0 && h == residual)) ||
        overlaps(outs[i], out_bytes[i], gain, cols * 2))
      return fail(ZS_ERR_ALIAS, "zs_rmsnorm_forward: an output overlaps an input%s");
    for (int j = i + 1; j < 5; ++j)
      if (overlaps(outs[i], out_bytes[i], outs[j], out_bytes[j]))
        return fail(ZS_ERR_ALIAS, "zs_rmsnorm_forward: two outputs overlap%s");
  }
  NormArgs a{x, residual, gain, static_cast<uint16_t *>(h), static_cast<uint16_t *>(y), rstd,
             codes, scales, rows, (uint32_t)cols, (uint32_t)padded, eps, 1.0 / (double)cols};
  const bool al = cols % 8 == 0 && aligned(x, 16) && aligned(residual, 16) && aligned(gain, 16) &&
                  aligned(h, 16) && aligned(y, 16);
  hipStream_t s = static_cast<hipStream_t>(stream);
  int rc = ZS_OK;
  with16(dtype, [&](auto dt) {
    with_bool(al, [&](auto v) {
      with_norm_shape(padded, [&](auto g, auto items) {
        constexpr int G = decltype(g)::value, block = G < 256 ? 256 : G, per = block / G;
        const uint64_t blocks = (rows + per - 1) / per;
        if (!fits(blocks, block)) {
          rc = fail(ZS_ERR_UNSUPPORTED, "zs_rmsnorm_forward: too many rows for one launch%s");
          return;
        }
        hipLaunchKernelGGL((norm_kernel<decltype(dt)::value, decltype(v)::value, G,
                                        decltype(items)::value>),
                           dim3((unsigned)blocks), dim3(block), 0, s, a);
        rc = launch_result();
      });
    });
  });
  return rc;
}

uint64_t zs_rmsnorm_backward_workspace(uint64_t rows, uint64_t cols) {
  return cols > kMaxNormCols ? 0 : (uint64_t)norm_parts(rows) * cols * 4;
}

int zs_rmsnorm_backward(const void *dy, const void *h, const float *rstd, const void *gain,
                        const void *dres, int dtype, uint64_t rows, uint64_t cols, void *dx,
                        float *dgain, void *workspace, uint64_t workspace_bytes, void *stream) {
  if (!valid16(dtype)) return fail(ZS_ERR_INVALID_ARG, "zs_rmsnorm_backward: bad dtype%s");
  if (matrix_too_big(rows, cols))
    return fail(ZS_ERR_UNSUPPORTED, "zs_rmsnorm_backward: more than 2^48 elements%s");
  if (cols > kMaxNormCols)
    return fail(ZS_ERR_UNSUPPORTED, "zs_rmsnorm_backward: rows of more than 65536 elements%s");
  if (cols == 0) return ZS_OK;
  if (!dgain) return fail(ZS_ERR_INVALID_ARG, "zs_rmsnorm_backward: null dgain%s");
  const uint64_t bytes = rows * cols * 2, need = zs_rmsnorm_backward_workspace(rows, cols);
  if (rows) {
    if (!dy || !h || !rstd || !gain || !dx)
      return fail(ZS_ERR_INVALID_ARG, "zs_rmsnorm_backward: null pointer%s");
    if (!workspace || workspace_bytes < need)
      return fail(ZS_ERR_INVALID_ARG, "zs_rmsnorm_backward: workspace too small%s");
    if (!aligned(workspace, 4) || !aligned(dy, 2) || !aligned(h, 2) || !aligned(gain, 2) ||
        !aligned(dres, 2) || !aligned(dx, 2) || !aligned(rstd, 4) || !aligned(dgain, 4))
      return fail(ZS_ERR_UNSUPPORTED, "zs_rmsnorm_backward: an operand is not aligned%s");
    const void *outs[] = {dx, dgain, workspace};
    const uint64_t out_bytes[] = {bytes, cols * 4, need};
    const void *ins[] = {dy, h, dres, rstd, gain};
    const uint64_t in_bytes[] = {bytes, bytes, bytes, rows * 4, cols * 2};
    for (int i = 0; i < 3; ++i) {
      /* dx may take the place of dy, h or dres */
      for (int j = 0; j < 5; ++j)
        if (overlaps(outs[i], out_bytes[i], ins[j], in_bytes[j]) &&
            !(i == 0 && j < 3 && dx == ins[j]))
          return fail(ZS_ERR_ALIAS, "zs_rmsnorm_backward: an output overlaps an input%s");
      for (int j = i + 1; j < 3; ++j)
        if (overlaps(outs[i], out_bytes[i], outs[j], out_bytes[j]))
          return fail(ZS_ERR_ALIAS, "zs_rmsnorm_backward: two outputs overlap%s");
    }
  }
  const uint32_t parts = norm_parts(rows);
  NormGradArgs a{dy, h, gain, dres, rstd, static_cast<uint16_t *>(dx),
                 static_cast<float *>(workspace), rows, (uint32_t)cols, parts};
  const bool al = cols % 8 == 0 && aligned(dy, 16) && aligned(h, 16) && aligned(gain, 16) &&
                  aligned(dres, 16) && aligned(dx, 16);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows) {
    with16(dtype, [&](auto dt) {
      with_bool(al, [&](auto v) {
        with_norm_shape(padded_of(cols), [&](auto g, auto items) {
          constexpr int G = decltype(g)::value, block = G < 256 ? 256 : G, per = block / G;
          hipLaunchKernelGGL((norm_grad_kernel<decltype(dt)::value, decltype(v)::value, G,
                                               decltype(items)::value>),
                             dim3((parts + per - 1) / per), dim3(block), 0, s, a);
        });
      });
    });
    if (int rc = launch_result()) return rc;
  }
  hipLaunchKernelGGL(norm_gain_kernel, dim3((unsigned)((cols + kGainCols - 1) / kGainCols)),
                     dim3(kGainCols * kGainRuns), 0, s, a.part, parts, (uint32_t)cols, dgain);
  return launch_result();
}

int zs_mx_quantize(const void *src, int src_dtype, uint64_t rows, uint64_t cols, uint64_t ld,
                   int format, int columns, uint8_t *codes, uint8_t *scales, void *values,
                   int values_dtype, void *stream) {
  if (!valid_any(src_dtype) || (values && !valid16(values_dtype)))
    return fail(ZS_ERR_INVALID_ARG, "zs_mx_quantize: bad dtype%s");
  if (!valid_format(format)) return fail(ZS_ERR_INVALID_ARG, "zs_mx_quantize: bad format%s");
  if (ld < cols) return fail(ZS_ERR_INVALID_ARG, "zs_mx_quantize: ld below cols%s");
  if (matrix_too_big(rows, ld))
    return fail(ZS_ERR_UNSUPPORTED, "zs_mx_quantize: more than 2^48 elements%s");
  if (rows == 0 || cols == 0) return ZS_OK;
  if (!src || !codes || !scales)
    return fail(ZS_ERR_INVALID_ARG, "zs_mx_quantize: null pointer%s");
  if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(src, esize(src_dtype)) ||
      !aligned(values, 2))
    return fail(ZS_ERR_UNSUPPORTED, "zs_mx_quantize: an operand is not aligned%s");
  const uint64_t orows = columns ? cols : rows, padded = padded_of(columns ? rows : cols);
  if (matrix_too_big(orows, padded))
    return fail(ZS_ERR_UNSUPPORTED, "zs_mx_quantize: more than 2^48 elements%s");
  const uint64_t src_bytes = extent(rows, cols, ld, esize(src_dtype));
  const void *outs[] = {codes, scales, values};
  const uint64_t out_bytes[] = {orows * code_bytes(format, padded), orows * padded / ZS_MX_BLOCK,
                                rows * cols * 2};
  for (int i = 0; i < 3; ++i) {
    if (overlaps(outs[i], out_bytes[i], src, src_bytes))
      return fail(ZS_ERR_ALIAS, "zs_mx_quantize: an output overlaps the source%s");
    for (int j = i + 1; j < 3; ++j)
      if (overlaps(outs[i], out_bytes[i], outs[j], out_bytes[j]))
        return fail(ZS_ERR_ALIAS, "zs_mx_quantize: two outputs overlap%s");
  }
  QuantArgs a{src, rows, cols, ld, codes, scales, static_cast<uint16_t *>(values), padded,
              rows * (padded / 8), 0, 0};
  const bool al = cols % 8 == 0 && aligned(src, 16) && ld * esize(src_dtype) % 16 == 0 &&
                  aligned(values, 16);
  uint64_t blocks = (a.vecs + kBlock - 1) / kBlock;
  if (columns) {
    const uint64_t across = kColTileW * (src_dtype == ZS_FP32 ? kColsPerWord<ZS_FP32>
                                                              : kColsPerWord<ZS_BF16>);
    const uint64_t tiles_c = (cols + across - 1) / across, tiles_r = padded / kColTileR;
    if (tiles_r > 65535)
      return fail(ZS_ERR_UNSUPPORTED, "zs_mx_quantize: too many rows along the columns%s");
    blocks = tiles_c * tiles_r;
    a.tiles_r = (uint32_t)tiles_r;
    a.tiles_c = (uint32_t)tiles_c;
  }
  if (!fits(blocks, kBlock))
    return fail(ZS_ERR_UNSUPPORTED, "zs_mx_quantize: too large for one launch%s");
  const dim3 grid((unsigned)blocks);
  hipStream_t s = static_cast<hipStream_t>(stream);
  with_any(src_dtype, [&](auto dt) {
    with16(values ? values_dtype : ZS_BF16, [&](auto vdt) {
      with_bool(al, [&](auto v) {
        with_format(format, [&](auto f) {
          if (columns)
            hipLaunchKernelGGL((quant_cols_kernel<decltype(dt)::value, decltype(v)::value,
                                                  decltype(f)::value, decltype(vdt)::value>),
                               grid, dim3(kBlock), 0, s, a);
          else
            hipLaunchKernelGGL((quant_rows_kernel<decltype(dt)::value, decltype(v)::value,
                                                  decltype(f)::value, decltype(vdt)::value>),
                               grid, dim3(kBlock), 0, s, a);
        });
      });
    });
  });
  return launch_result();
}

uint64_t zs_mx_matmul_workspace(uint64_t m, uint64_t n, uint64_t k) {
  if (!m || !n || too_big(m) || too_big(n) || matrix_too_big(m, n) || k > kMaxMatmulK) return 0;
  const MatmulSplit sp = matmul_split(m, n, padded_of(k), ~0ull);
  return sp.splits < 2 ? 0 : sp.splits * m * n * 4;
}

int zs_mx_matmul(const uint8_t *a_codes, const uint8_t *a_scales, int a_format,
                 const uint8_t *b_codes, const uint8_t *b_scales, uint64_t m, uint64_t n,
                 uint64_t k, void *c, int c_dtype, uint64_t ldc, void *workspace,
                 uint64_t workspace_bytes, void *stream) {
  if (!valid_format(a_format)) return fail(ZS_ERR_INVALID_ARG, "zs_mx_matmul: bad format%s");
  if (!valid_any(c_dtype)) return fail(ZS_ERR_INVALID_ARG, "zs_mx_matmul: bad dtype%s");
  if (c_dtype == ZS_FP32 && a_format == ZS_MX_E4M3)
    return fail(ZS_ERR_UNSUPPORTED, "zs_mx_matmul: fp32 results need 4-bit operands%s");
  if (ldc < n) return fail(ZS_ERR_INVALID_ARG, "zs_mx_matmul: ldc below n%s");
  constexpr uint64_t kMaxDim = 1ull << 30;
  if (m > kMaxDim || n > kMaxDim || k > kMaxMatmulK || matrix_too_big(m, ldc))
    return fail(ZS_ERR_UNSUPPORTED, "zs_mx_matmul: m or n above 2^30, or k above 2^22%s");
  if (m == 0 || n == 0) return ZS_OK;
  if (!c || (k && (!a_codes || !a_scales || !b_codes || !b_scales)))
    return fail(ZS_ERR_INVALID_ARG, "zs_mx_matmul: null pointer%s");
  if (!aligned(a_codes, 16) || !aligned(b_codes, 16) || !aligned(a_scales, 4) ||
      !aligned(b_scales, 4) || !aligned(c, esize(c_dtype)))
    return fail(ZS_ERR_UNSUPPORTED, "zs_mx_matmul: an operand is not aligned%s");
  const uint64_t padded = padded_of(k), c_bytes = extent(m, n, ldc, esize(c_dtype));
  const void *ins[] = {a_codes, a_scales, b_codes, b_scales};
  const uint64_t in_bytes[] = {m * code_bytes(a_format, padded), m * padded / ZS_MX_BLOCK,
                               n * padded / 2, n * padded / ZS_MX_BLOCK};
  for (int i = 0; i < 4; ++i)
    if (overlaps(c, c_bytes, ins[i], in_bytes[i]) ||
        overlaps(workspace, workspace_bytes, ins[i], in_bytes[i]))
      return fail(ZS_ERR_ALIAS, "zs_mx_matmul: an output overlaps an input%s");
  if (overlaps(c, c_bytes, workspace, workspace_bytes))
    return fail(ZS_ERR_ALIAS, "zs_mx_matmul: the result overlaps the workspace%s");
  if (workspace && !aligned(workspace, 16))
    return fail(ZS_ERR_UNSUPPORTED, "zs_mx_matmul: workspace not aligned%s");
  const MatmulArgs a{a_codes, a_scales, b_codes, b_scales, c, ldc,
                     (uint32_t)m, (uint32_t)n, (uint32_t)padded, nullptr, 0};
  hipStream_t s = static_cast<hipStream_t>(stream);
  int rc = ZS_OK;
  with_format(a_format, [&](auto f) {
    with_any(c_dtype, [&](auto dt) {
      rc = launch_matmul<decltype(f)::value, decltype(dt)::value>(
          a, NoEpilogue{}, static_cast<float *>(workspace), workspace ? workspace_bytes : 0, s);
    });
  });
  return rc;
}

}  /* extern "C" */

namespace {

/* ------------------------------------------------------------------------
 * A row per block where its registers hold it: blocks of 64 to 512 threads
 * of at most 16 vectors of 16 bytes, so that several rows are in flight per
 * CU; rows beyond 8192 vectors take 32 per thread and a CU to themselves.
 * One launch beats the parts' two for a few rows too (13 x 50257: 10 us
 * against 15; 1 x 128000: 17 against 23). In parts otherwise, so many that
 * some 1024 blocks run, and read up to three times (8192 x 152064 bf16: 1.9 ms,
 * 2.4 of its floors; 8192 x 128000 in a row per block 1.35); gradient rows that
 * are not aligned as the logits' go there in one part (8192 x 50257: 640 us,
 * aligned 375).
 * ---------------------------------------------------------------------- */
constexpr int kDistillThreads = 256, kRowItems = 32;

struct DistillSplit {
  uint32_t parts;      /* 0: a row per block */
  uint32_t part_vecs, vecs;
};

DistillSplit distill_split(uint64_t rows, uint64_t vocab, int dtype) {
  const uint64_t vecs = vocab * esize(dtype) / 16;
  /* two vectors' worth of elements hold one, whatever the row's alignment */
  if (vecs >= 2 && vecs <= 512 * kRowItems) return {0, 0, (uint32_t)vecs};
  uint64_t parts = rows < 1024 ? 1024 / rows : 1;
  const uint64_t most = (vecs + kDistillThreads - 1) / kDistillThreads;
  if (parts > most) parts = most;
  if (parts < 1) parts = 1;
  const uint64_t each = vecs ? (vecs + parts - 1) / parts : 1;
  /* as many as have vectors: the last part starts at the row's last vector at
   * the latest (a row that is not aligned has one fewer), and has what comes
   * after them, so the parts' shares of the vocabulary leave nothing out */
  parts = vecs ? (vecs + each - 1) / each : 1;
  return {(uint32_t)parts, (uint32_t)each, (uint32_t)vecs};
}

/* Blocks that walk the rows: as many as fit at the registers the kernel is
 * held to (four waves per SIMD up to 16 vectors a thread, two beyond). */
template <int DT, bool TAIL, int NT, int ITEMS>
void launch_rows(const DistillArgs &a, hipStream_t s) {
  const uint64_t fit = (uint64_t)cu_count() * (ITEMS <= 16 ? 16 : 8) / (NT / 64);
  hipLaunchKernelGGL((distill_row_kernel<DT, TAIL, NT, ITEMS>),
                     dim3((unsigned)(a.rows < fit ? a.rows : fit)), dim3(NT), slot_bytes(a.slots),
                     s, a);
}

template <int DT, bool TAIL>
int launch_distill(const DistillArgs &a, const DistillSplit &sp, hipStream_t s) {
  if (!sp.parts) {
    if (sp.vecs <= 128) launch_rows<DT, TAIL, 64, 2>(a, s);
    else if (sp.vecs <= 512) launch_rows<DT, TAIL, 64, 8>(a, s);
    else if (sp.vecs <= 1024) launch_rows<DT, TAIL, 64, 16>(a, s);
    else if (sp.vecs <= 2048) launch_rows<DT, TAIL, 128, 16>(a, s);
    else if (sp.vecs <= 4096) launch_rows<DT, TAIL, 256, 16>(a, s);
    else if (sp.vecs <= 8192) launch_rows<DT, TAIL, 512, 16>(a, s);
    else launch_rows<DT, TAIL, 512, kRowItems>(a, s);
    return launch_result();
  }
  constexpr int NT = kDistillThreads;
  const uint32_t blocks = a.grad ? sp.parts : 1;
  hipLaunchKernelGGL((distill_stats_kernel<DT, TAIL, NT>), dim3((unsigned)(a.rows * sp.parts)),
                     dim3(NT), slot_bytes(a.slots), s, a);
  if (int rc = launch_result()) return rc;
  hipLaunchKernelGGL((distill_grad_kernel<DT, TAIL, NT>), dim3((unsigned)(a.rows * blocks)),
                     dim3(NT), slot_bytes(a.slots), s, a, blocks);
  return launch_result();
}

}  // namespace

extern "C" {

uint64_t zs_distill_workspace(uint64_t rows, uint64_t vocab, uint32_t slots, int dtype) {
  if (rows == 0 || !valid_any(dtype) || matrix_too_big(rows, vocab)) return 0;
  const DistillSplit sp = distill_split(rows, vocab, dtype);
  /* one part where a row per block would do, for gradients that it cannot store */
  return sp.parts ? rows * (sp.parts * sizeof(DistillPart) + slots * 4ull)
                  : rows * sizeof(DistillPart);
}

int zs_distill(const void *logits, int dtype, uint64_t rows, uint64_t vocab, uint64_t ld,
               const int32_t *ids, const void *teacher, uint32_t slots, float temperature,
               const float *teacher_lse, const float *row_weight, float loss_scale,
               const zs_device_scaler *dev, float *loss, void *grad, uint64_t grad_ld,
               void *workspace, uint64_t workspace_bytes, void *stream) {
  if (!valid_any(dtype)) return fail(ZS_ERR_INVALID_ARG, "zs_distill: bad dtype%s");
  /* the reciprocal of anything smaller is no fp32 number */
  if (!(temperature >= 0x1p-126f) || !isfinite(temperature))
    return fail(ZS_ERR_INVALID_ARG, "zs_distill: temperature must be finite and at least 2^-126%s");
  if (!dev && (!(loss_scale > 0.0f) || !isfinite(loss_scale)))
    return fail(ZS_ERR_INVALID_ARG, "zs_distill: loss_scale must be finite and > 0%s");
  if (vocab == 0 || vocab > kMaxVocab || ld < vocab || (grad && grad_ld < vocab))
    return fail(ZS_ERR_INVALID_ARG,
                "zs_distill: need 0 < vocab < 2^31 and rows at least vocab apart%s");
  if (slots > kMaxSlots) return fail(ZS_ERR_UNSUPPORTED, "zs_distill: more than 1024 slots%s");
  if (matrix_too_big(rows, ld) || (grad && matrix_too_big(rows, grad_ld)))
    return fail(ZS_ERR_UNSUPPORTED, "zs_distill: more than 2^48 elements%s");
  if (rows == 0) return ZS_OK;
  if (!logits || !loss || (slots && (!ids || !teacher)))
    return fail(ZS_ERR_INVALID_ARG, "zs_distill: null pointer%s");
  const uint64_t esz = esize(dtype);
  DistillSplit sp = distill_split(rows, vocab, dtype);
  const uint64_t need = zs_distill_workspace(rows, vocab, slots, dtype);
  if (need && (!workspace || workspace_bytes < need))
    return fail(ZS_ERR_INVALID_ARG, "zs_distill: workspace too small%s");
  if (!aligned(logits, esz) || !aligned(grad, esz) || !aligned(workspace, 16) ||
      !aligned(dev, 8) || !aligned(ids, 4) || !aligned(teacher, esz) || !aligned(loss, 4) ||
      !aligned(teacher_lse, 4) || !aligned(row_weight, 4))
    return fail(ZS_ERR_UNSUPPORTED, "zs_distill: an operand is not aligned%s");
  const uint64_t z_bytes = extent(rows, vocab, ld, esz);
  const uint64_t g_bytes = grad ? extent(rows, vocab, grad_ld, esz) : 0;
  const void *outs[] = {grad, loss, workspace};
  const uint64_t out_bytes[] = {g_bytes, rows * 4, need};
  const void *ins[] = {logits, ids, teacher, teacher_lse, row_weight, dev};
  const uint64_t in_bytes[] = {z_bytes, rows * slots * 4, rows * slots * esz, rows * 4, rows * 4,
                               sizeof(zs_device_scaler)};
  for (int i = 0; i < 3; ++i) {
    /* the gradient may take the logits' place */
    for (int j = 0; j < 6; ++j)
      if (overlaps(outs[i], out_bytes[i], ins[j], in_bytes[j]) &&
          !(i == 0 && j == 0 && grad == logits && grad_ld == ld))
        return fail(ZS_ERR_ALIAS, "zs_distill: an output overlaps an input%s");
    for (int j = i + 1; j < 3; ++j)
      if (overlaps(outs[i], out_bytes[i], outs[j], out_bytes[j]))
        return fail(ZS_ERR_ALIAS, "zs_distill: two outputs overlap%s");
  }
  DistillArgs a{};
  a.z = logits;
  a.ids = ids;
  a.teacher = teacher;
  a.lse = teacher_lse;
  a.weight = row_weight;
  a.dev = dev;
  a.loss = loss;
  a.grad = grad;
  a.ws = static_cast<DistillPart *>(workspace);
  if (sp.parts) a.ws_z = reinterpret_cast<float *>(a.ws + rows * sp.parts);
  a.rows = rows;
  a.ld = ld;
  a.gld = grad_ld;
  a.vocab = (uint32_t)vocab;
  a.slots = slots;
  a.tau = temperature;
  a.inv_tau = 1.0f / temperature;
  a.inv_tau64 = 1.0 / temperature;
  a.log2_scale = (float)(1.4426950408889634 / temperature);
  a.scale = loss_scale;
  a.vec_store = grad && (((uintptr_t)grad ^ (uintptr_t)logits) & 15) == 0 &&
                (grad_ld - ld) * esz % 16 == 0;
  /* such a gradient is not the logits' own buffer: its slots' logits stay */
  if (!sp.parts && grad && !a.vec_store) sp = {1, sp.vecs, sp.vecs};
  /* rows are counted in 32 bits, with room for a grid more */
  if (rows >= 1ull << 31 || (sp.parts && !fits(rows * sp.parts, kDistillThreads)))
    return fail(ZS_ERR_UNSUPPORTED, "zs_distill: too many rows%s");
  a.parts = sp.parts;
  a.part_vecs = sp.part_vecs;
  hipStream_t s = static_cast<hipStream_t>(stream);
  int rc = ZS_OK;
  with_any(dtype, [&](auto dt) {
    with_bool(teacher_lse != nullptr, [&](auto tail) {
      rc = launch_distill<decltype(dt)::value, decltype(tail)::value>(a, sp, s);
    });
  });
  return rc;
}

}  /* extern "C" */
