/*
 * zs_tokens.hip -- libzeroshard's losses over the log-probabilities of given
 * tokens (gfx950): log-probabilities alone, the clipped policy loss and the
 * loss of paired sequences. Host side: argument validation, choice of the
 * kernels, launches. The device code is in zs_token_kernels.h.
 */
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "zeroshard.h"

#include "zs_ops_common.h"
#include "zs_token_kernels.h"

namespace {

using namespace zs;
using namespace zs_ops;

/* How a row's statistics are cut into parts: whole, a block for each row, but
 * for the policy's gradient of few long rows, which would leave most of the CUs
 * idle; then into parts of a vector or more for each of 256 threads, some 512
 * in all, which every block of the gradient joins for itself (13 x 50257 bf16
 * 8.4 us, a block for each row 12; but 13 x 4096 6.4 and 4.8). */
constexpr uint64_t kFewRows = 64, kLongRow = 2048;

struct TokenSplit {
  uint32_t parts, part_vecs;
};

TokenSplit token_split(uint64_t rows, uint64_t vocab, int dtype, bool cut) {
  const uint64_t vecs = vocab * esize(dtype) / 16;
  uint64_t parts = cut && rows <= kFewRows && vecs >= kLongRow ? 512 / rows : 1;
  if (parts > kMaxParts) parts = kMaxParts;
  if (parts > vecs / 256) parts = vecs / 256;
  if (parts < 1) parts = 1;
  const uint64_t each = vecs ? (vecs + parts - 1) / parts : 1;
  /* as many as have vectors; a row that is not aligned has one vector fewer,
   * and its last part then has that much less */
  parts = vecs ? (vecs + each - 1) / each : 1;
  return {(uint32_t)parts, (uint32_t)each};
}

/* `cut`: with room for parts; `pairs`: for pairs' log-probabilities. */
uint64_t token_workspace(uint64_t rows, uint64_t vocab, int dtype, bool cut, bool pairs) {
  if (rows == 0 || rows >> 31 || vocab == 0 || vocab > kMaxVocab || !valid_any(dtype) ||
      matrix_too_big(rows, vocab))
    return 0;
  return rows * (token_split(rows, vocab, dtype, cut).parts * sizeof(TokenPart) +
                 sizeof(TokenPlan) + sizeof(float) + (pairs ? sizeof(double) : 0));
}

/* What the three entry points put into `a` alike. */
void token_args(TokenArgs &a, const void *logits, int dtype, uint64_t rows, uint64_t vocab,
                uint64_t ld, const int32_t *ids, float temperature, bool cut,
                void *workspace) {
  a.z = logits;
  a.ids = ids;
  a.ld = ld;
  a.rows = (uint32_t)rows;
  a.vocab = (uint32_t)vocab;
  const TokenSplit sp = token_split(rows, vocab, dtype, cut);
  a.parts = sp.parts;
  a.part_vecs = sp.part_vecs;
  a.log2_scale = (float)(1.4426950408889634 / temperature);
  a.inv_tau = 1.0f / temperature;
  a.ws = static_cast<TokenPart *>(workspace);
  a.plan = reinterpret_cast<TokenPlan *>(a.ws + rows * sp.parts);
  a.own = reinterpret_cast<float *>(a.plan + rows);
}

/* Threads of a block for a part's statistics: a wave for short rows; as many
 * as there are where few rows leave the GPU idle. */
template <class F>
void with_token_threads(const TokenArgs &a, F f) {
  if (a.part_vecs <= 512) f(Tag<64>{});
  else if (a.rows * (uint64_t)a.parts >= 1024 || a.part_vecs <= 1024) f(Tag<256>{});
  else f(Tag<1024>{});
}

int launch_stats(const TokenArgs &a, int dtype, hipStream_t s) {
  with_any(dtype, [&](auto dt) {
    with_token_threads(a, [&](auto nt) {
      hipLaunchKernelGGL((token_stats_kernel<decltype(dt)::value, decltype(nt)::value>),
                         dim3(a.rows * a.parts), dim3(decltype(nt)::value), 0, s, a);
    });
  });
  return launch_result();
}

/* Logits of more than 2^32 vectors take several launches. */
int launch_grad(TokenArgs a, int dtype, bool join, hipStream_t s) {
  const uint64_t vecs = (uint64_t)a.vocab * esize(dtype) / 16;
  int rc = ZS_OK;
  auto launch = [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    a.blocks = vecs > NT ? (uint32_t)((vecs + NT - 1) / NT) : 1;
    const uint64_t most = 0xffffffffull / ((uint64_t)a.blocks * NT);   /* seven rows at least */
    for (a.row0 = 0; a.row0 < a.rows && !rc; a.row0 += (uint32_t)most) {
      const uint64_t n = a.rows - a.row0 < most ? a.rows - a.row0 : most;
      with_any(dtype, [&](auto dt) {
        with_bool(join, [&](auto j) {
          hipLaunchKernelGGL((token_grad_kernel<decltype(dt)::value, NT, decltype(j)::value>),
                             dim3((unsigned)(n * a.blocks)), dim3(NT), 0, s, a);
        });
      });
      rc = launch_result();
      if (n < most) break;   /* the row's number could wrap */
    }
  };
  if (vecs <= 64) launch(Tag<64>{});
  else launch(Tag<256>{});
  return rc;
}

/* Rows that a block's registers hold, and as many blocks as fit at the
 * registers the kernel is held to; a block for each of the shortest rows (65536
 * x 1000 bf16 46 us, walked 54; 65536 x 4096 205, walked 198). */
constexpr int kPolicyItems = 32;

template <int DT, int NT, int ITEMS>
void launch_policy_rows(const TokenArgs &a, hipStream_t s) {
  const uint64_t fit = (uint64_t)cu_count() * (ITEMS <= 16 ? 16 : 8) / (NT / 64);
  hipLaunchKernelGGL((policy_row_kernel<DT, NT, ITEMS>),
                     dim3((unsigned)(ITEMS <= 2 || a.rows < fit ? a.rows : fit)), dim3(NT), 0, s,
                     a);
}

/* Whether they do. Not where a row takes a CU to itself and there are fewer
 * rows than CUs: two passes over all CUs are faster then (65 x 128000 bf16 18
 * us, 21 in rows; 256 rows 33 and 38). */
bool policy_in_rows(const TokenArgs &a, int dtype) {
  const uint64_t vecs = (uint64_t)a.vocab * esize(dtype) / 16;
  if (vecs > 8192 && a.rows <= 256) return false;
  /* two vectors' worth of elements hold one, whatever the row's alignment */
  return a.grad && vecs >= 2 && vecs <= 512 * kPolicyItems &&
         (((uintptr_t)a.grad ^ (uintptr_t)a.z) & 15) == 0 &&
         (a.gld - a.ld) * esize(dtype) % 16 == 0;
}

int launch_policy(const TokenArgs &a, int dtype, hipStream_t s) {
  const uint64_t vecs = (uint64_t)a.vocab * esize(dtype) / 16;
  with_any(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (vecs <= 128) launch_policy_rows<DT, 64, 2>(a, s);
    else if (vecs <= 512) launch_policy_rows<DT, 64, 8>(a, s);
    else if (vecs <= 1024) launch_policy_rows<DT, 64, 16>(a, s);
    else if (vecs <= 2048) launch_policy_rows<DT, 128, 16>(a, s);
    else if (vecs <= 4096) launch_policy_rows<DT, 256, 16>(a, s);
    else if (vecs <= 8192) launch_policy_rows<DT, 512, 16>(a, s);
    else launch_policy_rows<DT, 512, kPolicyItems>(a, s);
  });
  return launch_result();
}

/* Whether the launches of a call stay below 2^32 threads. */
bool token_launch_fits(uint64_t rows, const TokenSplit &sp) {
  return rows < 1ull << 31 && fits(rows * sp.parts, 256);
}

/* Checks of logits, tokens, temperature and gradient. Names: one message per
 * fault and entry point. */
#define ZS_TOKEN_CHECKS(NAME)                                                                    \
  if (!valid_any(dtype)) return fail(ZS_ERR_INVALID_ARG, NAME ": bad dtype%s");                  \
  if (!(temperature >= 0x1p-126f) || !isfinite(temperature))                                     \
    return fail(ZS_ERR_INVALID_ARG, NAME ": temperature must be finite and at least 2^-126%s");  \
  if (vocab == 0 || vocab > kMaxVocab || ld < vocab || (grad && grad_ld < vocab))                \
    return fail(ZS_ERR_INVALID_ARG,                                                              \
                NAME ": need 0 < vocab < 2^31 and rows at least vocab apart%s");                 \
  if (matrix_too_big(rows, ld) || (grad && matrix_too_big(rows, grad_ld)))                       \
    return fail(ZS_ERR_UNSUPPORTED, NAME ": more than 2^48 elements%s")

/* Outputs against inputs and each other; grad may be the logits' own buffer. */
int alias_check(const void *const *outs, const uint64_t *out_bytes, int n_outs,
                const void *const *ins, const uint64_t *in_bytes, int n_ins, bool in_place,
                const char *input, const char *two) {
  for (int i = 0; i < n_outs; ++i) {
    for (int j = 0; j < n_ins; ++j)
      if (overlaps(outs[i], out_bytes[i], ins[j], in_bytes[j]) && !(i == 0 && j == 0 && in_place))
        return fail(ZS_ERR_ALIAS, input);
    for (int j = i + 1; j < n_outs; ++j)
      if (overlaps(outs[i], out_bytes[i], outs[j], out_bytes[j])) return fail(ZS_ERR_ALIAS, two);
  }
  return ZS_OK;
}

}  // namespace

extern "C" {

uint64_t zs_logprob_workspace(uint64_t rows, uint64_t vocab, int dtype) {
  return token_workspace(rows, vocab, dtype, false, false);
}

int zs_logprob(const void *logits, int dtype, uint64_t rows, uint64_t vocab, uint64_t ld,
               const int32_t *ids, float temperature, float *logp, void *workspace,
               uint64_t workspace_bytes, void *stream) {
  const void *grad = nullptr;
  const uint64_t grad_ld = 0;
  ZS_TOKEN_CHECKS("zs_logprob");
  if (rows == 0) return ZS_OK;
  if (!logits || !ids || !logp) return fail(ZS_ERR_INVALID_ARG, "zs_logprob: null pointer%s");
  if (!token_launch_fits(rows, token_split(rows, vocab, dtype, false)))
    return fail(ZS_ERR_UNSUPPORTED, "zs_logprob: too many rows%s");
  const uint64_t esz = esize(dtype), need = zs_logprob_workspace(rows, vocab, dtype);
  if (!workspace || workspace_bytes < need)
    return fail(ZS_ERR_INVALID_ARG, "zs_logprob: workspace too small%s");
  if (!aligned(logits, esz) || !aligned(ids, 4) || !aligned(logp, 4) || !aligned(workspace, 16))
    return fail(ZS_ERR_UNSUPPORTED, "zs_logprob: an operand is not aligned%s");
  const void *outs[] = {logp, workspace};
  const uint64_t out_bytes[] = {rows * 4, need};
  const void *ins[] = {logits, ids};
  const uint64_t in_bytes[] = {extent(rows, vocab, ld, esz), rows * 4};
  if (int rc = alias_check(outs, out_bytes, 2, ins, in_bytes, 2, false,
                           "zs_logprob: an output overlaps an input%s",
                           "zs_logprob: two outputs overlap%s"))
    return rc;
  TokenArgs a{};
  token_args(a, logits, dtype, rows, vocab, ld, ids, temperature, false, workspace);
  a.logp = logp;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return launch_stats(a, dtype, s);
}

uint64_t zs_policy_workspace(uint64_t rows, uint64_t vocab, int dtype) {
  return token_workspace(rows, vocab, dtype, true, false);
}

int zs_policy(const void *logits, int dtype, uint64_t rows, uint64_t vocab, uint64_t ld,
              const int32_t *ids, float temperature, const float *advantage,
              const float *old_logp, const float *ref_logp, float clip_low, float clip_high,
              float kl_weight, const float *row_weight, float loss_scale,
              const zs_device_scaler *dev, float *logp, float *loss, void *grad, uint64_t grad_ld,
              void *workspace, uint64_t workspace_bytes, void *stream) {
  ZS_TOKEN_CHECKS("zs_policy");
  if (!(clip_low >= 0.0f && clip_low <= 1.0f) || !(clip_high >= 0.0f) || !isfinite(clip_high))
    return fail(ZS_ERR_INVALID_ARG,
                "zs_policy: need 0 <= clip_low <= 1 and a finite clip_high >= 0%s");
  if (!isfinite(kl_weight)) return fail(ZS_ERR_INVALID_ARG, "zs_policy: kl_weight not finite%s");
  if (!dev && (!(loss_scale > 0.0f) || !isfinite(loss_scale)))
    return fail(ZS_ERR_INVALID_ARG, "zs_policy: loss_scale must be finite and > 0%s");
  if (rows == 0) return ZS_OK;
  if (!logits || !ids || !advantage || !loss)
    return fail(ZS_ERR_INVALID_ARG, "zs_policy: null pointer%s");
  if (!token_launch_fits(rows, token_split(rows, vocab, dtype, true)))
    return fail(ZS_ERR_UNSUPPORTED, "zs_policy: too many rows%s");
  const uint64_t esz = esize(dtype), need = zs_policy_workspace(rows, vocab, dtype);
  if (!workspace || workspace_bytes < need)
    return fail(ZS_ERR_INVALID_ARG, "zs_policy: workspace too small%s");
  if (!aligned(logits, esz) || !aligned(ids, 4) || !aligned(advantage, 4) ||
      !aligned(old_logp, 4) || !aligned(ref_logp, 4) || !aligned(row_weight, 4) ||
      !aligned(dev, 8) || !aligned(logp, 4) || !aligned(loss, 4) || !aligned(grad, esz) ||
      !aligned(workspace, 16))
    return fail(ZS_ERR_UNSUPPORTED, "zs_policy: an operand is not aligned%s");
  const void *outs[] = {grad, loss, logp, workspace};
  const uint64_t out_bytes[] = {grad ? extent(rows, vocab, grad_ld, esz) : 0, rows * 4, rows * 4,
                                need};
  const void *ins[] = {logits, ids, advantage, old_logp, ref_logp, row_weight, dev};
  const uint64_t in_bytes[] = {extent(rows, vocab, ld, esz), rows * 4, rows * 4, rows * 4,
                               rows * 4, rows * 4, sizeof(zs_device_scaler)};
  if (int rc = alias_check(outs, out_bytes, 4, ins, in_bytes, 7, grad == logits && grad_ld == ld,
                           "zs_policy: an output overlaps an input%s",
                           "zs_policy: two outputs overlap%s"))
    return rc;
  TokenArgs a{};
  token_args(a, logits, dtype, rows, vocab, ld, ids, temperature, grad != nullptr, workspace);
  a.weight = row_weight;
  a.dev = dev;
  a.advantage = advantage;
  a.old_logp = old_logp;
  a.ref_logp = kl_weight != 0.0f ? ref_logp : nullptr;   /* 0 times an infinity is no term */
  a.clip_low = clip_low;
  a.clip_high = clip_high;
  a.kl_weight = kl_weight;
  a.scale = loss_scale;
  a.logp = logp;
  a.loss = loss;
  a.grad = grad;
  a.gld = grad_ld;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.parts == 1 && policy_in_rows(a, dtype)) return launch_policy(a, dtype, s);
  if (int rc = launch_stats(a, dtype, s)) return rc;
  return grad ? launch_grad(a, dtype, a.parts > 1, s) : ZS_OK;
}

uint64_t zs_preference_workspace(uint64_t rows, uint64_t vocab, int dtype) {
  return token_workspace(rows, vocab, dtype, false, true);
}

int zs_preference(const void *logits, int dtype, uint64_t rows, uint64_t vocab, uint64_t ld,
                  const int32_t *ids, const int32_t *starts, uint64_t pairs, float temperature,
                  const float *ref_logp, int kind, float beta, float smoothing, int mean,
                  const float *pair_weight, float loss_scale, const zs_device_scaler *dev,
                  float *seq_logp, float *loss, void *grad, uint64_t grad_ld, int clear, void *workspace,
                  uint64_t workspace_bytes, void *stream) {
  ZS_TOKEN_CHECKS("zs_preference");
  if (kind != ZS_PREFERENCE_SIGMOID && kind != ZS_PREFERENCE_HINGE && kind != ZS_PREFERENCE_SQUARE)
    return fail(ZS_ERR_INVALID_ARG, "zs_preference: bad kind%s");
  if (!(beta > 0.0f) || !isfinite(beta))
    return fail(ZS_ERR_INVALID_ARG, "zs_preference: beta must be finite and > 0%s");
  if (!(smoothing >= 0.0f && smoothing <= 1.0f) ||
      (smoothing != 0.0f && kind != ZS_PREFERENCE_SIGMOID))
    return fail(ZS_ERR_INVALID_ARG,
                "zs_preference: smoothing must lie in [0, 1], and be 0 but for the sigmoid%s");
  if (!dev && (!(loss_scale > 0.0f) || !isfinite(loss_scale)))
    return fail(ZS_ERR_INVALID_ARG, "zs_preference: loss_scale must be finite and > 0%s");
  if (pairs >> 22) return fail(ZS_ERR_UNSUPPORTED, "zs_preference: 2^22 pairs or more%s");
  if (pairs == 0 && !(clear && grad && rows)) return ZS_OK;
  if (!starts || (pairs && !loss) || (rows && (!logits || !ids)))
    return fail(ZS_ERR_INVALID_ARG, "zs_preference: null pointer%s");
  const TokenSplit sp = rows ? token_split(rows, vocab, dtype, false) : TokenSplit{1, 1};
  if (!token_launch_fits(rows, sp))
    return fail(ZS_ERR_UNSUPPORTED, "zs_preference: too many rows%s");
  const uint64_t esz = esize(dtype), need = zs_preference_workspace(rows, vocab, dtype);
  if (need && (!workspace || workspace_bytes < need))
    return fail(ZS_ERR_INVALID_ARG, "zs_preference: workspace too small%s");
  if (!aligned(logits, esz) || !aligned(ids, 4) || !aligned(starts, 4) || !aligned(ref_logp, 4) ||
      !aligned(pair_weight, 4) || !aligned(dev, 8) || !aligned(seq_logp, 4) || !aligned(loss, 4) ||
      !aligned(grad, esz) || !aligned(workspace, 16))
    return fail(ZS_ERR_UNSUPPORTED, "zs_preference: an operand is not aligned%s");
  const void *outs[] = {grad, loss, seq_logp, workspace};
  const uint64_t out_bytes[] = {grad ? extent(rows, vocab, grad_ld, esz) : 0, pairs * 4, pairs * 8,
                                need};
  const void *ins[] = {logits, ids, starts, ref_logp, pair_weight, dev};
  const uint64_t in_bytes[] = {extent(rows, vocab, ld, esz), rows * 4, (2 * pairs + 1) * 4,
                               pairs * 8, pairs * 4, sizeof(zs_device_scaler)};
  if (int rc = alias_check(outs, out_bytes, 4, ins, in_bytes, 6, grad == logits && grad_ld == ld,
                           "zs_preference: an output overlaps an input%s",
                           "zs_preference: two outputs overlap%s"))
    return rc;
  TokenArgs a{};
  if (rows) {
    token_args(a, logits, dtype, rows, vocab, ld, ids, temperature, false, workspace);
    /* behind the plans, 16 bytes each: the doubles stay aligned */
    a.lp = reinterpret_cast<double *>(a.plan + rows);
    a.own = reinterpret_cast<float *>(a.lp + rows);
  }
  a.starts = starts;
  a.pairs = (uint32_t)pairs;
  a.ref_seq = ref_logp;
  a.kind = kind;
  a.beta = beta;
  a.smoothing = smoothing;
  a.mean = mean;
  a.clear = clear;
  a.pair_weight = pair_weight;
  a.dev = dev;
  a.scale = loss_scale;
  a.seq_logp = seq_logp;
  a.loss = loss;
  a.grad = grad;
  a.gld = grad_ld;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows && (pairs || clear)) {
    if (int rc = launch_stats(a, dtype, s)) return rc;
  }
  if (pairs) {
    hipLaunchKernelGGL(token_pair_kernel, dim3(a.pairs), dim3(kPairThreads), 0, s, a);
    if (int rc = launch_result()) return rc;
  }
  return rows && grad ? launch_grad(a, dtype, false, s) : ZS_OK;
}

}  /* extern "C" */
