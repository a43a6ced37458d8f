"""The output end of a student model, trained in low precision against a
teacher's top logits, on preferences or on rewards, between the 16-bit
parameters that the optimizer shard gives out and the loss-scaled 16-bit
gradients that it takes in.

    h = x + residual, y = rmsnorm(h) * gain          16 bits, and 8 with scales
    logits = y8 W4^T                                  8 x 4 bits
    loss, dlogits = distill(logits, teacher's top)    times the loss scale
                    (or the policy or preference loss of given tokens)
    dy = dlogits8 W4 ; dW = dlogits8^T y4             8 x 4 bits
    dx, dgain = rmsnorm backward                      16 bits, fp32

The product's right side is always 4 bits. For dW that is y, quantised anew from
its 16 bits along the rows: the weights' gradient sees it coarser than the
forward pass, which has it in 8 bits.

Everything is queued on one stream through the library's own kernels; with the
shard's device scaler nothing waits for the host, and a gradient that
overflows is skipped by the step that reads it.
"""
import torch

from . import zeroshard as zs


class _Head:
    """Norm gain [width] and head weights [vocab][width], laid out in this
    order in the flat parameter and gradient buffers; `rows` tokens a step.

    grads: the flat 16-bit gradient that step() fills; dx: the gradient of
    its x and residual. A subclass has the loss."""

    def __init__(self, rows, width, vocab, dtype, eps, temperature, device, loss_workspace):
        self.rows, self.width, self.vocab = rows, width, vocab
        self.eps, self.temperature, self.device = eps, temperature, device
        self.phi = width + vocab * width
        t16, t32 = dict(dtype=dtype, device=device), dict(dtype=torch.float32, device=device)
        self.h, self.y, self.dy, self.dx = (torch.empty(rows, width, **t16) for _ in range(4))
        self.logits = torch.empty(rows, vocab, **t16)      # the gradient takes its place
        self.rstd = torch.empty(rows, **t32)
        self.dgain = torch.empty(width, **t32)
        self.grads = torch.zeros(self.phi, **t16)
        e2, e4 = zs.ZS_MX_E2M1, zs.ZS_MX_E4M3
        self._y8 = zs.mx_empty(rows, width, e4, device)
        self._w4 = zs.mx_empty(vocab, width, e2, device)
        self._wt4 = zs.mx_empty(width, vocab, e2, device)
        self._d8 = zs.mx_empty(rows, vocab, e4, device)
        self._dt8 = zs.mx_empty(vocab, rows, e4, device)
        self._yt4 = zs.mx_empty(width, rows, e2, device)
        code = zs.ZS_BF16 if dtype == torch.bfloat16 else zs.ZS_FP16
        self._code = code
        # one workspace: the calls that use it follow each other on one stream
        need = max(16, loss_workspace(rows, vocab, code),
                   zs.zs_rmsnorm_backward_workspace(rows, width),
                   zs.zs_mx_matmul_workspace(rows, vocab, width),
                   zs.zs_mx_matmul_workspace(rows, width, vocab),
                   zs.zs_mx_matmul_workspace(vocab, width, rows))
        self._ws = torch.empty(need, dtype=torch.uint8, device=device)

    def split(self, flat):
        """(gain, weights) of a flat parameter or gradient buffer."""
        return flat[:self.width], flat[self.width:self.phi].view(self.vocab, self.width)

    def _norm(self, gain, x, residual, s):
        zs.zs_rmsnorm_forward(x, gain, self.eps, h=self.h, rstd=self.rstd, residual=residual,
                              codes=self._y8[0], scales=self._y8[1], y=self.y, **s)

    def _product(self, weight, s):
        """Logits of the norm's output."""
        zs.zs_mx_quantize(weight, zs.ZS_MX_E2M1, *self._w4, **s)
        zs.zs_mx_matmul(*self._y8, zs.ZS_MX_E4M3, *self._w4, self.logits, self.width,
                        workspace=self._ws, **s)

    def _product_backward(self, weight, dweight, s):
        """dy and the weights' gradient from the logits' gradient."""
        e2, e4 = zs.ZS_MX_E2M1, zs.ZS_MX_E4M3
        dlogits = self.logits
        zs.zs_mx_quantize(dlogits, e4, *self._d8, **s)
        zs.zs_mx_quantize(weight, e2, *self._wt4, columns=True, **s)
        zs.zs_mx_matmul(*self._d8, e4, *self._wt4, self.dy, self.vocab, workspace=self._ws, **s)
        zs.zs_mx_quantize(dlogits, e4, *self._dt8, columns=True, **s)
        zs.zs_mx_quantize(self.y, e2, *self._yt4, columns=True, **s)
        zs.zs_mx_matmul(*self._dt8, e4, *self._yt4, dweight, self.rows, workspace=self._ws, **s)

    def _step(self, params, x, residual, s, **loss):
        gain, weight = self.split(params)
        self._norm(gain, x, residual, s)
        self._product(weight, s)
        self._loss(s, **loss)
        self._product_backward(weight, self.split(self.grads)[1], s)
        zs.zs_rmsnorm_backward(self.dy, self.h, self.rstd, gain, self.dx, self.dgain, self._ws, **s)
        zs.zs_cast_gather(self.dgain, self.grads, self._code, 0, self.width, **s)
        return self.loss


class DistillHead(_Head):
    """Distillation from a teacher's top `slots` logits. loss: fp32 per row (row_weight
    included)."""

    def __init__(self, rows, width, vocab, slots, dtype=torch.bfloat16, eps=1e-5,
                 temperature=1.0, device="cuda"):
        super().__init__(rows, width, vocab, dtype, eps, temperature, device,
                         lambda r, v, code: zs.zs_distill_workspace(r, v, slots, code))
        self.slots = slots
        self.loss = torch.empty(rows, dtype=torch.float32, device=device)

    def _loss(self, s, ids, teacher, teacher_lse=None, row_weight=None, loss_scale=1.0,
              dev_scaler=None):
        zs.zs_distill(self.logits, ids, teacher, self.temperature, self.loss, grad=self.logits,
                      teacher_lse=teacher_lse, row_weight=row_weight, loss_scale=loss_scale,
                      dev_scaler=dev_scaler, workspace=self._ws, **s)

    def step(self, params, x, residual, ids, teacher, dev_scaler=None, loss_scale=1.0,
             teacher_lse=None, row_weight=None, stream=None):
        """Forward and backward of one batch: fills loss, grads and dx, all
        queued. params: the flat 16-bit parameters (e.g. ShardState.params);
        dev_scaler: ShardState.dev, whose scale the gradients then carry."""
        return self._step(params, x, residual, dict(stream=stream), ids=ids, teacher=teacher,
                          teacher_lse=teacher_lse, row_weight=row_weight, loss_scale=loss_scale,
                          dev_scaler=dev_scaler)


class PolicyHead(_Head):
    """Clipped policy loss with a KL term, against the sampler's and a reference model's
    log-probabilities of the tokens `ids` (an id below 0: a prompt's token, or padding). loss
    and logp: fp32 per row."""

    def __init__(self, rows, width, vocab, dtype=torch.bfloat16, eps=1e-5, temperature=1.0,
                 clip_low=0.2, clip_high=0.2, kl_weight=0.0, device="cuda"):
        super().__init__(rows, width, vocab, dtype, eps, temperature, device,
                         zs.zs_policy_workspace)
        self.clip_low, self.clip_high, self.kl_weight = clip_low, clip_high, kl_weight
        self.loss, self.logp = (torch.empty(rows, dtype=torch.float32, device=device)
                                for _ in range(2))

    def _loss(self, s, ids, advantage, **more):
        zs.zs_policy(self.logits, ids, advantage, self.loss, temperature=self.temperature,
                     clip_low=self.clip_low, clip_high=self.clip_high, kl_weight=self.kl_weight,
                     logp=self.logp, grad=self.logits, workspace=self._ws, **more, **s)

    def logprobs(self, params, x, residual, ids, stream=None):
        """Log-probability of each row's token, fp32: what old_logp and ref_logp are made of (with
        a block in front BlockStudent.logprobs: params are the head's own here)."""
        s = dict(stream=stream)
        gain, weight = self.split(params)
        self._norm(gain, x, residual, s)
        self._product(weight, s)
        zs.zs_logprob(self.logits, ids, self.logp, temperature=self.temperature,
                      workspace=self._ws, **s)
        return self.logp

    def step(self, params, x, residual, ids, advantage, old_logp=None, ref_logp=None,
             dev_scaler=None, loss_scale=1.0, row_weight=None, stream=None):
        """As DistillHead.step."""
        return self._step(params, x, residual, dict(stream=stream), ids=ids, advantage=advantage,
                          old_logp=old_logp, ref_logp=ref_logp, row_weight=row_weight,
                          loss_scale=loss_scale, dev_scaler=dev_scaler)


class PreferenceHead(_Head):
    """Preference loss of `pairs` pairs of sequences, rows starts[s] to starts[s + 1] each, of
    which the first is preferred. loss: fp32 per pair; seq_logp: fp32 per sequence."""

    def __init__(self, rows, width, vocab, pairs, beta, kind=zs.ZS_PREFERENCE_SIGMOID,
                 smoothing=0.0, mean=False, dtype=torch.bfloat16, eps=1e-5, temperature=1.0,
                 device="cuda"):
        super().__init__(rows, width, vocab, dtype, eps, temperature, device,
                         zs.zs_preference_workspace)
        self.pairs, self.beta, self.kind = pairs, beta, kind
        self.smoothing, self.mean = smoothing, mean
        self.loss = torch.empty(pairs, dtype=torch.float32, device=device)
        self.seq_logp = torch.empty(2 * pairs, dtype=torch.float32, device=device)

    def _loss(self, s, ids, starts, **more):
        # zeros outside all sequences, where the logits would stay: the products sum over all rows
        zs.zs_preference(self.logits, ids, starts, self.beta, self.loss, kind=self.kind,
                         smoothing=self.smoothing, mean=self.mean, temperature=self.temperature,
                         seq_logp=self.seq_logp, grad=self.logits, clear=True, workspace=self._ws,
                         **more, **s)

    def step(self, params, x, residual, ids, starts, ref_logp=None, dev_scaler=None,
             loss_scale=1.0, pair_weight=None, stream=None):
        """As DistillHead.step. starts: int32 [2 * pairs + 1] on the device; rows outside all
        sequences (padding) have no gradient."""
        return self._step(params, x, residual, dict(stream=stream), ids=ids, starts=starts,
                          ref_logp=ref_logp, pair_weight=pair_weight, loss_scale=loss_scale,
                          dev_scaler=dev_scaler)
