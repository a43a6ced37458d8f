"""The output end of a student model, trained in low precision against a
teacher's top logits, between the 16-bit parameters that the optimizer shard
gives out and the loss-scaled 16-bit gradients that it takes in.

    h = x + residual, y = rmsnorm(h) * gain          16 bits, and 8 with scales
    logits = y8 W4^T                                  8 x 4 bits
    loss, dlogits = distill(logits, teacher's top)    times the loss scale
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


class DistillHead:
    """Norm gain [width] and head weights [vocab][width], laid out in this
    order in the flat parameter and gradient buffers; `rows` tokens a step.

    grads: the flat 16-bit gradient that step() fills; dx: the gradient of
    its x and residual; loss: fp32 per row (row_weight included)."""

    def __init__(self, rows, width, vocab, slots, dtype=torch.bfloat16, eps=1e-5,
                 temperature=1.0, device="cuda"):
        self.rows, self.width, self.vocab, self.slots = rows, width, vocab, slots
        self.eps, self.temperature = eps, temperature
        self.phi = width + vocab * width
        t16, t32 = dict(dtype=dtype, device=device), dict(dtype=torch.float32, device=device)
        self.h, self.y, self.dy, self.dx = (torch.empty(rows, width, **t16) for _ in range(4))
        self.logits = torch.empty(rows, vocab, **t16)      # the gradient takes its place
        self.rstd, self.loss = torch.empty(rows, **t32), torch.empty(rows, **t32)
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
        need = max(16, zs.zs_distill_workspace(rows, vocab, slots, code),
                   zs.zs_rmsnorm_backward_workspace(rows, width),
                   zs.zs_mx_matmul_workspace(rows, vocab, width),
                   zs.zs_mx_matmul_workspace(rows, width, vocab),
                   zs.zs_mx_matmul_workspace(vocab, width, rows))
        self._ws = torch.empty(need, dtype=torch.uint8, device=device)

    def split(self, flat):
        """(gain, weights) of a flat parameter or gradient buffer."""
        return flat[:self.width], flat[self.width:self.phi].view(self.vocab, self.width)

    def step(self, params, x, residual, ids, teacher, dev_scaler=None, loss_scale=1.0,
             teacher_lse=None, row_weight=None, stream=None):
        """Forward and backward of one batch: fills loss, grads and dx, all
        queued. params: the flat 16-bit parameters (e.g. ShardState.params);
        dev_scaler: ShardState.dev, whose scale the gradients then carry."""
        s = dict(stream=stream)
        e2, e4 = zs.ZS_MX_E2M1, zs.ZS_MX_E4M3
        gain, weight = self.split(params)
        _, dweight = self.split(self.grads)
        zs.zs_rmsnorm_forward(x, gain, self.eps, h=self.h, rstd=self.rstd, residual=residual,
                              codes=self._y8[0], scales=self._y8[1], y=self.y, **s)
        zs.zs_mx_quantize(weight, e2, *self._w4, **s)
        zs.zs_mx_matmul(*self._y8, e4, *self._w4, self.logits, self.width, workspace=self._ws, **s)
        zs.zs_distill(self.logits, ids, teacher, self.temperature, self.loss, grad=self.logits,
                      teacher_lse=teacher_lse, row_weight=row_weight, loss_scale=loss_scale,
                      dev_scaler=dev_scaler, workspace=self._ws, **s)
        dlogits = self.logits
        zs.zs_mx_quantize(dlogits, e4, *self._d8, **s)
        zs.zs_mx_quantize(weight, e2, *self._wt4, columns=True, **s)
        zs.zs_mx_matmul(*self._d8, e4, *self._wt4, self.dy, self.vocab, workspace=self._ws, **s)
        zs.zs_mx_quantize(dlogits, e4, *self._dt8, columns=True, **s)
        zs.zs_mx_quantize(self.y, e2, *self._yt4, columns=True, **s)
        zs.zs_mx_matmul(*self._dt8, e4, *self._yt4, dweight, self.rows, workspace=self._ws, **s)
        zs.zs_rmsnorm_backward(self.dy, self.h, self.rstd, gain, self.dx, self.dgain, self._ws, **s)
        zs.zs_cast_gather(self.dgain, self.grads, self._code, 0, self.width, **s)
        return self.loss
