"""A student's last block and output end, trained in low precision between the
16-bit parameters that the optimizer shard gives out and the loss-scaled 16-bit
gradients that it takes in.

    h0 = x + residual, y0 = rmsnorm(h0) * gain0              16 bits, and 8 with scales
    a = act(y0 W1^T + b1)                                     8 x 4 bits, a to 8
    o = a W2^T + b2                                           8 x 4 bits
    h = l h0 + s dropout(gate * rmsnorm(o) * post_gain), y = rmsnorm(h) * gain
    logits, loss and back: the head (head.py), whose norm is the block's last
    do, dh0, its gains and the gate's gradient: the block norm's backward pass
    da = do8 W2, dpre = da act'(pre), dy0 = dpre8 W1 and the weights' gradients

As in the head, the products' right side is always 4 bits: the weights'
gradients see a and y0 coarser than the forward pass. Everything is queued on
one stream through the library's own kernels.
"""
import torch

from . import zeroshard as zs


class MlpBlock:
    """Parameters, in this order in the flat buffers: gain0 [width], W1 [hidden][width], b1
    [hidden], W2 [width][hidden], b2 [width], post_gain [width], gate [width]; `rows` tokens a
    step. dropout: p; the mask is a function of `seed` and of the offset that a step is given."""

    def __init__(self, rows, width, hidden, activation=zs.ZS_ACT_GELU, dropout=0.0, seed=0,
                 residual_scale=1.0, branch_scale=1.0, dtype=torch.bfloat16, eps=1e-5,
                 device="cuda"):
        self.rows, self.width, self.hidden, self.activation = rows, width, hidden, activation
        self.dropout, self.seed, self.eps = dropout, seed, eps
        self.scales = dict(residual_scale=residual_scale, branch_scale=branch_scale)
        self.shapes = ((width,), (hidden, width), (hidden,), (width, hidden), (width,), (width,),
                       (width,))
        self.phi = sum(torch.Size(s).numel() for s in self.shapes)
        t16, t32 = dict(dtype=dtype, device=device), dict(dtype=torch.float32, device=device)
        self.h0, self.y0, self.o, self.do, self.dh0, self.dy0, self.dx = (
            torch.empty(rows, width, **t16) for _ in range(7))
        self.a, self.pre, self.da = (torch.empty(rows, hidden, **t16) for _ in range(3))
        self.rstd0, self.post_rstd = (torch.empty(rows, **t32) for _ in range(2))
        # the fp32 gradients of the vectors, by their place among the parameters
        self.sums = {i: torch.empty(*self.shapes[i], **t32) for i in (0, 2, 4, 5, 6)}
        e2, e4 = zs.ZS_MX_E2M1, zs.ZS_MX_E4M3
        mx = lambda r, k, fmt: zs.mx_empty(r, k, fmt, device)
        self._y8, self._a8 = mx(rows, width, e4), mx(rows, hidden, e4)
        self._w1, self._w2 = mx(hidden, width, e2), mx(width, hidden, e2)
        self._w1t, self._w2t = mx(width, hidden, e2), mx(hidden, width, e2)
        self._do8, self._dot8 = mx(rows, width, e4), mx(width, rows, e4)
        self._dp8, self._dpt8 = mx(rows, hidden, e4), mx(hidden, rows, e4)
        self._at4, self._yt4 = mx(hidden, rows, e2), mx(width, rows, e2)
        self._code = zs.ZS_BF16 if dtype == torch.bfloat16 else zs.ZS_FP16
        need = max([16, zs.zs_rmsnorm_backward_workspace(rows, width),
                    zs.zs_block_norm_backward_workspace(rows, width),
                    zs.zs_activation_backward_workspace(rows, width),
                    zs.zs_activation_backward_workspace(rows, hidden)]
                   + [zs.zs_mx_matmul_workspace(*mnk) for mnk in
                      ((rows, hidden, width), (rows, width, hidden), (width, hidden, rows),
                       (hidden, width, rows))])
        self._ws = torch.empty(need, dtype=torch.uint8, device=device)

    def split(self, flat):
        """The parameters, or gradients, as views of a flat buffer."""
        out, at = [], 0
        for shape in self.shapes:
            n = torch.Size(shape).numel()
            out.append(flat[at:at + n].view(shape))
            at += n
        return out

    def _rule(self, offset):
        """offset: a number of the step's own, or (number, CUDA int64 tensor added to it); None:
        no dropout."""
        if not self.dropout or offset is None:
            return None
        return (self.dropout, self.seed, *(offset if isinstance(offset, tuple) else (offset,)))

    def forward(self, params, x, residual, gain, h, rstd, codes, scales, y, offset=0,
                stream=None):
        """The block up to the next norm (its gain, and its outputs as in
        zs_block_norm_forward)."""
        s = dict(stream=stream)
        e2, e4 = zs.ZS_MX_E2M1, zs.ZS_MX_E4M3
        gain0, w1, b1, w2, b2, post_gain, gate = self.split(params)
        zs.zs_rmsnorm_forward(x, gain0, self.eps, h=self.h0, rstd=self.rstd0, residual=residual,
                              codes=self._y8[0], scales=self._y8[1], y=self.y0, **s)
        zs.zs_mx_quantize(w1, e2, *self._w1, **s)
        zs.zs_mx_linear(*self._y8, e4, *self._w1, self.a, self.width, bias=b1,
                        activation=self.activation, pre=self.pre, workspace=self._ws, **s)
        zs.zs_mx_quantize(self.a, e4, *self._a8, **s)
        zs.zs_mx_quantize(w2, e2, *self._w2, **s)
        zs.zs_mx_linear(*self._a8, e4, *self._w2, self.o, self.hidden, bias=b2,
                        workspace=self._ws, **s)
        zs.zs_block_norm_forward(self.o, self.h0, gain, self.eps, h, rstd=rstd,
                                 post_gain=post_gain, post_rstd=self.post_rstd, gate=gate,
                                 dropout=self._rule(offset), codes=codes, scales=scales, y=y,
                                 **self.scales, **s)

    def backward(self, params, grads, dy, gain, h, rstd, dgain, offset=0, stream=None):
        """From the next norm's output's gradient dy to dx and the flat grads; dgain: the next
        norm's. offset: as in forward."""
        s = dict(stream=stream)
        e2, e4 = zs.ZS_MX_E2M1, zs.ZS_MX_E4M3
        gain0, w1, _, w2, _, post_gain, gate = self.split(params)
        _, dw1, _, dw2, *_ = self.split(grads)
        zs.zs_block_norm_backward(dy, h, rstd, gain, self.do, self.dh0, dgain, self._ws, x=self.o,
                                  post_gain=post_gain, post_rstd=self.post_rstd, gate=gate,
                                  dpost_gain=self.sums[5], dgate=self.sums[6],
                                  dropout=self._rule(offset), **self.scales, **s)
        zs.zs_activation_backward(self.do, None, zs.ZS_ACT_NONE, dbias=self.sums[4],
                                  workspace=self._ws, **s)
        zs.zs_mx_quantize(self.do, e4, *self._do8, **s)
        zs.zs_mx_quantize(w2, e2, *self._w2t, columns=True, **s)
        zs.zs_mx_matmul(*self._do8, e4, *self._w2t, self.da, self.width, workspace=self._ws, **s)
        zs.zs_mx_quantize(self.do, e4, *self._dot8, columns=True, **s)
        zs.zs_mx_quantize(self.a, e2, *self._at4, columns=True, **s)
        zs.zs_mx_matmul(*self._dot8, e4, *self._at4, dw2, self.rows, workspace=self._ws, **s)
        zs.zs_activation_backward(self.da, self.pre, self.activation, self.da, dbias=self.sums[2],
                                  workspace=self._ws, **s)
        zs.zs_mx_quantize(self.da, e4, *self._dp8, **s)
        zs.zs_mx_quantize(w1, e2, *self._w1t, columns=True, **s)
        zs.zs_mx_matmul(*self._dp8, e4, *self._w1t, self.dy0, self.hidden, workspace=self._ws, **s)
        zs.zs_mx_quantize(self.da, e4, *self._dpt8, columns=True, **s)
        zs.zs_mx_quantize(self.y0, e2, *self._yt4, columns=True, **s)
        zs.zs_mx_matmul(*self._dpt8, e4, *self._yt4, dw1, self.rows, workspace=self._ws, **s)
        zs.zs_rmsnorm_backward(self.dy0, self.h0, self.rstd0, gain0, self.dx, self.sums[0],
                               self._ws, dres=self.dh0, **s)
        at = 0
        for i, shape in enumerate(self.shapes):
            n = torch.Size(shape).numel()
            if i in self.sums:
                zs.zs_cast_gather(self.sums[i], grads, self._code, at, n, **s)
            at += n


class BlockStudent:
    """An MlpBlock and a head (DistillHead, PolicyHead or PreferenceHead) of the same rows and
    width, their parameters one after the other in the flat buffers. grads: the flat 16-bit
    gradient that step() fills; dx: the gradient of its x and residual; logp: fp32 per row, what
    logprobs() fills."""

    def __init__(self, block, head):
        if (block.rows, block.width, block._code) != (head.rows, head.width, head._code):
            raise ValueError("block and head differ in rows, width or dtype")
        self.block, self.head = block, head
        self.phi = block.phi + head.phi
        device = head.grads.device
        self.grads = torch.zeros(self.phi, dtype=head.grads.dtype, device=device)
        self.dx = block.dx
        self.logp = torch.empty(head.rows, dtype=torch.float32, device=device)
        need = zs.zs_logprob_workspace(head.rows, head.vocab, head._code)
        self._ws = head._ws if head._ws.numel() >= need else \
            torch.empty(need, dtype=torch.uint8, device=device)

    def split(self, flat):
        """(the block's, the head's) part of a flat buffer."""
        return flat[:self.block.phi], flat[self.block.phi:self.phi]

    def forward(self, params, x, residual, offset=0, stream=None):
        """Logits of a batch, in head.logits, with the step's dropout (offset None: without)."""
        mine, heads = self.split(params)
        gain, weight = self.head.split(heads)
        h = self.head
        self.block.forward(mine, x, residual, gain, h.h, h.rstd, *h._y8, h.y, offset=offset,
                           stream=stream)
        h._product(weight, dict(stream=stream))
        return h.logits

    def logprobs(self, params, x, residual, ids, offset=None, stream=None):
        """Log-probability of each row's token under the block and the head, without dropout or
        with an offset's, fp32: what old_logp and ref_logp are made of. (The head's own is that of
        a student without a block.)"""
        h = self.head
        self.forward(params, x, residual, offset, stream)
        zs.zs_logprob(h.logits, ids, self.logp, temperature=h.temperature, workspace=self._ws,
                      stream=stream)
        return self.logp

    def step(self, params, x, residual, offset=0, stream=None, **loss):
        """Forward and backward of one batch, all queued; loss: the head's step's arguments from
        ids on. Returns the head's loss."""
        s = dict(stream=stream)
        mine, heads = self.split(params)
        dmine, dheads = self.split(self.grads)
        gain, weight = self.head.split(heads)
        h = self.head
        self.forward(params, x, residual, offset, stream)
        h._loss(s, **loss)
        h._product_backward(weight, h.split(dheads)[1], s)
        self.block.backward(mine, dmine, h.dy, gain, h.h, h.rstd, h.dgain, offset=offset,
                            stream=stream)
        zs.zs_cast_gather(h.dgain, dheads, h._code, 0, h.width, **s)
        return h.loss
