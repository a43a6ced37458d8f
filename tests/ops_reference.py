"""Plain 64-bit forms of the output end's operators, on the CPU (not collected
by pytest). Everything is torch float64 from the definitions in
include/zeroshard.h; nothing here calls the library."""
import math

import torch

F64 = torch.float64
BLOCK, GROUP = 32, 128
EMAX = {"e2m1": 2, "e4m3": 8}
GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=F64)


def padded(k):
    return -(-k // GROUP) * GROUP


def pow2(e):
    """2^e for whole e, exactly."""
    return torch.ldexp(torch.ones(e.shape, dtype=F64), e.to(torch.int32))


def mx_quantize(x, fmt):
    """(codes, scale bytes, values) of the rows of a float64 matrix."""
    r, k = x.shape
    p = padded(k)
    b = torch.zeros(r, p, dtype=F64)
    b[:, :k] = x
    b = b.view(r, p // BLOCK, BLOCK)
    bad = ~torch.isfinite(b).all(2)
    top = torch.where(bad, 0.0, torch.nan_to_num(b).abs().amax(2))
    # E of the fp32 exponent field: subnormals and zero have 0
    e = torch.where(top >= 2.0 ** -126, torch.frexp(top).exponent.to(torch.int64) + 126, 0)
    byte = (e - EMAX[fmt]).clamp(min=1)
    v = torch.nan_to_num(b) / pow2(byte - 127).unsqueeze(2)
    mag = v.abs()
    if fmt == "e2m1":
        lo = torch.searchsorted(GRID, mag.contiguous(), right=True) - 1
        hi = (lo + 1).clamp(max=7)
        mid = (GRID[lo] + GRID[hi]) / 2
        idx = torch.where((mag > mid) | ((mag == mid) & (lo % 2 == 1)), hi, lo)
        q = GRID[idx]
        code = idx + 8 * torch.signbit(v)
    else:
        ex = (torch.frexp(mag).exponent.to(torch.int64) - 1).clamp(min=-6)
        ex = torch.where(mag > 0, ex, -6)
        n = torch.round(mag / pow2(ex - 3))           # in units of the last place
        ex = torch.where(n == 16, ex + 1, ex)
        n = torch.where(n == 16, 8.0, n)
        q = n * pow2(ex - 3)
        over = q > 448
        q = torch.where(over, 448.0, q)
        code = torch.where(n < 8, n.long(), ((ex + 7) << 3) + n.long() - 8)
        code = torch.where(over, 0x7e, code) + 128 * torch.signbit(v)
    code = torch.where(bad.unsqueeze(2), 0, code).view(r, p)
    byte = torch.where(bad, 255, byte)
    val = torch.copysign(q, v) * pow2(torch.where(bad, 0, byte - 127)).unsqueeze(2)
    val = torch.where(bad.unsqueeze(2), math.nan, val).view(r, p)[:, :k]
    if fmt == "e2m1":
        code = code[:, 0::2] + 16 * code[:, 1::2]
    return code.to(torch.uint8), byte.to(torch.uint8), val


def mx_values(codes, byte, fmt, k):
    """The values of microscaled rows."""
    c = codes.long()
    if fmt == "e2m1":
        c = torch.stack([c & 15, c >> 4], 2).flatten(1)
        q = GRID[c & 7] * torch.where(c > 7, -1.0, 1.0)
    else:
        m, e = c & 7, (c >> 3) & 15
        q = torch.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * pow2(e - 7))
        q = q * torch.where(c > 127, -1.0, 1.0)
    s = pow2(byte.long() - 127)
    s = torch.where(byte == 255, math.nan, s)
    return (q * s.repeat_interleave(BLOCK, 1))[:, :k]


def rmsnorm(h, gain, eps):
    """(y, rstd) of float64 rows."""
    rstd = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return h * rstd * gain, rstd.squeeze(1)


def rmsnorm_grad(dy, h, rstd, gain, dres):
    """(dx, dgain), and the sums of magnitudes that bound their rounding."""
    r = rstd.unsqueeze(1)
    gdy = dy * gain
    s = (gdy * h).mean(1, keepdim=True) * r * r
    dx = r * (gdy - h * s) + (0 if dres is None else dres)
    mag = r * (gdy.abs() + h.abs() * r * r * (gdy * h).abs().mean(1, keepdim=True))
    mag = mag + (0 if dres is None else dres.abs())
    return dx, (dy * h * r).sum(0), mag, (dy * h * r).abs().sum(0)


def distill(z, ids, teacher, tau, lse=None, weight=None, scale=1.0):
    """(loss, gradient, bound): bound is S w tau (q + p), what a relative error
    of the probabilities scales with. Row by row, slot by slot."""
    rows, vocab = z.shape
    loss = torch.zeros(rows, dtype=F64)
    grad = torch.zeros(rows, vocab, dtype=F64)
    bound = torch.zeros(rows, vocab, dtype=F64)
    for i in range(rows):
        w = 1.0 if weight is None else float(weight[i])
        ok = (ids[i] >= 0) & (ids[i] < vocab)
        tok, t = ids[i][ok].long(), teacher[i][ok].to(F64) / tau
        if w == 0 or tok.numel() == 0:
            continue
        if lse is None and not bool((t > -math.inf).any() | torch.isnan(t).any()):
            continue
        logp = t - (torch.logsumexp(t, 0) if lse is None else lse[i].to(F64))
        u = z[i].to(F64) / tau
        logq = torch.log_softmax(u, 0)
        q, p = logq.exp(), logp.exp()
        part = torch.where(p == 0, 0.0, p * (logp - logq[tok]))
        total = part.sum()
        target = torch.zeros(vocab, dtype=F64).index_add_(0, tok, p)
        g = q - target
        if lse is not None:
            off = torch.ones(vocab, dtype=torch.bool)
            off[tok] = False
            pr, qr = 1 - float(p.sum()), float(q[off].sum())
            pr = pr if pr >= 2.0 ** -20 else 0.0
            if pr > 0:
                total = total + pr * (math.log(pr) - (math.log(qr) if qr > 0 else -math.inf))
            g = torch.where(off, q * (1 - pr / qr) if qr > 0 else torch.zeros(vocab, dtype=F64), g)
        loss[i] = w * tau * tau * total
        grad[i] = scale * w * tau * g
        bound[i] = abs(scale * w * tau) * (q + target)
    return loss, grad, bound
