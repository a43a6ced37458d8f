"""Plain 64-bit forms of the last block's operators, on the CPU (not collected
by pytest), from the definitions in include/zeroshard.h; nothing here calls the
library."""
import math

import torch

F64 = torch.float64
LOW = 0xFFFFFFFF


def philox(counter, key, rounds=7):
    """Philox4x32 of four counter words and two key words, in Python's integers."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & LOW, (a >> 32) ^ c[3] ^ k[1], a & LOW]
        k = [(k[0] + 0x9E3779B9) & LOW, (k[1] + 0xBB67AE85) & LOW]
    return c


def threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def keep_factor(rows, cols, p, seed, offset):
    """Each element's factor: 0 or 1 / (1 - p)."""
    drop = threshold(p)
    f = torch.ones(rows, cols, dtype=F64)
    if not drop:
        return f
    key, up = (seed & LOW, seed >> 32 & LOW), (offset & LOW, offset >> 32 & LOW)
    for r in range(rows):
        for b in range(-(-cols // 8)):
            w = philox((b, r, *up), key)
            for j in range(min(8, cols - 8 * b)):
                f[r, 8 * b + j] = (w[j // 2] >> 16 * (j % 2)) & 0xFFFF
    return (f >= drop).to(F64) * (65536 / (65536 - drop) if drop < 65536 else 0.0)


def dropped(x, factor):
    """x times its factor; what is dropped is 0 whatever it was."""
    return torch.where(factor > 0, x * factor, 0.0)


def rounded(v, dtype):
    """float64 values to the nearest of a 16-bit type, ties to even, as float64. (torch goes by
    way of float32, which makes ties of values that are none.)"""
    bits, low = (8, -133) if dtype == torch.bfloat16 else (11, -24)
    e = (torch.frexp(v).exponent - bits).clamp(min=low)
    step = torch.ldexp(torch.ones_like(v), e)
    r = torch.where(torch.isfinite(v), torch.round(v / step) * step, v)
    top = torch.finfo(dtype).max
    return torch.where(r.abs() > top, torch.copysign(torch.full_like(r, math.inf), r), r)


def block(x, res, post_gain, gate, gain, eps, residual_scale, branch_scale, factor, dtype):
    """(h rounded to dtype, as float64, h before it, post_rstd, rstd, y)."""
    n, post_rstd = x, None
    if post_gain is not None:
        post_rstd = 1 / torch.sqrt((x * x).mean(1) + eps)
        n = x * post_rstd.unsqueeze(1) * post_gain
    if gate is not None:
        n = n * gate
    wide = residual_scale * res + branch_scale * dropped(n, factor)
    h = rounded(wide, dtype)
    rstd = 1 / torch.sqrt((h * h).mean(1) + eps)
    return h, wide, post_rstd, rstd, h * rstd.unsqueeze(1) * gain


def block_grad(dy, h, rstd, gain, dres, x, post_rstd, post_gain, gate, residual_scale,
               branch_scale, factor):
    """(gradients by name, sums of magnitudes that bound their rounding)."""
    r = rstd.unsqueeze(1)
    gdy = dy * gain
    dh = r * (gdy - h * r * r * (gdy * h).mean(1, keepdim=True))
    mag = r * (gdy.abs() + h.abs() * r * r * (gdy * h).abs().mean(1, keepdim=True))
    if dres is not None:
        dh, mag = dh + dres, mag + dres.abs()
    out = {"dresidual": residual_scale * dh, "dgain": (dy * h * r).sum(0)}
    bound = {"dresidual": abs(residual_scale) * mag, "dgain": (dy * h * r).abs().sum(0)}
    t, tm = branch_scale * dropped(dh, factor), abs(branch_scale) * mag * factor
    q = torch.ones_like(gain)
    if post_gain is not None:
        q = q * post_gain
    if gate is not None:
        q = q * gate
    r1 = post_rstd.unsqueeze(1) if post_gain is not None else torch.ones(1, 1, dtype=F64)
    if post_gain is not None or gate is not None:
        u, um = (t * x * r1).sum(0), (tm * (x * r1).abs()).sum(0)
        if post_gain is not None:
            g = 1.0 if gate is None else gate
            out["dpost_gain"], bound["dpost_gain"] = u * g, um * abs(g)
        if gate is not None:
            g = 1.0 if post_gain is None else post_gain
            out["dgate"], bound["dgate"] = u * g, um * abs(g)
    out["dx"], bound["dx"] = t * q, tm * q.abs()
    if post_gain is not None:
        out["dx"] = r1 * (t * q - x * r1 * r1 * (t * q * x).mean(1, keepdim=True))
        bound["dx"] = r1 * (tm * q.abs() + x.abs() * r1 * r1
                            * (tm * (q * x).abs()).mean(1, keepdim=True))
    return out, bound
