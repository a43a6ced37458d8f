"""Plain 64-bit forms of the losses on given tokens' log-probabilities, on the
CPU (not collected by pytest), from the definitions in include/zeroshard.h;
nothing here calls the library."""
import math

import torch

F64 = torch.float64


def logprob(z, ids, tau):
    """(logp, softmax, which rows have a token) of float64 logits."""
    live = (ids >= 0) & (ids < z.shape[1])
    u = z / tau
    at = torch.where(live, ids, 0).long().unsqueeze(1)
    logq = torch.log_softmax(u, 1)
    mine = logq.gather(1, at).squeeze(1)
    # where the token has most of the mass 1 + x would round x away: log1p of the others' terms
    others = torch.exp(u - u.gather(1, at)).scatter(1, at, 0.0).sum(1)
    mine = torch.where(others < 1, -torch.log1p(others), mine)
    return torch.where(live, mine, 0.0), logq.exp(), live


def logit_grad(q, ids, slope):
    """slope (1[j = a] - q), with 1 - q of the token as the sum of the others."""
    g = -q * slope.unsqueeze(1)
    for i in torch.nonzero((ids >= 0) & (ids < q.shape[1])).flatten().tolist():
        a = int(ids[i])
        others = q[i].clone()
        others[a] = 0
        g[i, a] = slope[i] * others.sum()
    return g


def policy(z, ids, tau, adv, old, ref, low, high, kl, weight, scale):
    """(logp, loss, gradient, sum of magnitudes of the slope in logp times scale / tau)."""
    logp, q, live = logprob(z, ids, tau)
    w = torch.ones_like(adv) if weight is None else weight
    live = live & (w != 0)
    logp = torch.where(live, logp, 0.0)
    r = torch.ones_like(logp) if old is None else torch.exp(logp - old)
    flat = ((adv > 0) & (r > 1 + high)) | ((adv < 0) & (r < 1 - low))
    loss = -torch.where(flat, r.clamp(1 - low, 1 + high), r) * adv
    slope = torch.where(flat, 0.0, -adv * r)
    mag = slope.abs()
    if ref is not None:
        d = ref - logp
        loss = loss + kl * (torch.expm1(d) - d)
        slope = slope - kl * torch.expm1(d)
        mag = mag + abs(kl) * (torch.expm1(d).abs() + torch.exp(d))
    k = w * scale / tau
    loss, slope, mag = (torch.where(live, t, 0.0) for t in (w * loss, k * slope, k * mag))
    q = torch.where(live.unsqueeze(1), q, 0.0)
    return logp, loss, logit_grad(q, torch.where(live, ids, -1), slope), mag


def pair_loss(delta, kind, beta, smoothing):
    """(loss, its slope) of one pair's difference of log ratios, in Python's floats."""
    m = beta * delta
    if kind == "sigmoid":
        soft = lambda x: max(x, 0.0) + math.log1p(math.exp(-abs(x)))
        sig = lambda x: 1 / (1 + math.exp(-x)) if x > -700 else 0.0
        return ((1 - smoothing) * soft(-m) + smoothing * soft(m),
                beta * (smoothing * sig(m) - (1 - smoothing) * sig(-m)))
    if kind == "hinge":
        return max(0.0, 1 - m), (-beta if m < 1 else 0.0)
    d = delta - 1 / (2 * beta)
    return d * d, 2 * d


def preference(z, ids, starts, tau, ref, kind, beta, smoothing, mean, weight, scale):
    """(loss, seq_logp, gradient, |slope| per row, which rows belong to a sequence)."""
    logp, q, live = logprob(z, ids, tau)
    pairs = (len(starts) - 1) // 2
    seq, count = torch.zeros(2 * pairs, dtype=F64), torch.zeros(2 * pairs, dtype=F64)
    for s in range(2 * pairs):
        a, b = starts[s], starts[s + 1]
        count[s] = max(1, int(live[a:b].sum())) if mean else 1
        seq[s] = logp[a:b].sum() / count[s]
    slope = torch.zeros(z.shape[0], dtype=F64)
    loss = torch.zeros(pairs, dtype=F64)
    for p in range(pairs):
        w = 1.0 if weight is None else float(weight[p])
        ratio = seq[2 * p:2 * p + 2] - (0 if ref is None else ref[2 * p:2 * p + 2])
        if w == 0:
            continue
        value, k = pair_loss(float(ratio[0] - ratio[1]), kind, beta, smoothing)
        loss[p] = w * value
        for side in (0, 1):
            s = 2 * p + side
            slope[starts[s]:starts[s + 1]] = (1, -1)[side] * w * k * scale / tau / float(count[s])
    slope = torch.where(live, slope, 0.0)
    inside = torch.zeros(z.shape[0], dtype=torch.bool)
    inside[starts[0]:starts[-1]] = True
    return loss, seq, logit_grad(torch.where(live.unsqueeze(1), q, 0.0), ids, slope), \
        slope.abs(), inside
