"""The operators of a student's last block and of its training on preferences
and rewards, as they are measured.

Each case is one call that a training or serving program makes:

  dropout     out = residual + x * mask / (1 - p), the mask from a counter-based generator
  block_norm  a block's end: its output normed, gated, dropped out, scaled and
              added to the scaled residual stream, and the next block's norm
              of the sum (forward), and all of their gradients (backward)
  linear      product of microscaled operands with bias, activation and
              residual in its epilogue, or the gradient of that epilogue
  policy      clipped policy loss with a KL term and the logits' gradient, or
              the tokens' log-probabilities alone
  preference  loss of paired sequences' log ratios and the logits' gradient

Microscaled rows are padded with zeros to whole groups of 128 elements;
32 elements share a power-of-two scale held as an E8M0 byte.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32
GROUP = 128
EMAX = {"e2m1": 2, "e4m3": 8}
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5


def padded(k):
    return -(-k // GROUP) * GROUP


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # a short ragged batch between two layers of odd width, fp16: latency
        {"name": "dropout-ragged", "op": "dropout", "rows": 203, "cols": 1599, "dtype": "fp16",
         "p": 0.1, "residual": False},
        # a training micro-batch of a 7B-sized model's width, added to the residual stream
        {"name": "dropout-batch", "op": "dropout", "rows": 16384, "cols": 4096, "dtype": "bf16",
         "p": 0.1, "residual": True},
        # one decoded token of the GPT-2-small-shaped model: latency, no dropout
        {"name": "block-token", "op": "block_norm", "rows": 1, "cols": 768, "dtype": "bf16",
         "backward": False, "post": True, "gate": True, "p": 0.0, "out": "e4m3"},
        # the training micro-batch with dropout, 8-bit output for the next product
        {"name": "block-batch", "op": "block_norm", "rows": 16384, "cols": 4096, "dtype": "bf16",
         "backward": False, "post": True, "gate": True, "p": 0.1, "out": "e4m3"},
        # its gradient
        {"name": "block-grad-batch", "op": "block_norm", "rows": 16384, "cols": 4096,
         "dtype": "bf16", "backward": True, "post": True, "gate": True, "p": 0.1, "dres": True},
        # a short ragged prompt through a layer that ends in the residual stream, 4-bit activations
        {"name": "linear-prompt", "op": "linear", "m": 77, "n": 1600, "k": 6400, "a": "e2m1",
         "dtype": "fp16", "act": "none", "residual": True, "pre": False, "backward": False},
        # a training micro-batch through an MLP's first layer, its pre-activation kept
        {"name": "linear-batch", "op": "linear", "m": 8192, "n": 16384, "k": 4096, "a": "e4m3",
         "dtype": "bf16", "act": "gelu", "residual": False, "pre": True, "backward": False},
        # the gradient of that layer's activation and bias
        {"name": "linear-grad-batch", "op": "linear", "m": 8192, "n": 16384, "k": 4096, "a": "e4m3",
         "dtype": "bf16", "act": "gelu", "residual": False, "pre": True, "backward": True},
        # a few sampled tokens of GPT-2-small-shaped logits, asymmetric clip
        {"name": "policy-few", "op": "policy", "rows": 13, "vocab": 50257, "dtype": "fp16",
         "temperature": 0.7, "old": True, "ref": True, "only_logp": False},
        # a micro-batch of samples over a large vocabulary
        {"name": "policy-batch", "op": "policy", "rows": 8192, "vocab": 128000, "dtype": "bf16",
         "temperature": 1.0, "old": True, "ref": True, "only_logp": False},
        # two short pairs of GPT-2-small-shaped logits
        {"name": "preference-few", "op": "preference", "rows": 131, "pairs": 2, "vocab": 50257,
         "dtype": "fp16", "kind": "square", "mean": True, "smoothing": 0.0},
        # a micro-batch of pairs of answers over a 7B-sized model's vocabulary
        {"name": "preference-batch", "op": "preference", "rows": 16384, "pairs": 16,
         "vocab": 32000, "dtype": "bf16", "kind": "sigmoid", "mean": False, "smoothing": 0.1},
    ]


def _between(rng, lo, hi):
    """A whole number spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dropout", "block_norm", "block_norm", "linear", "linear", "policy",
                     "preference"])
    if op == "dropout":
        cols = _between(rng, 1, 16384)
        rows = _between(rng, 1, min(65536, (16384 * 4096) // cols))
        return {"op": op, "rows": rows, "cols": cols if rng.random() < 0.4 else -(-cols // 32) * 32,
                "dtype": rng.choice(["bf16", "fp16"] + ["fp32"] * (rows * cols < 1 << 25)),
                "p": rng.choice([0.0, 0.05, 0.1, 0.5, 0.9]), "residual": rng.random() < 0.5}
    if op == "block_norm":
        cols = _between(rng, 64, 8192)
        rows = _between(rng, 1, min(16384, (16384 * 4096) // cols))
        c = {"op": op, "rows": rows, "cols": cols if rng.random() < 0.4 else -(-cols // 32) * 32,
             "dtype": rng.choice(["bf16", "fp16"]), "backward": rng.random() < 0.5,
             "post": rng.random() < 0.7, "gate": rng.random() < 0.7,
             "p": rng.choice([0.0, 0.1, 0.3])}
        if c["backward"]:
            c["dres"] = rng.random() < 0.7
        else:
            c["out"] = rng.choice(["e4m3", "16"])
        return c
    if op == "linear":
        m = _between(rng, 1, 8192)
        n = _between(rng, 64, 16384)
        k = _between(rng, 64, 8192)
        while m * n * k > 8192 ** 3 // 4:
            n = max(64, n // 2)
        act = rng.choice(["none", "relu", "gelu", "silu"])
        return {"op": op, "m": m, "n": n, "k": k, "a": rng.choice(["e2m1", "e4m3"]),
                "dtype": rng.choice(["bf16", "fp16"]), "act": act,
                "residual": rng.random() < 0.5, "pre": act != "none" and rng.random() < 0.5,
                "backward": rng.random() < 0.3}
    vocab = _between(rng, 1000, 200000)
    dt = rng.choice(["bf16", "fp16", "fp32"])
    most = min(16384, ((1 << 30) if dt != "fp32" else (1 << 28)) // vocab)
    if op == "policy":
        return {"op": op, "rows": _between(rng, 1, most), "vocab": vocab, "dtype": dt,
                "temperature": rng.choice([1.0, 0.7, 2.0]), "old": rng.random() < 0.8,
                "ref": rng.random() < 0.7, "only_logp": rng.random() < 0.25}
    most = min(most, 16384 * 32000 // vocab)
    pairs = _between(rng, 1, max(1, most // 32))
    rows = _between(rng, 4 * pairs, max(4 * pairs, most))
    kind = rng.choice(["sigmoid", "hinge", "square"])
    return {"op": op, "rows": rows, "pairs": pairs, "vocab": vocab, "dtype": dt, "kind": kind,
            "mean": kind == "square", "smoothing": 0.1 if kind == "sigmoid" else 0.0}


# ---- inputs ------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _bytes(*shape):
    return torch.empty(*shape, dtype=torch.uint8, device="cuda")


def _width(fmt, k):
    """Bytes of a microscaled row of k elements."""
    return padded(k) // 2 if fmt == "e2m1" else padded(k)


def _packed(values, fmt):
    """Codes and scale bytes of a float32 matrix, as a program keeps them."""
    scale, q = _quantized(_pad(values), fmt)
    if fmt == "e4m3":
        codes = q.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        mag = q.abs()
        code = torch.where(mag < 2, mag * 2, torch.where(mag < 4, mag + 2, mag / 2 + 4))
        code = code.to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << 3)
        codes = code[:, 0::2] | (code[:, 1::2] << 4)
    return codes.contiguous(), scale


def _logits(g, rows, vocab, dt):
    """Logits of a student that knows something of the tokens it is given."""
    z = torch.randn(rows, vocab, generator=g, device="cuda",
                    dtype=torch.bfloat16 if dt == torch.bfloat16 else torch.float32)
    z *= 2
    ids = torch.randint(0, vocab, (rows, 1), generator=g, device="cuda")
    z.scatter_add_(1, ids, (4 + 2 * _randn(g, rows, 1)).to(z.dtype))
    z = z.to(dt)
    # prompt tokens and padding carry no loss
    live = torch.ones(rows, dtype=torch.bool, device="cuda")
    live[torch.randperm(rows, generator=g, device="cuda")[:rows // 8]] = False
    return z, ids.squeeze(1), live


def _logp32(z, ids, tau):
    """Log-probabilities to a few digits, some gigabytes at a time."""
    out = []
    for first in range(0, z.shape[0], 2048):
        u = z[first:first + 2048].float() / tau
        out.append(u.gather(1, ids[first:first + 2048, None]).squeeze(1) - torch.logsumexp(u, 1))
    return torch.cat(out)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    dt = DTYPE[case["dtype"]]
    if op in ("dropout", "block_norm"):
        # a run's seed, and a number of its own for each layer and step
        s["seed"] = 0x9E3779B97F4A7C15 ^ (seed * 0x100000001)
        s["offset"] = (1 << 33) + seed
    if op == "dropout":
        t, d = case["rows"], case["cols"]
        s["x"] = _randn(g, t, d).to(dt)
        s["res"] = (_randn(g, t, d) * 2).to(dt) if case["residual"] else None
        s["out"] = torch.empty(t, d, dtype=dt, device="cuda")
    elif op == "block_norm":
        t, d = case["rows"], case["cols"]
        # a branch whose rows differ in size, as a block's output does
        s["x"] = (_randn(g, t, d) * (0.2 + 2 * _rand(g, t, 1))).to(dt)
        s["gain"] = (1 + 0.1 * _randn(g, d)).to(dt)
        s["post_gain"] = (1 + 0.1 * _randn(g, d)).to(dt) if case["post"] else None
        s["gate"] = (0.3 + 0.2 * _randn(g, d)).to(dt) if case["gate"] else None
        s["residual_scale"], s["branch_scale"] = 0.875, 0.5
        if case["backward"]:
            s["h"] = (_randn(g, t, d) * (0.5 + 2 * _rand(g, t, 1))).to(dt)
            s["rstd"] = (s["h"].float().square().mean(1) + EPS).rsqrt()
            s["post_rstd"] = (s["x"].float().square().mean(1) + EPS).rsqrt() \
                if case["post"] else None
            s["dy"] = (_randn(g, t, d) * 0.05).to(dt)
            s["dres"] = (_randn(g, t, d) * 0.05).to(dt) if case["dres"] else None
            s["dx"], s["dresidual"] = (torch.empty(t, d, dtype=dt, device="cuda") for _ in range(2))
            for name, there in (("dgain", True), ("dpost_gain", case["post"]),
                                ("dgate", case["gate"])):
                s[name] = torch.empty(d, device="cuda") if there else None
            # room for the partial sums over the rows
            s["workspace"] = _bytes(1024 * d * 8)
        else:
            s["res"] = (_randn(g, t, d) * 2).to(dt)
            s["h"] = torch.empty(t, d, dtype=dt, device="cuda")
            s["rstd"] = torch.empty(t, device="cuda")
            s["post_rstd"] = torch.empty(t, device="cuda") if case["post"] else None
            if case["out"] == "e4m3":
                s["codes"], s["scales"] = _bytes(t, padded(d)), _bytes(t, padded(d) // BLOCK)
            else:
                s["y"] = torch.empty(t, d, dtype=dt, device="cuda")
    elif op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        if case["backward"]:
            s["dc"] = (_randn(g, m, n) * 0.05).to(dt)
            s["saved"] = (_randn(g, m, n) * 1.5).to(dt)
            s["dpre"] = torch.empty(m, n, dtype=dt, device="cuda")
            s["dbias"] = torch.empty(n, device="cuda")
            # room for the partial sums over the rows
            s["workspace"] = _bytes(1024 * n * 4)
            return s
        s["a_codes"], s["a_scales"] = _packed(_randn(g, m, k), case["a"])
        s["b_codes"], s["b_scales"] = _packed(_randn(g, n, k) * (1.2 / math.sqrt(k)), "e2m1")
        s["bias"] = (_randn(g, n) * 0.3).to(dt)
        s["res"] = (_randn(g, m, n) * 2).to(dt) if case["residual"] else None
        s["pre_out"] = torch.empty(m, n, dtype=dt, device="cuda") if case["pre"] else None
        s["c"] = torch.empty(m, n, dtype=dt, device="cuda")
        # room for the partial sums of a product split along k
        s["workspace"] = _bytes(32 << 20)
    elif op == "policy":
        t, v, tau = case["rows"], case["vocab"], case["temperature"]
        s["logits"], ids, live = _logits(g, t, v, dt)
        s["ids"] = torch.where(live, ids, -1).to(torch.int32)
        s["logp"] = torch.empty(t, device="cuda")
        s["workspace"] = _bytes(4 << 20)
        if case["only_logp"]:
            return s
        s["clip_low"], s["clip_high"], s["kl_weight"] = 0.2, 0.28, 0.04
        logp = _logp32(s["logits"], ids, tau)
        # the sampler's log-probabilities, some updates ago; no ratio lies within 1e-4 of the
        # clip's two ends, where 32 and 64 bits may choose differently
        drift = 0.15 * _randn(g, t)
        for end in (math.log1p(-s["clip_low"]), math.log1p(s["clip_high"])):
            drift = torch.where((drift - end).abs() < 2e-4, drift + 1e-3, drift)
        s["old_logp"] = logp - drift if case["old"] else None
        s["ref_logp"] = logp + 0.3 * _randn(g, t) if case["ref"] else None
        s["advantage"] = _randn(g, t)
        # the mean over the micro-batch's tokens
        s["weight"] = torch.full((t,), 1.0 / t, device="cuda")
        s["scale"] = 65536.0 if dt != torch.float16 else 1024.0
        s["loss"] = torch.empty(t, device="cuda")
        s["grad"] = torch.empty_like(s["logits"])
    else:
        t, v, pairs = case["rows"], case["vocab"], case["pairs"]
        s["logits"], ids, live = _logits(g, t, v, dt)
        s["ids"] = torch.where(live, ids, -1).to(torch.int32)
        # ragged answers, none of them empty
        cuts = torch.randperm(t - 1, generator=g, device="cuda")[:2 * pairs - 1].sort().values + 1
        s["starts"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), t)]).to(torch.int32)
        s["beta"] = 0.1
        logp = torch.where(live, _logp32(s["logits"], ids, 1.0), 0.0).double()
        seq = torch.searchsorted(s["starts"].long(), torch.arange(t, device="cuda"), right=True) - 1
        total = torch.zeros(2 * pairs, dtype=torch.float64, device="cuda").index_add_(0, seq, logp)
        count = torch.zeros_like(total).index_add_(0, seq, live.double()).clamp(min=1)
        # the reference model's log-probabilities of the same answers
        apart = 0.3 * _randn(g, 2 * pairs) if case["mean"] else 8 * _randn(g, 2 * pairs)
        s["ref_logp"] = ((total / count if case["mean"] else total) + apart).float()
        s["weight"] = torch.full((pairs,), 1.0 / pairs, device="cuda")
        s["scale"] = 65536.0 if dt != torch.float16 else 1024.0
        s["seq_logp"], s["loss"] = torch.empty(2 * pairs, device="cuda"), \
            torch.empty(pairs, device="cuda")
        s["grad"] = torch.empty_like(s["logits"])
        # room for the rows' statistics
        s["workspace"] = _bytes(4 << 20)
    return s


# ---- plain forms -------------------------------------------------------------

def _pad(x):
    return torch.nn.functional.pad(x, (0, padded(x.shape[1]) - x.shape[1]))


def _quantized(x, fmt):
    """(scale bytes [R, K/32], element values [R, K]) of a padded float32 matrix."""
    blocks = x.view(x.shape[0], -1, BLOCK)
    exponent = (blocks.abs().amax(2).view(torch.int32) >> 23) - EMAX[fmt]
    byte = exponent.clamp(1, 254)
    v = blocks / (byte << 23).view(torch.float32).unsqueeze(2)
    if fmt == "e4m3":
        q = v.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    else:
        mag = v.abs()
        mag = torch.where(mag < 2, torch.round(mag * 2) / 2,
                          torch.where(mag < 4, torch.round(mag), torch.round(mag / 2) * 2))
        q = torch.copysign(mag.clamp(max=6), v)
    return byte.to(torch.uint8), q.view(x.shape)


def _unpacked(codes, scales, fmt):
    if fmt == "e4m3":
        q = codes.view(torch.float8_e4m3fn).float()
    else:
        code = torch.stack([codes & 15, codes >> 4], 2).view(codes.shape[0], -1)
        low = (code & 7).float()
        mag = torch.where(low < 4, low / 2, torch.where(low < 6, low - 2, low * 2 - 8))
        q = torch.where(code > 7, -mag, mag)
    scale = (scales.to(torch.int32) << 23).view(torch.float32)
    return (q.view(q.shape[0], -1, BLOCK) * scale.unsqueeze(2)).view(q.shape)


def _threshold(p):
    """Of 65536 equally likely numbers, how many drop an element."""
    return int(math.floor(p * 65536 + 0.5))


def _random_words(rows, cols, seed, offset):
    """Philox4x32, 7 rounds: four words for each 8 neighbouring elements of a row. Products of
    32-bit numbers in halves, for 64-bit integers here are signed."""
    m32 = 0xFFFFFFFF
    blocks = -(-cols // 8)
    c0 = torch.arange(blocks, device="cuda").repeat(rows, 1)
    c1 = torch.arange(rows, device="cuda").unsqueeze(1).repeat(1, blocks)
    c2, c3 = torch.full_like(c0, offset & m32), torch.full_like(c0, offset >> 32)
    k0, k1 = seed & m32, seed >> 32

    def product(c, m):
        low = (c & 0xFFFF) * m
        return ((c >> 16) * m + (low >> 16)) >> 16, (c * m) & m32

    for _ in range(7):
        h0, l0 = product(c0, 0xD2511F53)
        h1, l1 = product(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    return c0, c1, c2, c3


def _kept(s):
    """Which elements stay, and the factor that they get."""
    t, d, drop = s["rows"], s["cols"], _threshold(s["p"])
    if not drop:
        return torch.ones(t, d, dtype=torch.bool, device="cuda"), 1.0
    words = torch.stack(_random_words(t, d, s["seed"], s["offset"]), 2)
    halves = torch.stack([words & 0xFFFF, words >> 16], 3).view(t, -1)[:, :d]
    return halves >= drop, 65536 / (65536 - drop)


def _rounded(v, dt):
    """A float64 tensor rounded once to 16 bits: through float32 rounded to odd, not to nearest,
    which would make ties of values that are none."""
    y = v.float()
    rest = v - y.double()
    bits = y.view(torch.int32)
    odd = (bits - ((rest < 0) != (y < 0)).int()) | 1
    return torch.where(rest != 0, odd, bits).view(torch.float32).to(dt)


def _plain_dropout(s):
    kept, factor = _kept(s)
    out = torch.where(kept, s["x"].float() * factor, 0.0)
    if s["res"] is not None:
        out = out + s["res"].float()
    return {"out": out.to(s["x"].dtype)}


def _plain_block(s):
    kept, factor = _kept(s)
    # in 64 bits: h's rounding decides what the second norm and its codes see, and y lies next
    # to a border of its codes and scales here and there
    n = s["x"].double()
    out = {}
    if s["post"]:
        post_rstd = (n.square().mean(1) + EPS).rsqrt()
        n = n * post_rstd.unsqueeze(1) * s["post_gain"].double()
        out["post_rstd"] = post_rstd.float()
    if s["gate"] is not None:
        n = n * s["gate"].double()
    n = torch.where(kept, n * factor, 0.0)
    h = _rounded(s["res"].double() * s["residual_scale"] + n * s["branch_scale"], s["x"].dtype)
    v = h.double()
    rstd = (v.square().mean(1) + EPS).rsqrt()
    y = (v * rstd.unsqueeze(1) * s["gain"].double()).float()
    out.update(h=h, rstd=rstd.float())
    if s["out"] == "e4m3":
        byte, q = _quantized(_pad(y), "e4m3")
        out.update(y=q.to(torch.float8_e4m3fn), scale=byte.view(torch.float8_e8m0fnu))
    else:
        out.update(y=y.to(s["x"].dtype))
    return out


def _plain_block_grad(s):
    kept, factor = _kept(s)
    h, rstd, dy = s["h"].float(), s["rstd"].unsqueeze(1), s["dy"].float()
    gdy = dy * s["gain"].float()
    dh = rstd * (gdy - h * rstd.square() * (gdy * h).mean(1, keepdim=True))
    if s["dres"] is not None:
        dh = dh + s["dres"].float()
    out = {"dresidual": (dh * s["residual_scale"]).to(s["h"].dtype),
           "dgain": (dy * h * rstd).sum(0)}
    d = torch.where(kept, dh * (factor * s["branch_scale"]), 0.0)
    x = s["x"].float()
    gate = s["gate"].float() if s["gate"] is not None else 1.0
    if s["post"]:
        post, r = s["post_gain"].float(), s["post_rstd"].unsqueeze(1)
        u = (d * x * r).sum(0)
        out["dpost_gain"] = u * gate
        if s["gate"] is not None:
            out["dgate"] = u * post
        d = d * gate * post
        dx = r * (d - x * r.square() * (d * x).mean(1, keepdim=True))
    else:
        if s["gate"] is not None:
            out["dgate"] = (d * x).sum(0)
        dx = d * gate
    out["dx"] = dx.to(s["h"].dtype)
    return out


_GELU = math.sqrt(2 / math.pi)


def _act(x, act):
    if act == "relu":
        return x.clamp(min=0)
    if act == "gelu":     # 0.5 x (1 + tanh u) is x times the logistic function of 2 u
        return x / (1 + torch.exp(-2 * _GELU * (x + 0.044715 * x * x * x)))
    if act == "silu":
        return x / (1 + torch.exp(-x))
    return x


def _act_slope(x, act):
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "none":
        return torch.ones_like(x)
    if act == "gelu":
        u, du = 2 * _GELU * (x + 0.044715 * x * x * x), 2 * _GELU * (1 + 3 * 0.044715 * x * x)
    else:
        u, du = x, 1.0
    p = 1 / (1 + torch.exp(-u))
    return p + x * p * (1 / (1 + torch.exp(u))) * du


def _plain_linear(s):
    if s["backward"]:
        dpre = s["dc"].float() * _act_slope(s["saved"].float(), s["act"])
        return {"dpre": dpre.to(s["dc"].dtype), "dbias": dpre.sum(0)}
    a = _unpacked(s["a_codes"], s["a_scales"], s["a"])
    b = _unpacked(s["b_codes"], s["b_scales"], "e2m1")
    pre = torch.matmul(a, b.t()) + s["bias"].float()
    c = _act(pre, s["act"])
    if s["res"] is not None:
        c = c + s["res"].float()
    out = {"c": c.to(s["c"].dtype)}
    if s["pre"]:
        out["pre"] = pre.to(s["c"].dtype)
    return out


def _plain_tokens(s, tau):
    """(terms, their sums, log-probability of each row's token, which rows have one)."""
    z = s["logits"].float() / tau
    ids = s["ids"].long()
    live = ids >= 0
    z = z - z.amax(1, keepdim=True)
    mine = z.gather(1, ids.clamp(min=0).unsqueeze(1)).squeeze(1)
    e = z.exp()
    total = e.sum(1)
    return e, total, torch.where(live, mine - total.log(), 0.0), live


def _plain_grad(s, e, total, live, slope):
    """slope: d loss / d log-probability, over the temperature and times the loss scale."""
    slope = torch.where(live, slope, 0.0)
    grad = e * (-slope / total).unsqueeze(1)
    grad.scatter_add_(1, s["ids"].long().clamp(min=0).unsqueeze(1), slope.unsqueeze(1))
    return grad.to(s["logits"].dtype)


def _plain_policy(s):
    tau = s["temperature"]
    e, total, logp, live = _plain_tokens(s, tau)
    if s["only_logp"]:
        return {"logp": logp}
    a = s["advantage"]
    r = (logp - s["old_logp"]).exp() if s["old"] else torch.ones_like(logp)
    low, high = 1 - s["clip_low"], 1 + s["clip_high"]
    loss = -torch.minimum(r * a, r.clamp(low, high) * a)
    flat = ((a > 0) & (r > high)) | ((a < 0) & (r < low))
    slope = torch.where(flat, 0.0, -a * r)
    if s["ref"]:
        # in 64 bits: exp(d) - 1 - d of a small d
        d = s["ref_logp"].double() - logp.double()
        loss = loss + s["kl_weight"] * (torch.expm1(d) - d).float()
        slope = slope - s["kl_weight"] * torch.expm1(d).float()
    w = s["weight"]
    return {"logp": logp, "loss": torch.where(live, w * loss, 0.0),
            "grad": _plain_grad(s, e, total, live, w * slope * (s["scale"] / tau))}


def _plain_preference(s):
    e, total, logp, live = _plain_tokens(s, 1.0)
    pairs, beta = s["pairs"], s["beta"]
    at = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(s["starts"].long(), at, right=True) - 1
    # long sums, in 64 bits
    zero = torch.zeros(2 * pairs, dtype=torch.float64, device="cuda")
    q = zero.index_add(0, seq, logp.double())
    each = torch.ones_like(q)
    if s["mean"]:
        each = 1 / zero.index_add(0, seq, live.double()).clamp(min=1)
        q = q * each
    ratio = (q - s["ref_logp"].double()).view(pairs, 2)
    delta = ratio[:, 0] - ratio[:, 1]
    m = beta * delta
    if s["kind"] == "sigmoid":
        eps = s["smoothing"]
        small = torch.log1p(torch.exp(-m.abs()))
        loss = (1 - eps) * (small + (-m).clamp(min=0)) + eps * (small + m.clamp(min=0))
        slope = beta * (eps / (1 + torch.exp(-m)) - (1 - eps) / (1 + torch.exp(m)))
    elif s["kind"] == "hinge":
        loss = (1 - m).clamp(min=0)
        slope = torch.where(m < 1, -beta, 0.0)
    else:
        loss = (delta - 1 / (2 * beta)).square()
        slope = 2 * (delta - 1 / (2 * beta))
    w = s["weight"].double()
    sides = torch.stack([w * slope, -w * slope], 1).view(-1) * each * s["scale"]
    return {"loss": (w * loss).float(), "seq_logp": q.float(),
            "grad": _plain_grad(s, e, total, live, sides[seq].float())}


# ---- one pass ----------------------------------------------------------------

def _own(s):
    from sharded_mixed_precision_zs_amd import zeroshard as zs
    op = s["op"]
    if op == "dropout":
        zs.zs_dropout(s["x"], s["out"], (s["p"], s["seed"], s["offset"]), residual=s["res"])
        return {"out": s["out"]}
    if op == "block_norm":
        how = dict(post_gain=s["post_gain"], post_rstd=s["post_rstd"], gate=s["gate"],
                   residual_scale=s["residual_scale"], branch_scale=s["branch_scale"],
                   dropout=(s["p"], s["seed"], s["offset"]) if s["p"] else None)
        if s["backward"]:
            zs.zs_block_norm_backward(s["dy"], s["h"], s["rstd"], s["gain"], s["dx"],
                                      s["dresidual"], s["dgain"], s["workspace"], x=s["x"],
                                      dres=s["dres"], dpost_gain=s["dpost_gain"],
                                      dgate=s["dgate"], **how)
            return {k: s[k] for k in ("dresidual", "dgain", "dpost_gain", "dgate", "dx")
                    if s[k] is not None}
        wide = s["out"] == "16"
        zs.zs_block_norm_forward(s["x"], s["res"], s["gain"], EPS, s["h"], rstd=s["rstd"],
                                 codes=None if wide else s["codes"],
                                 scales=None if wide else s["scales"],
                                 y=s["y"] if wide else None, **how)
        out = {"post_rstd": s["post_rstd"]} if s["post"] else {}
        out.update(h=s["h"], rstd=s["rstd"])
        if wide:
            out.update(y=s["y"])
        else:
            out.update(y=s["codes"].view(torch.float8_e4m3fn),
                       scale=s["scales"].view(torch.float8_e8m0fnu))
        return out
    if op == "linear":
        act = {"none": zs.ZS_ACT_NONE, "relu": zs.ZS_ACT_RELU, "gelu": zs.ZS_ACT_GELU,
               "silu": zs.ZS_ACT_SILU}[s["act"]]
        if s["backward"]:
            zs.zs_activation_backward(s["dc"], s["saved"], act, s["dpre"], dbias=s["dbias"],
                                      workspace=s["workspace"])
            return {"dpre": s["dpre"], "dbias": s["dbias"]}
        fmt = zs.ZS_MX_E2M1 if s["a"] == "e2m1" else zs.ZS_MX_E4M3
        zs.zs_mx_linear(s["a_codes"], s["a_scales"], fmt, s["b_codes"], s["b_scales"], s["c"],
                        s["k"], bias=s["bias"], activation=act, residual=s["res"],
                        pre=s["pre_out"], workspace=s["workspace"])
        return {"c": s["c"], "pre": s["pre_out"]} if s["pre"] else {"c": s["c"]}
    if op == "policy":
        if s["only_logp"]:
            zs.zs_logprob(s["logits"], s["ids"], s["logp"], temperature=s["temperature"],
                          workspace=s["workspace"])
            return {"logp": s["logp"]}
        zs.zs_policy(s["logits"], s["ids"], s["advantage"], s["loss"],
                     temperature=s["temperature"], old_logp=s["old_logp"], ref_logp=s["ref_logp"],
                     clip_low=s["clip_low"], clip_high=s["clip_high"], kl_weight=s["kl_weight"],
                     row_weight=s["weight"], loss_scale=s["scale"], logp=s["logp"],
                     grad=s["grad"], workspace=s["workspace"])
        return {"logp": s["logp"], "loss": s["loss"], "grad": s["grad"]}
    kind = {"sigmoid": zs.ZS_PREFERENCE_SIGMOID, "hinge": zs.ZS_PREFERENCE_HINGE,
            "square": zs.ZS_PREFERENCE_SQUARE}[s["kind"]]
    zs.zs_preference(s["logits"], s["ids"], s["starts"], s["beta"], s["loss"], kind=kind,
                     smoothing=s["smoothing"], mean=s["mean"], ref_logp=s["ref_logp"],
                     pair_weight=s["weight"], loss_scale=s["scale"], seq_logp=s["seq_logp"],
                     grad=s["grad"], workspace=s["workspace"])
    return {"loss": s["loss"], "seq_logp": s["seq_logp"], "grad": s["grad"]}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "dropout":
        return _plain_dropout(state)
    if op == "block_norm":
        return _plain_block_grad(state) if state["backward"] else _plain_block(state)
    if op == "linear":
        return _plain_linear(state)
    return _plain_policy(state) if op == "policy" else _plain_preference(state)


# ---- work --------------------------------------------------------------------

def work(case):
    op = case["op"]
    size = SIZE[case["dtype"]]
    if op == "dropout":
        n = case["rows"] * case["cols"]
        return {"bytes": n * size * (3 if case["residual"] else 2), "flops": 2 * n}
    if op == "block_norm":
        t, d = case["rows"], case["cols"]
        vectors = 2 * d * (1 + case["post"] + case["gate"])
        if case["backward"]:
            x = case["post"] or case["gate"]
            return {"bytes": t * d * 2 * (4 + x + case["dres"]) + 4 * t * (1 + case["post"])
                    + vectors * 3, "flops": 16 * t * d}
        y = padded(d) * 33 // 32 if case["out"] == "e4m3" else 2 * d
        return {"bytes": t * (6 * d + y + 4 + 4 * case["post"]) + vectors, "flops": 12 * t * d}
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        if case["backward"]:
            return {"bytes": m * n * 2 * (3 if case["act"] != "none" else 2) + 4 * n,
                    "flops": 16 * m * n}
        scales = padded(k) // BLOCK
        return {"bytes": m * (_width(case["a"], k) + scales) + n * (_width("e2m1", k) + scales + 2)
                + m * n * 2 * (1 + case["residual"] + case["pre"]), "flops": 2 * m * n * k}
    t, v = case["rows"], case["vocab"]
    live = t - t // 8          # the other rows' logits need not be read
    if op == "policy":
        if case["only_logp"]:
            return {"bytes": live * v * size + 8 * t, "flops": 4 * live * v}
        return {"bytes": (live + t) * v * size + t * (16 + 4 * case["old"] + 4 * case["ref"]),
                "flops": 6 * live * v}
    return {"bytes": (live + t) * v * size + 4 * t + 24 * case["pairs"], "flops": 6 * live * v}


# ---- 64 bits -----------------------------------------------------------------

F64 = torch.float64


def _power(e):
    """2^e in float64 for whole e, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def _exact_e4m3(x):
    """(scales, element values) of a float64 matrix's rows, from the format's definition."""
    r, k = x.shape
    wide = torch.zeros(r, padded(k), dtype=F64, device=x.device)
    wide[:, :k] = x
    b = wide.reshape(r, -1, BLOCK)
    top = b.abs().max(2).values
    # floor(log2(top)) from the binary exponent; an empty block takes the lowest scale
    e = torch.frexp(top).exponent.to(torch.int64) - 1
    e = torch.where(top > 0, e - 8, torch.full_like(e, -126)).clamp(-126, 127)
    v = b * _power(-e).unsqueeze(2)
    step = _power((torch.frexp(v.abs()).exponent - 1).clamp(min=-6) - 3)
    q = torch.copysign((torch.round(v.abs() / step) * step).clamp(max=448), v)
    return _power(e), q.reshape(r, -1)


def _exact_unpacked(codes, scales, fmt, k):
    if fmt == "e4m3":
        q = codes.view(torch.float8_e4m3fn).to(F64)
    else:
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=F64, device=codes.device)
        table = torch.cat([table, -table])
        q = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=F64, device=codes.device)
        q[:, 0::2], q[:, 1::2] = table[(codes & 15).long()], table[(codes >> 4).long()]
    return (q * _power(scales.to(torch.int64) - 127).repeat_interleave(BLOCK, 1))[:, :k]


def _exact_factor(s):
    """Each element's factor, 0 or 1 / (1 - p), from the generator's definition on the host."""
    t, d = s["rows"], s["cols"]
    drop = _threshold(s["p"])
    if drop == 0:
        return torch.ones(t, d, dtype=F64, device="cuda")
    low, wide = np.uint64(0xFFFFFFFF), np.uint64(32)
    counter = [np.empty((t, -(-d // 8)), dtype=np.uint64) for _ in range(4)]
    counter[0][:] = np.arange(counter[0].shape[1], dtype=np.uint64)[None, :]
    counter[1][:] = np.arange(t, dtype=np.uint64)[:, None]
    counter[2][:] = np.uint64(s["offset"] % 2 ** 32)
    counter[3][:] = np.uint64(s["offset"] // 2 ** 32)
    for i in range(7):
        key = [np.uint64((s["seed"] % 2 ** 32 + i * 0x9E3779B9) % 2 ** 32),
               np.uint64((s["seed"] // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32)]
        a, b = counter[0] * np.uint64(0xD2511F53), counter[2] * np.uint64(0xCD9E8D57)
        counter = [(b >> wide) ^ counter[1] ^ key[0], b & low,
                   (a >> wide) ^ counter[3] ^ key[1], a & low]
    number = np.empty((t, counter[0].shape[1], 8), dtype=np.uint16)
    for j in range(8):
        number[:, :, j] = (counter[j // 2] >> np.uint64(16 * (j % 2))).astype(np.uint16)
    kept = torch.from_numpy(number.reshape(t, -1)[:, :d] >= drop).cuda()
    return kept.to(F64) * (65536.0 / (65536 - drop))


def _exact_tokens(s, tau):
    """Per row: softmax numerators' logsumexp and the token's log-probability."""
    lse, logp = [], []
    for first in range(0, s["rows"], 1024):          # some gigabytes at a time
        u = s["logits"][first:first + 1024].to(F64) / tau
        ids = s["ids"][first:first + 1024].long()
        lse.append(torch.logsumexp(u, 1))
        mine = u[torch.arange(u.shape[0], device="cuda"), ids.clamp(min=0)] - lse[-1]
        logp.append(torch.where(ids >= 0, mine, torch.zeros_like(mine)))
    return torch.cat(lse), torch.cat(logp)


def _exact_grad(s, tau, lse, slope):
    grad = torch.zeros(s["rows"], s["vocab"], dtype=F64, device="cuda")
    for first in range(0, s["rows"], 1024):
        part = slice(first, first + 1024)
        ids = s["ids"][part].long()
        k = torch.where(ids >= 0, slope[part], torch.zeros_like(slope[part]))
        g = grad[part]
        g.sub_(torch.softmax(s["logits"][part].to(F64) / tau, 1) * k.unsqueeze(1))
        g[torch.arange(g.shape[0], device="cuda"), ids.clamp(min=0)] += k
    return grad


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dropout":
        out = s["x"].to(F64) * _exact_factor(s)
        return {"out": out if s["res"] is None else out + s["res"].to(F64)}
    if op == "block_norm":
        x, gain = s["x"].to(F64), s["gain"].to(F64)
        post = s["post_gain"].to(F64) if case["post"] else torch.ones_like(gain)
        gate = s["gate"].to(F64) if case["gate"] else torch.ones_like(gain)
        factor = _exact_factor(s) * s["branch_scale"]
        if case["backward"]:
            h, dy, r2 = s["h"].to(F64), s["dy"].to(F64), s["rstd"].to(F64).unsqueeze(1)
            n2 = h * r2
            d2 = dy * gain
            dh = r2 * (d2 - n2 * torch.mean(d2 * n2, 1, keepdim=True))
            if s["dres"] is not None:
                dh = dh + s["dres"].to(F64)
            r1 = s["post_rstd"].to(F64).unsqueeze(1) if case["post"] else 1.0
            n1 = x * r1
            du = dh * factor
            dn = du * gate * post
            dx = r1 * (dn - n1 * torch.mean(dn * n1, 1, keepdim=True)) if case["post"] else dn
            out = {"dresidual": dh * s["residual_scale"], "dgain": torch.sum(dy * n2, 0)}
            if case["post"]:
                out["dpost_gain"] = torch.sum(du * gate * n1, 0)
            if case["gate"]:
                out["dgate"] = torch.sum(du * n1 * post, 0)
            return dict(out, dx=dx)
        out = {}
        if case["post"]:
            rms = torch.sqrt(torch.mean(x * x, 1) + EPS)
            out["post_rstd"] = 1 / rms
            x = x / rms.unsqueeze(1) * post
        h = (s["res"].to(F64) * s["residual_scale"] + x * gate * factor)
        out["h"] = h
        # to the nearest of 8 or 11 significant bits, ties to even
        step = _power((torch.frexp(h).exponent - (8 if case["dtype"] == "bf16" else 11)).clamp(
            min=-133 if case["dtype"] == "bf16" else -24))
        h = torch.round(h / step) * step
        rms = torch.sqrt(torch.mean(h * h, 1) + EPS)
        out["rstd"] = 1 / rms
        y = h / rms.unsqueeze(1) * gain
        if case["out"] != "e4m3":
            return dict(out, y=y)
        scale, q = _exact_e4m3(y)
        return dict(out, y=q, scale=scale)
    if op == "linear":
        act = case["act"]
        if case["backward"]:
            x = s["saved"].to(F64).requires_grad_(True)
        else:
            a = _exact_unpacked(s["a_codes"], s["a_scales"], case["a"], case["k"])
            b = _exact_unpacked(s["b_codes"], s["b_scales"], "e2m1", case["k"])
            x = a @ b.t() + s["bias"].to(F64)
        if act == "relu":
            c = torch.relu(x)
        elif act == "gelu":
            c = torch.nn.functional.gelu(x, approximate="tanh")
        elif act == "silu":
            c = x * torch.sigmoid(x)
        else:
            c = x * 1.0
        if case["backward"]:
            dpre, = torch.autograd.grad(c, x, s["dc"].to(F64))
            return {"dpre": dpre, "dbias": dpre.sum(0)}
        if s["res"] is not None:
            c = c + s["res"].to(F64)
        return {"c": c, "pre": x} if case["pre"] else {"c": c}
    tau = float(case.get("temperature", 1.0))
    lse, logp = _exact_tokens(s, tau)
    if op == "policy":
        if case["only_logp"]:
            return {"logp": logp}
        a, w = s["advantage"].to(F64), s["weight"].to(F64)
        v = logp.clone().requires_grad_(True)
        ratio = torch.exp(v - (s["old_logp"].to(F64) if case["old"] else logp))
        clipped = torch.clamp(ratio, 1 - s["clip_low"], 1 + s["clip_high"])
        loss = -torch.minimum(ratio * a, clipped * a)
        if case["ref"]:
            d = s["ref_logp"].to(F64) - v
            loss = loss + s["kl_weight"] * (torch.expm1(d) - d)
        loss = w * loss
        slope, = torch.autograd.grad(loss.sum(), v)
        return {"logp": logp, "loss": torch.where(s["ids"] >= 0, loss.detach(), 0.0),
                "grad": _exact_grad(s, tau, lse, slope * (s["scale"] / tau))}
    starts = s["starts"].tolist()
    v = logp.clone().requires_grad_(True)
    there = (s["ids"] >= 0).to(F64)
    q = []
    for first, last in zip(starts, starts[1:]):
        q.append(v[first:last].sum() / (there[first:last].sum().clamp(min=1) if case["mean"] else 1))
    q = torch.stack(q)
    ratio = q - s["ref_logp"].to(F64)
    delta = ratio[0::2] - ratio[1::2]
    m = s["beta"] * delta
    if case["kind"] == "sigmoid":
        logs = torch.nn.functional.logsigmoid
        loss = -(1 - s["smoothing"]) * logs(m) - s["smoothing"] * logs(-m)
    elif case["kind"] == "hinge":
        loss = torch.relu(1 - m)
    else:
        loss = (delta - 1 / (2 * s["beta"])) ** 2
    loss = s["weight"].to(F64) * loss
    slope, = torch.autograd.grad(loss.sum(), v)
    return {"loss": loss.detach(), "seq_logp": q.detach(),
            "grad": _exact_grad(s, tau, lse, slope * s["scale"])}
