"""The operators of a low-precision student's output end, as they are measured.

Each case is one call that a training or serving program makes:

  norm      root-mean-square norm with the residual's addition and an 8-bit
            microscaled output (forward), and its gradient (backward)
  quantize  microscaled 4- or 8-bit copy of a matrix, along rows or columns
  product   C = A B^T of microscaled operands (A in 8 or 4 bits, B in 4), or
            "linear": 16-bit activations quantised and multiplied in one go
  distill   loss and logits' gradient against a teacher's top logits

Microscaled rows are padded with zeros to whole groups of 128 elements;
32 elements share a power-of-two scale held as an E8M0 byte.
"""
import math

import torch

own = False

BLOCK = 32
GROUP = 128
EMAX = {"e2m1": 2, "e4m3": 8}
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def padded(k):
    return -(-k // GROUP) * GROUP


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # one decoded token of the GPT-2-small-shaped model: latency
        {"name": "norm-token", "op": "norm", "rows": 1, "cols": 768, "dtype": "bf16",
         "backward": False, "residual": True},
        # a training micro-batch of a 7B-sized model's width
        {"name": "norm-batch", "op": "norm", "rows": 16384, "cols": 4096, "dtype": "bf16",
         "backward": False, "residual": True},
        # a ragged batch in fp16, backward, no gradient from the residual stream
        {"name": "norm-grad-ragged", "op": "norm", "rows": 1003, "cols": 1600, "dtype": "fp16",
         "backward": True, "residual": False},
        # the training micro-batch, backward
        {"name": "norm-grad-batch", "op": "norm", "rows": 16384, "cols": 4096, "dtype": "bf16",
         "backward": True, "residual": True},
        # the fp32 master copy of a GPT-2-small-shaped head to 4 bits after an optimizer step
        {"name": "quantize-master", "op": "quantize", "rows": 50257, "cols": 768, "dtype": "fp32",
         "format": "e2m1", "columns": False},
        # gradients of a micro-batch along the tokens, for the weights' gradient
        {"name": "quantize-columns", "op": "quantize", "rows": 8191, "cols": 4096,
         "dtype": "bf16", "format": "e4m3", "columns": True},
        # one decoded token through a 4-bit head, 8-bit activations
        {"name": "product-token", "op": "product", "m": 1, "n": 32000, "k": 4096, "a": "e4m3",
         "out": "bf16", "linear": False},
        # a short ragged prompt through the GPT-2-small-shaped head, 4-bit activations
        {"name": "product-prompt", "op": "product", "m": 77, "n": 50257, "k": 768, "a": "e2m1",
         "out": "fp16", "linear": False},
        # a training micro-batch through one square layer, 8-bit activations
        {"name": "product-batch", "op": "product", "m": 8192, "n": 4096, "k": 4096, "a": "e4m3",
         "out": "bf16", "linear": False},
        # the largest: activations quantised to 4 bits and multiplied
        {"name": "linear-batch", "op": "product", "m": 8192, "n": 8192, "k": 8192, "a": "e2m1",
         "out": "bf16", "linear": True},
        # a few rows of GPT-2-small-shaped logits, the teacher's tail mass known
        {"name": "distill-few", "op": "distill", "rows": 13, "vocab": 50257, "slots": 32,
         "dtype": "fp16", "tail": True, "temperature": 2.0},
        # a training micro-batch over a large vocabulary
        {"name": "distill-batch", "op": "distill", "rows": 8192, "vocab": 128000, "slots": 64,
         "dtype": "bf16", "tail": False, "temperature": 1.0},
    ]


def _between(rng, lo, hi):
    """A whole number spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quantize", "product", "product", "distill", "distill"])
    if op == "norm":
        cols = _between(rng, 64, 8192)
        rows = _between(rng, 1, min(16384, (16384 * 4096) // cols))
        return {"op": op, "rows": rows, "cols": cols if rng.random() < 0.4 else -(-cols // 32) * 32,
                "dtype": rng.choice(["bf16", "fp16"]), "backward": rng.random() < 0.5,
                "residual": rng.random() < 0.7}
    if op == "quantize":
        cols = _between(rng, 33, 16384)
        rows = _between(rng, 1, min(50257, (50257 * 768) // cols))
        return {"op": op, "rows": rows, "cols": cols if rng.random() < 0.4 else -(-cols // 32) * 32,
                "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "format": rng.choice(["e2m1", "e4m3"]), "columns": rng.random() < 0.5}
    if op == "product":
        m = _between(rng, 1, 8192)
        n = _between(rng, 64, 50257)
        k = _between(rng, 64, 8192)
        while m * n * k > 8192 ** 3 // 4:
            n = max(64, n // 2)
        a = rng.choice(["e2m1", "e4m3"])
        # 32-bit results are for 4-bit operands, whose sums are exact in 32 bits
        return {"op": op, "m": m, "n": n, "k": k, "a": a,
                "out": rng.choice(["bf16", "fp16"] + ["fp32"] * (a == "e2m1")),
                "linear": rng.random() < 0.3}
    vocab = _between(rng, 1000, 200000)
    rows = _between(rng, 1, min(8192, (8192 * 100000) // vocab))
    return {"op": op, "rows": rows, "vocab": vocab, "slots": _between(rng, 1, 128),
            "dtype": rng.choice(["bf16", "fp16", "fp32"]) if rows * vocab < 1 << 28 else "bf16",
            "tail": rng.random() < 0.5, "temperature": rng.choice([1.0, 2.0, 0.7])}


# ---- inputs ------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


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


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    if op == "norm":
        t, d, dt = case["rows"], case["cols"], DTYPE[case["dtype"]]
        s["eps"] = 1e-5
        s["gain"] = (1 + 0.1 * _randn(g, d)).to(dt)
        if case["backward"]:
            s["h"] = (_randn(g, t, d) * (0.5 + 2 * torch.rand(t, 1, generator=g, device="cuda"))
                      ).to(dt)
            s["rstd"] = (s["h"].float().square().mean(1) + s["eps"]).rsqrt()
            s["dy"] = (_randn(g, t, d) * 0.05).to(dt)
            s["dres"] = (_randn(g, t, d) * 0.05).to(dt) if case["residual"] else None
            s["dx"] = torch.empty(t, d, dtype=dt, device="cuda")
            s["dgain"] = torch.empty(d, device="cuda")
            # room for the partial sums of the gain's gradient
            s["workspace"] = _bytes(1024 * d * 4)
        else:
            s["x"] = _randn(g, t, d).to(dt)
            s["res"] = (_randn(g, t, d) * 2).to(dt) if case["residual"] else None
            s["h"] = torch.empty(t, d, dtype=dt, device="cuda")
            s["rstd"] = torch.empty(t, device="cuda")
            s["codes"] = _bytes(t, padded(d))
            s["scales"] = _bytes(t, padded(d) // BLOCK)
    elif op == "quantize":
        r, c, dt = case["rows"], case["cols"], DTYPE[case["dtype"]]
        # rows of different sizes, as weights and gradients have
        s["src"] = (_randn(g, r, c) * 0.02 * torch.exp(_randn(g, r, 1))).to(dt)
        ro, k = (c, r) if case["columns"] else (r, c)
        s["codes"] = _bytes(ro, _width(case["format"], k))
        s["scales"] = _bytes(ro, padded(k) // BLOCK)
        s["values"] = torch.empty(r, c, dtype=torch.bfloat16, device="cuda")
    elif op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        x = _randn(g, m, k)
        if case["linear"]:
            s["x"] = x.to(torch.bfloat16)
            s["a_codes"], s["a_scales"] = _bytes(m, _width(case["a"], k)), _bytes(m, padded(k) // BLOCK)
        else:
            s["a_codes"], s["a_scales"] = _packed(x, case["a"])
        s["b_codes"], s["b_scales"] = _packed(_randn(g, n, k) * 0.02, "e2m1")
        s["c"] = torch.empty(m, n, dtype=DTYPE[case["out"]], device="cuda")
        # room for the partial sums of a product split along k
        s["workspace"] = _bytes(32 << 20)
    else:
        t, v, k, dt = case["rows"], case["vocab"], case["slots"], DTYPE[case["dtype"]]
        z = torch.randn(t, v, generator=g, device="cuda", dtype=torch.bfloat16 if dt == torch.bfloat16
                        else torch.float32)
        z *= 2
        # distinct tokens in ascending gaps, as far apart as the vocabulary lets them be
        gaps = torch.randint(1, max(2, v // k), (t, k), generator=g, device="cuda")
        ids = (gaps.cumsum(1) + torch.randint(0, v, (t, 1), generator=g, device="cuda")) % v
        teacher = (_randn(g, t, k) * 2 + 6).sort(1, descending=True).values
        # the student has learnt some of the teacher's choice
        z.scatter_add_(1, ids, (teacher - 2 + _randn(g, t, k)).to(z.dtype))
        s["logits"] = z.to(dt)
        # some rows have fewer slots than others (empty ones are -1), one has none
        have = torch.randint(max(1, k // 2), k + 1, (t, 1), generator=g, device="cuda")
        have[t // 2] = have[t // 2] * 0 if t > 4 else have[t // 2]
        s["ids"] = torch.where(torch.arange(k, device="cuda") < have, ids, -1).to(torch.int32)
        s["teacher"] = teacher.to(dt)
        # the teacher's logsumexp over its whole vocabulary: some mass lies off its top logits
        kept = s["teacher"].float() / case["temperature"]
        s["lse"] = kept.logsumexp(1) + 0.3 * torch.rand(t, generator=g, device="cuda") \
            if case["tail"] else None
        # prompt tokens carry no loss
        s["weight"] = (torch.rand(t, generator=g, device="cuda") > 0.1).float() / t
        s["scale"] = 65536.0 if dt != torch.float16 else 1024.0
        s["loss"] = torch.empty(t, device="cuda")
        s["grad"] = torch.empty_like(s["logits"])
        # room for the partial statistics of rows that several workgroups share
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


def _values(byte, q):
    scale = (byte.to(torch.int32) << 23).view(torch.float32)
    return (q.view(q.shape[0], -1, BLOCK) * scale.unsqueeze(2)).view(q.shape)


def _unpacked(codes, scales, fmt):
    if fmt == "e4m3":
        q = codes.view(torch.float8_e4m3fn).float()
    else:
        code = torch.stack([codes & 15, codes >> 4], 2).view(codes.shape[0], -1)
        low = (code & 7).float()
        mag = torch.where(low < 4, low / 2, torch.where(low < 6, low - 2, low * 2 - 8))
        q = torch.where(code > 7, -mag, mag)
    return _values(scales, q)


def _plain_norm(s):
    h = s["x"].float()
    if s["res"] is not None:
        h = (h + s["res"].float()).to(s["x"].dtype).float()
    rstd = (h.square().mean(1) + s["eps"]).rsqrt()
    y = h * rstd.unsqueeze(1) * s["gain"].float()
    byte, q = _quantized(_pad(y), "e4m3")
    return {"h": h.to(s["x"].dtype), "rstd": rstd, "y": q.to(torch.float8_e4m3fn),
            "scale": byte.view(torch.float8_e8m0fnu)}


def _plain_norm_grad(s):
    h, rstd = s["h"].float(), s["rstd"].unsqueeze(1)
    dy = s["dy"].float()
    gdy = dy * s["gain"].float()
    dx = rstd * (gdy - h * rstd.square() * (gdy * h).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["h"].dtype), "dgain": (dy * h * rstd).sum(0)}


def _plain_quantize(s):
    x = s["src"].float()
    r, c = x.shape
    x = x.t().contiguous() if s["columns"] else x
    byte, q = _quantized(_pad(x), s["format"])
    v = _values(byte, q)[:, : r if s["columns"] else c]
    return {"values": (v.t() if s["columns"] else v).to(torch.bfloat16).contiguous(),
            "scale": byte.view(torch.float8_e8m0fnu)}


def _plain_product(s):
    if s["linear"]:
        a = _values(*_quantized(_pad(s["x"].float()), s["a"]))
    else:
        a = _unpacked(s["a_codes"], s["a_scales"], s["a"])
    b = _unpacked(s["b_codes"], s["b_scales"], "e2m1")
    return {"c": torch.matmul(a, b.t()).to(s["c"].dtype)}


def _plain_distill(s):
    z, tau = s["logits"].float() / s["temperature"], s["temperature"]
    valid = s["ids"] >= 0
    ids = s["ids"].clamp(min=0).long()
    t = (s["teacher"].float() / tau).masked_fill(~valid, -math.inf)
    top = t.amax(1, keepdim=True).clamp(min=-1e30)
    lse = s["lse"].unsqueeze(1) if s["tail"] else \
        ((t - top).exp().sum(1, keepdim=True).log() + top).clamp(min=-1e30)
    logp = t - lse
    p = logp.exp()
    m = z.amax(1, keepdim=True)
    e = (z - m).exp()
    total = e.sum(1, keepdim=True)
    zk = z.gather(1, ids)
    logq = zk - m - total.log()
    kl = torch.where(p > 0, p * (logp - logq), 0.0).sum(1, keepdim=True)
    off = torch.ones_like(kl)
    if s["tail"]:
        # student's mass off the slots, summed without them
        rest = e.scatter(1, torch.where(valid, ids, ids[:, :1]), 0.0).sum(1, keepdim=True) / total
        pr = (1 - p.sum(1, keepdim=True)).clamp(min=0)
        kl = kl + torch.where(pr > 0, pr * (pr.log() - rest.log()), 0.0)
        off = 1 - pr / rest
    grad = e * (off / total)
    # on the slots: q - p in place of the share that the others have
    on = torch.where(valid, logq.exp() * (1 - off) - p, 0.0)
    grad.scatter_add_(1, ids, on)
    some = valid.any(1, keepdim=True)
    w = s["weight"].unsqueeze(1)
    live = some & (w != 0)
    loss = torch.where(live, w * tau * tau * kl, 0.0).squeeze(1)
    grad = torch.where(live, grad * (s["scale"] * tau * w), 0.0)
    return {"loss": loss, "grad": grad.to(s["logits"].dtype)}


# ---- one pass ----------------------------------------------------------------

def _own(s):
    from sharded_mixed_precision_zs_amd import zeroshard as zs
    op = s["op"]
    if op == "norm" and s["backward"]:
        zs.zs_rmsnorm_backward(s["dy"], s["h"], s["rstd"], s["gain"], s["dx"], s["dgain"],
                               s["workspace"], dres=s["dres"])
        return {"dx": s["dx"], "dgain": s["dgain"]}
    if op == "norm":
        zs.zs_rmsnorm_forward(s["x"], s["gain"], s["eps"], s["h"], s["rstd"], residual=s["res"],
                              codes=s["codes"], scales=s["scales"])
        return {"h": s["h"], "rstd": s["rstd"], "y": s["codes"].view(torch.float8_e4m3fn),
                "scale": s["scales"].view(torch.float8_e8m0fnu)}
    formats = {"e2m1": zs.ZS_MX_E2M1, "e4m3": zs.ZS_MX_E4M3}
    if op == "quantize":
        zs.zs_mx_quantize(s["src"], formats[s["format"]], s["codes"], s["scales"],
                          columns=s["columns"], values=s["values"])
        return {"values": s["values"], "scale": s["scales"].view(torch.float8_e8m0fnu)}
    if op == "product":
        if s["linear"]:
            zs.zs_mx_quantize(s["x"], formats[s["a"]], s["a_codes"], s["a_scales"])
        zs.zs_mx_matmul(s["a_codes"], s["a_scales"], formats[s["a"]], s["b_codes"], s["b_scales"],
                        s["c"], s["k"], workspace=s["workspace"])
        return {"c": s["c"]}
    zs.zs_distill(s["logits"], s["ids"], s["teacher"], s["temperature"], s["loss"],
                  grad=s["grad"], teacher_lse=s["lse"], row_weight=s["weight"],
                  loss_scale=s["scale"], workspace=s["workspace"])
    return {"loss": s["loss"], "grad": s["grad"]}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "norm":
        return _plain_norm_grad(state) if state["backward"] else _plain_norm(state)
    if op == "quantize":
        return _plain_quantize(state)
    if op == "product":
        return _plain_product(state)
    return _plain_distill(state)


# ---- work --------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "norm":
        t, d = case["rows"], case["cols"]
        if case["backward"]:
            return {"bytes": t * d * 2 * (4 if case["residual"] else 3) + 4 * t + 6 * d,
                    "flops": 9 * t * d}
        return {"bytes": t * d * 2 * (3 if case["residual"] else 2) + t * padded(d) * 33 // 32
                + 4 * t + 2 * d, "flops": 7 * t * d}
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        ro, k = (c, r) if case["columns"] else (r, c)
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": r * c * (size + 2) + ro * (_width(case["format"], k) + padded(k) // BLOCK),
                "flops": 3 * r * c}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        scales = padded(k) // BLOCK
        a = m * k * 2 if case["linear"] else m * (_width(case["a"], k) + scales)
        return {"bytes": a + n * (_width("e2m1", k) + scales) + m * n * (4 if case["out"] == "fp32" else 2),
                "flops": 2 * m * n * k}
    t, v, k = case["rows"], case["vocab"], case["slots"]
    size = 4 if case["dtype"] == "fp32" else 2
    return {"bytes": 2 * t * v * size + t * k * (4 + size) + t * 12, "flops": 6 * t * v}


# ---- 64 bits -----------------------------------------------------------------

def _power(e):
    """2^e in float64 for whole e, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_quantized(x, fmt):
    """(scale bytes, values) of a float64 matrix along its rows, from the format's definition."""
    r, k = x.shape
    wide = torch.zeros(r, padded(k), dtype=torch.float64, device=x.device)
    wide[:, :k] = x
    b = wide.reshape(r, -1, BLOCK)
    top = b.abs().max(2).values
    # floor(log2(top)) from the binary exponent; an empty block takes the lowest scale
    e = torch.frexp(top).exponent.to(torch.int64) - 1
    e = torch.where(top > 0, e - EMAX[fmt], torch.full_like(e, -126)).clamp(-126, 127)
    v = b * _power(-e).unsqueeze(2)
    mag = v.abs()
    if fmt == "e2m1":
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
        lo = torch.searchsorted(grid, mag.contiguous(), right=True) - 1
        hi = (lo + 1).clamp(max=7)
        mid = (grid[lo] + grid[hi]) / 2
        up = (mag > mid) | ((mag == mid) & (lo % 2 == 1))
        q = torch.where(up, grid[hi], grid[lo])
    else:
        step = _power((torch.frexp(mag).exponent - 1).clamp(min=-6) - 3)
        q = (torch.round(mag / step) * step).clamp(max=448)
    q = torch.copysign(q, v)
    val = q * _power(e).unsqueeze(2)
    return (_power(e), q.reshape(r, -1), val.reshape(r, -1)[:, :k])


def _exact_unpacked(codes, scales, fmt):
    if fmt == "e4m3":
        q = codes.view(torch.float8_e4m3fn).to(torch.float64)
    else:
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=codes.device)
        table = torch.cat([table, -table])
        q = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
        q[:, 0::2], q[:, 1::2] = table[(codes & 15).long()], table[(codes >> 4).long()]
    return q * _power(scales.to(torch.int64) - 127).repeat_interleave(BLOCK, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "norm" and case["backward"]:
        h, dy, gain = s["h"].to(f64), s["dy"].to(f64), s["gain"].to(f64)
        n = h * s["rstd"].to(f64).unsqueeze(1)          # the normalised rows
        dn = dy * gain
        dx = s["rstd"].to(f64).unsqueeze(1) * (dn - n * torch.mean(dn * n, 1, keepdim=True))
        if s["dres"] is not None:
            dx += s["dres"].to(f64)
        return {"dx": dx, "dgain": torch.sum(dy * n, 0)}
    if op == "norm":
        h = s["x"].to(f64)
        if s["res"] is not None:
            h = (h + s["res"].to(f64)).to(s["x"].dtype).to(f64)
        rms = torch.sqrt(torch.mean(h * h, 1) + s["eps"])
        scale, q, _ = _exact_quantized(h / rms.unsqueeze(1) * s["gain"].to(f64), "e4m3")
        return {"h": h, "rstd": 1 / rms, "y": q, "scale": scale}
    if op == "quantize":
        x = s["src"].to(f64)
        scale, _, v = _exact_quantized(x.t() if case["columns"] else x, case["format"])
        return {"values": v.t().contiguous() if case["columns"] else v, "scale": scale}
    if op == "product":
        if case["linear"]:
            a = _exact_quantized(s["x"].to(f64), case["a"])[2]
        else:
            a = _exact_unpacked(s["a_codes"], s["a_scales"], case["a"])[:, :case["k"]]
        b = _exact_unpacked(s["b_codes"], s["b_scales"], "e2m1")[:, :case["k"]]
        return {"c": a @ b.t()}
    tau = float(case["temperature"])
    loss = torch.zeros(case["rows"], dtype=f64, device="cuda")
    grad = torch.zeros(case["rows"], case["vocab"], dtype=f64, device="cuda")
    for first in range(0, case["rows"], 1024):          # some gigabytes at a time
        part = slice(first, first + 1024)
        u = s["logits"][part].to(f64) / tau
        ids, w = s["ids"][part].to(torch.int64), s["weight"][part].to(f64)
        row, slot = torch.nonzero(ids >= 0, as_tuple=True)
        target = torch.full_like(u, 0.0)
        t = torch.full(ids.shape, -math.inf, dtype=f64, device="cuda")
        t[row, slot] = s["teacher"][part].to(f64)[row, slot] / tau
        some = (ids >= 0).any(1)
        if case["tail"]:
            logp = t - s["lse"][part].to(f64).unsqueeze(1)
        else:
            logp = t - torch.where(some, torch.logsumexp(t, 1), 0.0).unsqueeze(1)
        logq = u - torch.logsumexp(u, 1, keepdim=True)
        q = logq.exp()
        target[row, ids[row, slot]] = logp[row, slot].exp()
        kl = torch.zeros(u.shape[0], dtype=f64, device="cuda")
        kl.index_add_(0, row, logp[row, slot].exp() * (logp[row, slot] - logq[row, ids[row, slot]]))
        d = q - target
        if case["tail"]:
            away = torch.ones_like(u)
            away[row, ids[row, slot]] = 0.0
            qr = torch.sum(q * away, 1)
            pr = torch.clamp(1 - target.sum(1), min=0.0)
            kl += torch.where(pr > 0, pr * torch.log(torch.where(pr > 0, pr, 1.0) / qr), 0.0)
            d = torch.where(away > 0, q * (1 - (pr / qr).unsqueeze(1)), d)
        keep = (some & (w != 0)).to(f64)
        loss[part] = keep * w * tau * tau * kl
        grad[part] = (keep * w * (s["scale"] * tau)).unsqueeze(1) * d
    return {"loss": loss, "grad": grad}
