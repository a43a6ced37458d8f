"""The last block's operators on the GPU against their 64-bit plain forms.

Tolerances, fixed before the first run. A rounding to a type t is off by at
most half a step, relative eps(t)/2 (U below), or half its smallest
subnormal. An fp32 sum of n magnitudes adding up to M is off by at most
n * 2^-24 * M, n the length of its longest chain of additions.
"""
import math
import zlib

import pytest
import torch

import block_reference as ref
import ops_reference as ops
from gpu_util import announce

pytestmark = pytest.mark.gpu
BF16, FP16, FP32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
U = {t: torch.finfo(t).eps / 2 for t in (BF16, FP16, FP32)}
TINY = {BF16: 2.0 ** -134, FP16: 2.0 ** -25, FP32: 2.0 ** -126}
SENTINEL = 0xA5
SEED, OFFSET = 0x0123456789ABCDEF, (5 << 32) + 9


@pytest.fixture(scope="module")
def zs(hip_built):
    from sharded_mixed_precision_zs_amd import zeroshard
    return zeroshard


def gen(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def randn(g, *shape):
    return torch.randn(*shape, generator=g, dtype=FP32)


def guarded(shape, dtype, pad=64):
    """A tensor between two stretches of a known byte, and a check that they are whole."""
    n = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
    raw = torch.full((n + 2 * pad,), SENTINEL, dtype=torch.uint8, device="cuda")

    def whole():
        return bool((raw[:pad] == SENTINEL).all()) and bool((raw[pad + n:] == SENTINEL).all())

    return raw[pad:pad + n].view(dtype).view(shape), whole


def close(got, want, tol, what):
    got, want = got.double().cpu(), want.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN positions differ"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    ok = ~inf & ~torch.isnan(want)
    err, tol = (got - want).abs()[ok], torch.as_tensor(tol, dtype=F64).expand(want.shape)[ok]
    bad = err > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {err.numel()} off; worst "
                           f"{float((err / tol.clamp(min=1e-300)).max()):.3g} times the tolerance")


def cu(t):
    return None if t is None else t.cuda()


def dbl(t):
    return None if t is None else t.double()


# ---- dropout -------------------------------------------------------------------

DROPOUT = [(1, 1), (1, 8), (3, 7), (5, 33), (2, 768), (17, 100), (70, 9), (1, 4099)]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=str)
@pytest.mark.parametrize("p", [0.0, 0.1, 0.75, 1.0])
def test_dropout_against_64_bits(zs, dtype, p):
    for r, c in DROPOUT:
        announce(f"dropout {dtype} p={p} {r}x{c}")
        g = gen("d", r, c)
        x, res = randn(g, r, c).to(dtype), (2 * randn(g, r, c)).to(dtype)
        f = ref.keep_factor(r, c, p, SEED, OFFSET)
        for with_res in (False, True):
            out, whole = guarded((r, c), dtype)
            zs.zs_dropout(x.cuda(), out, (p, SEED, OFFSET), residual=res.cuda() if with_res else None)
            want = ref.dropped(x.double(), f) + (res.double() if with_res else 0)
            # factor, product and sum in fp32, then the type's own rounding
            inner = 2.0 ** -24 * (2 * (x.double() * f).abs() + want.abs())
            close(out, want, U[dtype] * (want.abs() + inner) + inner + TINY[dtype], f"{r}x{c}")
            assert whole()
            if not with_res:
                assert torch.equal(out.cpu() == 0, (f == 0) | (x == 0))


def test_dropout_mask_goes_with_place_seed_and_offset(zs):
    x = torch.ones(64, 200, device="cuda")
    draw = lambda rows, seed, offset, **k: zs.zs_dropout(x[:rows], out[:rows], (0.5, seed, offset), **k)
    out = torch.empty_like(x)
    draw(64, SEED, OFFSET)
    whole = out.clone()
    draw(20, SEED, OFFSET)
    assert torch.equal(out[:20], whole[:20])
    for seed, offset in ((SEED + 1, OFFSET), (SEED ^ 1 << 40, OFFSET), (SEED, OFFSET + 1),
                         (SEED, OFFSET + (1 << 32))):
        draw(64, seed, offset)
        # two independent masks of 12800 elements agree on half of them, give or take five
        # standard deviations of 56.6
        assert abs(int((out == whole).sum()) - 6400) < 284


def test_dropout_in_place_and_masked_values_gone(zs):
    g = gen("inplace")
    x = randn(g, 33, 130).to(BF16)
    f = ref.keep_factor(33, 130, 0.4, SEED, OFFSET)
    x[f == 0] = torch.tensor([math.nan, math.inf, -math.inf]).to(BF16).repeat(
        int((f == 0).sum()))[:int((f == 0).sum())]
    d, res = x.cuda(), torch.full((33, 130), 3.0, dtype=BF16).cuda()
    zs.zs_dropout(d, res, (0.4, SEED, OFFSET), residual=res)
    assert torch.isfinite(res.float()).all() and bool((res.cpu()[f == 0] == 3).all())
    want = torch.empty_like(d)
    zs.zs_dropout(d, want, (0.4, SEED, OFFSET))
    zs.zs_dropout(d, d, (0.4, SEED, OFFSET))
    assert torch.equal(d, want) and bool((d.cpu()[f == 0] == 0).all())


def test_dropout_unaligned_rows(zs):
    base = randn(gen("ua"), 1, 6001).to(FP16)
    for off, r, c in ((1, 7, 100), (3, 5, 64), (8, 9, 128)):
        announce(f"dropout unaligned {off}")
        n = r * c
        x = base[0, off:off + n].view(r, c)
        raw = torch.zeros(off + n + 8, dtype=FP16, device="cuda")
        out = raw[off:off + n].view(r, c)
        zs.zs_dropout(base.cuda()[0, off:off + n].view(r, c), out, (0.1, SEED, OFFSET))
        f = ref.keep_factor(r, c, 0.1, SEED, OFFSET)
        inner = 2.0 ** -23 * (x.double() * f).abs()
        close(out, x.double() * f, U[FP16] * (x.double() * f).abs() * (1 + 2.0 ** -20) + inner
              + TINY[FP16], "unaligned")
        assert not bool(raw[:off].any()) and not bool(raw[off + n:].any())


def test_dropout_offset_on_the_device_in_a_graph(zs):
    """Replays draw anew; each matches the eager call with the same sum of offsets."""
    x = torch.randn(50, 96, device="cuda").to(BF16)
    out, step = torch.empty_like(x), torch.zeros(1, dtype=torch.int64, device="cuda")
    zs.zs_dropout(x, out, (0.5, SEED, OFFSET, step))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        zs.zs_dropout(x, out, (0.5, SEED, OFFSET, step))
        step += 1
    seen = []
    for i in range(3):
        graph.replay()
        want = torch.empty_like(x)
        zs.zs_dropout(x, want, (0.5, SEED, OFFSET + i))
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        seen.append(out.clone())
    assert not torch.equal(seen[0], seen[1])


# ---- the block's end -----------------------------------------------------------

BLOCK = [(1, 1), (2, 7), (3, 32), (5, 100), (1, 768), (9, 520), (7, 1000), (3, 1600), (2, 2047),
         (5, 4096), (2, 4099), (2, 8200), (1, 20000)]


def problem(r, c, dtype, post, gate, p):
    g = gen("b", r, c)
    v = dict(x=(randn(g, r, c) * (0.2 + torch.rand(r, 1, generator=g))).to(dtype),
             res=(2 * randn(g, r, c)).to(dtype), gain=(1 + 0.1 * randn(g, c)).to(dtype),
             post_gain=(1 + 0.1 * randn(g, c)).to(dtype) if post else None,
             gate=(0.3 + 0.2 * randn(g, c)).to(dtype) if gate else None)
    # one mask for all of a shape's variants: the pure Python generator is slow
    return v, ref.keep_factor(r, c, p, SEED, OFFSET)


def run_forward(zs, v, dtype, p, eps=1e-5, rs=0.875, bs=0.55):
    r, c = v["x"].shape
    h, ok_h = guarded((r, c), dtype)
    y, ok_y = guarded((r, c), dtype)
    cs, ss = zs.mx_shapes(r, c, zs.ZS_MX_E4M3)
    codes, ok_c = guarded(cs, torch.uint8)
    scales, ok_s = guarded(ss, torch.uint8)
    rstd = torch.empty(r, device="cuda")
    post_rstd = torch.empty(r, device="cuda") if v["post_gain"] is not None else None
    zs.zs_block_norm_forward(cu(v["x"]), cu(v["res"]), cu(v["gain"]), eps, h, rstd=rstd,
                             post_gain=cu(v["post_gain"]), post_rstd=post_rstd, gate=cu(v["gate"]),
                             residual_scale=rs, branch_scale=bs,
                             dropout=(p, SEED, OFFSET) if p else None, codes=codes, scales=scales,
                             y=y)
    assert ok_h() and ok_y() and ok_c() and ok_s()
    return h, post_rstd, rstd, y, codes, scales


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=str)
@pytest.mark.parametrize("post,gate,p", [(True, True, 0.25), (True, False, 0.0), (False, True, 0.0),
                                         (False, False, 0.25)])
def test_block_forward_against_64_bits(zs, dtype, post, gate, p):
    """h is the 64-bit sum rounded once, bit for bit: the kernel's own sum is off by some
    2^-50, and none of these values lies that near to a tie. y's 8 bits are the 64-bit form's."""
    rs, bs = 0.875, float(torch.tensor(0.55))
    for r, c in BLOCK:
        announce(f"block forward {dtype} {post} {gate} {p} {r}x{c}")
        v, f = problem(r, c, dtype, post, gate, p)
        h, post_rstd, rstd, y, codes, scales = run_forward(zs, v, dtype, p)
        want = ref.block(*(dbl(v[k]) for k in ("x", "res", "post_gain", "gate", "gain")),
                         float(torch.tensor(1e-5)), rs, bs, f, dtype)
        assert torch.equal(h.cpu().double(), want[0])
        if post:
            close(post_rstd, want[2], 2.0 ** -23 * want[2], "post_rstd")
        close(rstd, want[3], 2.0 ** -23 * want[3], "rstd")
        assert torch.equal(y.cpu().double(), ref.rounded(want[4], dtype))
        wc, wb, _ = ops.mx_quantize(want[4], "e4m3")
        assert torch.equal(codes.cpu(), wc) and torch.equal(scales.cpu(), wb)


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=str)
@pytest.mark.parametrize("post,gate,p,with_dres", [(True, True, 0.25, True), (True, False, 0.0, False),
                                                   (False, True, 0.25, True), (False, False, 0.0, True)])
def test_block_backward_against_64_bits(zs, dtype, post, gate, p, with_dres):
    rs, bs = 0.875, float(torch.tensor(0.55))
    for r, c in BLOCK + [(300, 72), (1100, 40)]:
        announce(f"block backward {dtype} {post} {gate} {p} {r}x{c}")
        v, f = problem(r, c, dtype, post, gate, p)
        g = gen("g", r, c)
        h, dy = randn(g, r, c).to(dtype), (0.1 * randn(g, r, c)).to(dtype)
        dres = (0.1 * randn(g, r, c)).to(dtype) if with_dres else None
        rstd = 1 / torch.sqrt(h.double().square().mean(1) + 1e-5)
        post_rstd = 1 / torch.sqrt(v["x"].double().square().mean(1) + 1e-5) if post else None
        rstd, post_rstd = rstd.float(), None if post_rstd is None else post_rstd.float()
        dx, ok1 = guarded((r, c), dtype)
        dresidual, ok2 = guarded((r, c), dtype)
        sums = {k: torch.empty(c, device="cuda") for k, there in
                (("dgain", True), ("dpost_gain", post), ("dgate", gate)) if there}
        ws = torch.empty(zs.zs_block_norm_backward_workspace(r, c), dtype=torch.uint8, device="cuda")
        args = dict(x=cu(v["x"]), post_gain=cu(v["post_gain"]), post_rstd=cu(post_rstd),
                    gate=cu(v["gate"]), dres=cu(dres), residual_scale=rs, branch_scale=bs,
                    dropout=(p, SEED, OFFSET) if p else None,
                    dpost_gain=sums.get("dpost_gain"), dgate=sums.get("dgate"))
        if not post and not gate:
            args["x"] = None
        zs.zs_block_norm_backward(dy.cuda(), h.cuda(), rstd.cuda(), cu(v["gain"]), dx, dresidual,
                                  sums["dgain"], ws, **args)
        assert ok1() and ok2()
        want, mag = ref.block_grad(dy.double(), h.double(), rstd.double(), dbl(v["gain"]), dbl(dres),
                                   dbl(v["x"]), dbl(post_rstd), dbl(v["post_gain"]), dbl(v["gate"]),
                                   rs, bs, f)
        # a mean's chain: at most 64 elements of a thread, 6 levels of lanes, 16 waves; some ten
        # single roundings beside it, twice for dx
        chain = (64 + 6 + 16 + 10) * 2.0 ** -24
        for k, got in (("dx", dx), ("dresidual", dresidual)):
            inner = (2 if k == "dx" else 1) * chain * mag[k]
            close(got, want[k], U[dtype] * (want[k].abs() + inner) + inner + TINY[dtype], k)
        # a sum over rows: a share's rows, 8 of 32 shares at a time, 32 runs; each term's own chain
        rows_chain = (-(-r // 256) + 32 + 32 + 3) * 2.0 ** -24
        for k, got in sums.items():
            own = 5 * 2.0 ** -24 if k == "dgain" else chain
            close(got, want[k], (rows_chain + own) * mag[k] + TINY[FP32], k)


def test_block_forward_in_place_and_backward_in_place(zs):
    v, _ = problem(37, 520, BF16, True, True, 0.25)
    want = run_forward(zs, v, BF16, 0.25)
    for which in ("x", "res"):
        d = {k: cu(t) for k, t in v.items()}
        zs.zs_block_norm_forward(d["x"], d["res"], d["gain"], 1e-5, d[which], gate=d["gate"],
                                 post_gain=d["post_gain"], residual_scale=0.875, branch_scale=0.55,
                                 dropout=(0.25, SEED, OFFSET), y=torch.empty_like(want[3]))
        assert torch.equal(d[which], want[0])
    g = gen("bip")
    dy, dres = (0.1 * randn(g, 37, 520)).to(BF16), (0.1 * randn(g, 37, 520)).to(BF16)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")

    def backward(dx, dresidual, t):
        s = [torch.empty(520, device="cuda") for _ in range(3)]
        zs.zs_block_norm_backward(t["dy"], t["h"], want[2], cu(v["gain"]), dx, dresidual, s[0], ws,
                                  x=t["x"], post_gain=cu(v["post_gain"]), post_rstd=want[1],
                                  gate=cu(v["gate"]), dpost_gain=s[1], dgate=s[2], dres=t["dres"],
                                  residual_scale=0.875, branch_scale=0.55,
                                  dropout=(0.25, SEED, OFFSET))
        return [dx.clone(), dresidual.clone(), *s]

    fresh = lambda: {"dy": dy.cuda(), "h": want[0].clone(), "x": cu(v["x"]), "dres": dres.cuda()}
    t = fresh()
    plain = backward(torch.empty_like(t["dy"]), torch.empty_like(t["dy"]), t)
    for a, b in (("dy", "h"), ("x", "dres"), ("h", "x"), ("dres", "dy")):
        t = fresh()
        for p, q in zip(backward(t[a], t[b], t), plain):
            assert torch.equal(p, q)


def test_block_masked_places_and_rows_that_are_not_finite(zs):
    """What dropout takes out of the branch is gone from the sum, not from the first norm; a NaN
    or infinity spoils its own row alone."""
    v, f = problem(6, 96, BF16, False, True, 0.25)
    v["x"][f == 0] = math.nan
    h, *_ = run_forward(zs, v, BF16, 0.25)
    assert torch.isfinite(h.float()).all()
    v, f = problem(6, 96, BF16, True, True, 0.25)
    clean = run_forward(zs, v, BF16, 0.25)
    v["x"][2, 5], v["res"][4, 7] = math.nan, math.inf
    got = run_forward(zs, v, BF16, 0.25)
    rows = [0, 1, 3, 5]
    for a, b in zip(got, clean):
        assert torch.equal(a[rows], b[rows])
    assert torch.isnan(got[1][2]) and torch.isnan(got[3][2].float()).any()
    assert bool((got[5][4] == 255).any())


def test_block_zero_rows(zs):
    """A zero branch, a zero sum, and no rows at all."""
    v, _ = problem(4, 64, FP16, True, False, 0.0)
    v["x"][1] = 0
    v["x"][2], v["res"][2] = 0, 0
    h, post_rstd, rstd, y, _, scales = run_forward(zs, v, FP16, 0.0)
    want = ref.block(*(dbl(v[k]) for k in ("x", "res", "post_gain", "gate", "gain")),
                     float(torch.tensor(1e-5)), 0.875, float(torch.tensor(0.55)),
                     torch.ones(4, 64, dtype=F64), FP16)
    assert torch.equal(h.cpu().double(), want[0])
    assert not bool(y[2].any()) and bool((scales[2] == 1).all())
    dgain, dpost = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    none = torch.empty(0, 64, dtype=FP16, device="cuda")
    zs.zs_block_norm_backward(none, none, torch.empty(0, device="cuda"), cu(v["gain"]), none, none,
                              dgain, None, x=none, post_gain=cu(v["post_gain"]),
                              post_rstd=torch.empty(0, device="cuda"), dpost_gain=dpost)
    assert not bool(dgain.any()) and not bool(dpost.any())


def test_block_on_another_stream_and_in_a_graph(zs):
    v, _ = problem(64, 768, BF16, True, True, 0.25)
    d = {k: cu(t) for k, t in v.items()}
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    h, y, dx, dr = (torch.empty_like(d["x"]) for _ in range(4))
    rstd, prstd = torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    s3 = [torch.empty(768, device="cuda") for _ in range(3)]
    ws = torch.empty(zs.zs_block_norm_backward_workspace(64, 768), dtype=torch.uint8, device="cuda")

    def both(rule):
        how = dict(post_gain=d["post_gain"], post_rstd=prstd, gate=d["gate"], dropout=rule)
        zs.zs_block_norm_forward(d["x"], d["res"], d["gain"], 1e-5, h, rstd=rstd, y=y, **how)
        zs.zs_block_norm_backward(y, h, rstd, d["gain"], dx, dr, s3[0], ws, x=d["x"],
                                  dpost_gain=s3[1], dgate=s3[2], **how)
        return [t.clone() for t in (h, y, dx, dr, *s3)]

    both((0.25, SEED, OFFSET, step))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        how = dict(post_gain=d["post_gain"], post_rstd=prstd, gate=d["gate"],
                   dropout=(0.25, SEED, OFFSET, step))
        zs.zs_block_norm_forward(d["x"], d["res"], d["gain"], 1e-5, h, rstd=rstd, y=y, **how)
        zs.zs_block_norm_backward(y, h, rstd, d["gain"], dx, dr, s3[0], ws, x=d["x"],
                                  dpost_gain=s3[1], dgate=s3[2], **how)
        step += 1
    other = torch.cuda.Stream()
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (h, y, dx, dr, *s3)]
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            want = both((0.25, SEED, OFFSET + i))
        torch.cuda.current_stream().wait_stream(other)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_more_than_32_bits_of_elements(zs):
    """A matrix of more than 2^32 elements: its last rows have the mask of their own numbers."""
    rows, cols = (1 << 20) + 3, 4104
    x = torch.ones(rows, cols, dtype=BF16, device="cuda")
    zs.zs_dropout(x, x, (0.5, SEED, OFFSET))
    for r in (0, 1, rows - 2):
        want = torch.empty(cols, dtype=F64)
        for b in range(cols // 8):
            w = ref.philox((b, r, OFFSET & ref.LOW, OFFSET >> 32), (SEED & ref.LOW, SEED >> 32))
            for j in range(8):
                want[8 * b + j] = 2.0 * ((w[j // 2] >> 16 * (j % 2) & 0xFFFF) >= 32768)
        assert torch.equal(x[r].double().cpu(), want)


def test_block_wide_rows_and_their_gradient(zs):
    """Rows that take every launch shape up to the widest. (The 64-bit forms run
    on the CPU: torch.ldexp on the GPU is not exact.)"""
    for r, c in ((3, 1000), (5, 2040), (3, 6000), (4, 12296), (2, 20001), (3, 40000), (2, 65536)):
        announce(f"block wide {r}x{c}")
        v, _ = problem(r, c, BF16, True, True, 0.0)
        d = {k: t.cuda() for k, t in v.items()}
        h, post_rstd, rstd, y, *_ = run_forward(zs, v, BF16, 0.0)
        want = ref.block(*(dbl(v[k]) for k in ("x", "res", "post_gain", "gate", "gain")),
                         float(torch.tensor(1e-5)), 0.875, float(torch.tensor(0.55)),
                         torch.ones(r, c, dtype=F64), BF16)
        assert torch.equal(h.cpu().double(), want[0])
        assert torch.equal(y.cpu().double(), ref.rounded(want[4], BF16))
        g = gen("w", r, c)
        dy = (0.1 * randn(g, r, c)).to(BF16).cuda()
        dx, dr = torch.empty_like(h), torch.empty_like(h)
        s3 = [torch.empty(c, device="cuda") for _ in range(3)]
        ws = torch.empty(zs.zs_block_norm_backward_workspace(r, c), dtype=torch.uint8, device="cuda")
        zs.zs_block_norm_backward(dy, h, rstd, d["gain"], dx, dr, s3[0], ws, x=d["x"],
                                  post_gain=d["post_gain"], post_rstd=post_rstd, gate=d["gate"],
                                  dpost_gain=s3[1], dgate=s3[2], residual_scale=0.875,
                                  branch_scale=0.55)
        w, mag = ref.block_grad(dbl(dy.cpu()), dbl(h.cpu()), dbl(rstd.cpu()), dbl(v["gain"]), None,
                                dbl(v["x"]), dbl(post_rstd.cpu()), dbl(v["post_gain"]), dbl(v["gate"]),
                                0.875, float(torch.tensor(0.55)), torch.ones(r, c, dtype=F64))
        # as above: 64 elements of a thread, 6 levels of lanes, 16 waves, ten roundings
        chain = (64 + 6 + 16 + 10) * 2.0 ** -24
        for k, got in (("dx", dx), ("dresidual", dr)):
            inner = (2 if k == "dx" else 1) * chain * mag[k]
            close(got, w[k], U[BF16] * (w[k].abs() + inner) + inner + TINY[BF16], k)
        for k, got in zip(("dgain", "dpost_gain", "dgate"), s3):
            close(got, w[k], (70 * 2.0 ** -24 + chain) * mag[k] + TINY[FP32], k)
        dy2, h2, again = dy.clone(), h.clone(), [torch.empty_like(t) for t in s3]
        zs.zs_block_norm_backward(dy2, h2, rstd, d["gain"], h2, dy2, again[0], ws, x=d["x"],
                                  post_gain=d["post_gain"], post_rstd=post_rstd, gate=d["gate"],
                                  dpost_gain=again[1], dgate=again[2], residual_scale=0.875,
                                  branch_scale=0.55)
        assert torch.equal(h2, dx) and torch.equal(dy2, dr)
        assert all(torch.equal(a, b) for a, b in zip(again, s3))


def test_block_wide_rows_shares(zs):
    """More rows than shares, with dropout, where the shares are added to in memory."""
    r, c = 600, 16392
    g = gen("shares")
    v = dict(x=randn(g, r, c).to(BF16), gain=(1 + 0.1 * randn(g, c)).to(BF16),
             post_gain=(1 + 0.1 * randn(g, c)).to(BF16), gate=(0.3 + 0.2 * randn(g, c)).to(BF16))
    h, dy, dres = randn(g, r, c).to(BF16), (0.1 * randn(g, r, c)).to(BF16), randn(g, r, c).to(BF16)
    d = {k: t.cuda() for k, t in v.items()}
    rstd = 1 / torch.sqrt(h.double().square().mean(1) + 1e-5)
    post_rstd = 1 / torch.sqrt(v["x"].double().square().mean(1) + 1e-5)
    rstd, post_rstd = rstd.float(), post_rstd.float()
    mask = torch.ones(r, c, dtype=BF16, device="cuda")
    zs.zs_dropout(mask, mask, (0.5, SEED, OFFSET))     # its bits are tested above: 0 and 2
    dx, dr = torch.empty_like(mask), torch.empty_like(mask)
    s3 = [torch.empty(c, device="cuda") for _ in range(3)]
    ws = torch.empty(zs.zs_block_norm_backward_workspace(r, c), dtype=torch.uint8, device="cuda")
    zs.zs_block_norm_backward(dy.cuda(), h.cuda(), rstd.cuda(), d["gain"], dx, dr, s3[0], ws,
                              x=d["x"], post_gain=d["post_gain"], post_rstd=post_rstd.cuda(),
                              gate=d["gate"], dpost_gain=s3[1], dgate=s3[2], dres=dres.cuda(),
                              branch_scale=0.5, dropout=(0.5, SEED, OFFSET))
    w, mag = ref.block_grad(dbl(dy), dbl(h), dbl(rstd), dbl(v["gain"]), dbl(dres), dbl(v["x"]),
                            dbl(post_rstd), dbl(v["post_gain"]), dbl(v["gate"]), 1.0, 0.5,
                            dbl(mask.cpu()))
    # a mean's chain: 24 elements of a thread, 6 levels of lanes, 16 waves; ten roundings
    chain = (24 + 6 + 16 + 10) * 2.0 ** -24
    for k, got in (("dx", dx), ("dresidual", dr)):
        inner = (2 if k == "dx" else 1) * chain * mag[k]
        close(got, w[k], U[BF16] * (w[k].abs() + inner) + inner + TINY[BF16], k)
    for k, got in zip(("dgain", "dpost_gain", "dgate"), s3):
        # a share's three rows, 8 of 32 shares at a time, 32 runs
        close(got, w[k], ((3 + 32 + 32 + 3) * 2.0 ** -24 + chain) * mag[k] + TINY[FP32], k)


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=str)
@pytest.mark.parametrize("rs", [1.0, 0.875, 0.3])
def test_block_infinite_residual_stays_infinite(zs, dtype, rs):
    """An infinite residual under a dropped and a kept element: h has the infinity, and the norm
    behind it is NaN there and 0 in the rest of the row. A very large one stays what it is."""
    for c in (96, 1001, 4096):
        announce(f"block inf {dtype} {rs} {c}")
        v, f = problem(5, c, dtype, True, True, 0.25)
        for row, sign, keeps in ((1, 1, False), (2, -1, False), (3, 1, True)):
            at = int(torch.nonzero((f[row] > 0) == keeps)[7])
            v["res"][row, at] = sign * math.inf
        # finite, but not its size twice
        v["res"][4, int(torch.nonzero(f[4] == 0)[5])] = 2e38 if dtype is BF16 else 6e4
        h, post_rstd, rstd, y, *_ = run_forward(zs, v, dtype, 0.25, rs=rs)
        want = ref.block(*(dbl(v[k]) for k in ("x", "res", "post_gain", "gate", "gain")),
                         float(torch.tensor(1e-5)), float(torch.tensor(rs)),
                         float(torch.tensor(0.55)), f, dtype)
        assert torch.equal(h.cpu().double(), want[0])
        close(rstd, want[3], 2.0 ** -23 * want[3], "rstd")
        close(y, want[4], U[dtype] * want[4].abs() * 1.01 + TINY[dtype], "y")
        assert int(torch.isnan(y.float()).sum()) == 3


def test_block_scales_below_fp32s_range(zs):
    """Rows so large, and branch scales so small, that the branch's whole factor is no normal
    fp32 number: h is still the 64-bit sum rounded once."""
    for size, bs in ((2e38, 1.0), (2e38, 0.003), (1e35, 0.001), (1e20, 2.0 ** -60), (1.0, 0.0)):
        for p in (0.0, 0.25):
            announce(f"block small scale {size} {bs} {p}")
            v, f = problem(20, 1000, BF16, True, True, p)
            v["x"] = ((0.5 + 0.5 * torch.rand(20, 1000, generator=gen("sub"))) * size).to(BF16)
            v["post_gain"] = (0.4 + 0.5 * torch.rand(1000, generator=gen("g"))).to(BF16)
            v["res"] = (v["res"].float() * bs).to(BF16)
            h, *_ = run_forward(zs, v, BF16, p, bs=bs)
            want = ref.block(*(dbl(v[k]) for k in ("x", "res", "post_gain", "gate", "gain")),
                             float(torch.tensor(1e-5)), 0.875, float(torch.tensor(bs)), f, BF16)
            assert torch.equal(h.cpu().double(), want[0])


def test_block_backward_masked_places(zs):
    """What dropout replaced has no part in the gate's gradient, whatever it was: as if it had
    been 0. dx is 0 there."""
    for r, c in ((6, 96), (600, 1001), (3, 16392)):
        announce(f"block backward masked {r}x{c}")
        g = gen("bm", r, c)
        x, gate = randn(g, r, c).to(BF16), (0.3 + 0.2 * randn(g, c)).to(BF16)
        h, dy = randn(g, r, c).to(BF16), (0.1 * randn(g, r, c)).to(BF16)
        gain = (1 + 0.1 * randn(g, c)).to(BF16)
        rstd = (1 / torch.sqrt(h.double().square().mean(1) + 1e-5)).float()
        mask = torch.ones(r, c, dtype=BF16, device="cuda")
        zs.zs_dropout(mask, mask, (0.25, SEED, OFFSET))
        gone = mask.cpu() == 0
        clean = torch.where(gone, 0.0, x.float()).to(BF16)
        spoilt = x.clone()
        spoilt[gone] = torch.tensor([math.nan, math.inf, -math.inf]).to(BF16)[
            torch.arange(int(gone.sum())) % 3]
        outs = []
        for t in (clean, spoilt):
            dx, dr = torch.empty(r, c, dtype=BF16, device="cuda"), torch.empty(r, c, dtype=BF16,
                                                                               device="cuda")
            s2 = [torch.empty(c, device="cuda") for _ in range(2)]
            ws = torch.empty(zs.zs_block_norm_backward_workspace(r, c), dtype=torch.uint8,
                             device="cuda")
            zs.zs_block_norm_backward(dy.cuda(), h.cuda(), rstd.cuda(), gain.cuda(), dx, dr, s2[0],
                                      ws, x=t.cuda(), gate=gate.cuda(), dgate=s2[1],
                                      dropout=(0.25, SEED, OFFSET))
            assert not dx[gone.cuda()].any()
            outs.append((dx, dr, *s2))
        assert torch.isfinite(outs[0][3]).all()
        for a, b in zip(*outs):
            assert torch.equal(a, b)


@pytest.mark.parametrize("c", [1000, 12001, 16392, 20001])
def test_block_backward_of_large_and_small_rows(zs, c):
    """bf16 rows beyond 1e19 and below 1e-19, whose squares and cubes of scales leave fp32."""
    for hs, xs, ds in ((1e25, 1e-10, 1.0), (1e25, 1e20, 1e8), (1e-20, 1.0, 1e-3), (1e-25, 1e10, 1e-10),
                       (1e30, 1.0, 1e5)):
        announce(f"block backward {c} h {hs} x {xs} dy {ds}")
        r, g = 3, gen("size", c)
        x, h = (randn(g, r, c) * xs).to(BF16), (randn(g, r, c) * hs).to(BF16)
        dy, dres = (0.1 * randn(g, r, c) * ds).to(BF16), (0.1 * randn(g, r, c) * ds / hs).to(BF16)
        gain, post_gain = ((1 + 0.1 * randn(g, c)).to(BF16) for _ in range(2))
        gate = (0.3 + 0.2 * randn(g, c)).to(BF16)
        rstd = (1 / torch.sqrt(h.double().square().mean(1))).float()
        post_rstd = (1 / torch.sqrt(x.double().square().mean(1))).float()
        dx, dr = (torch.empty(r, c, dtype=BF16, device="cuda") for _ in range(2))
        s3 = [torch.empty(c, device="cuda") for _ in range(3)]
        ws = torch.empty(zs.zs_block_norm_backward_workspace(r, c), dtype=torch.uint8, device="cuda")
        zs.zs_block_norm_backward(dy.cuda(), h.cuda(), rstd.cuda(), gain.cuda(), dx, dr, s3[0], ws,
                                  x=x.cuda(), post_gain=post_gain.cuda(), post_rstd=post_rstd.cuda(),
                                  gate=gate.cuda(), dpost_gain=s3[1], dgate=s3[2], dres=dres.cuda(),
                                  branch_scale=0.5)
        w, mag = ref.block_grad(dbl(dy), dbl(h), dbl(rstd), dbl(gain), dbl(dres), dbl(x),
                                dbl(post_rstd), dbl(post_gain), dbl(gate), 1.0, 0.5,
                                torch.ones(r, c, dtype=F64))
        # as for wide rows: 64 elements of a thread, 6 levels of lanes, 16 waves, ten roundings;
        # a value below fp32's normal range is off by 2^-150 at each of some ten steps
        chain = (64 + 6 + 16 + 10) * 2.0 ** -24
        for k, got in (("dx", dx), ("dresidual", dr)):
            inner = (2 if k == "dx" else 1) * chain * mag[k] + 10 * 2.0 ** -150
            close(got, w[k], U[BF16] * (w[k].abs() + inner) + inner + TINY[BF16], k)
        for k, got in zip(("dgain", "dpost_gain", "dgate"), s3):
            close(got, w[k], (70 * 2.0 ** -24 + chain) * mag[k] + TINY[FP32], k)


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=str)
def test_block_backward_rows_walked(zs, dtype):
    """Groups of one wave up to sixteen that take a third row, with its next row's loads and both
    sums' shares in registers and in LDS."""
    r = 600
    for c in (500, 1000, 1999, 4000, 4095, 8000, 8191, 12001, 16384):
        announce(f"block backward walk {dtype} {r}x{c}")
        g = gen("walk", c)
        x, h = (randn(g, r, c) * (0.2 + torch.rand(r, 1, generator=g))).to(dtype), randn(g, r, c).to(dtype)
        gain, post_gain = ((1 + 0.1 * randn(g, c)).to(dtype) for _ in range(2))
        gate = (0.3 + 0.2 * randn(g, c)).to(dtype)
        dy, dres = (0.1 * randn(g, r, c)).to(dtype), (0.1 * randn(g, r, c)).to(dtype)
        rstd = (1 / torch.sqrt(h.double().square().mean(1) + 1e-5)).float()
        post_rstd = (1 / torch.sqrt(x.double().square().mean(1) + 1e-5)).float()
        mask = torch.ones(r, c, dtype=dtype, device="cuda")
        zs.zs_dropout(mask, mask, (0.5, SEED, OFFSET))     # its bits are tested above: 0 and 2
        for post in (True, False):
            dx, dr = (torch.empty(r, c, dtype=dtype, device="cuda") for _ in range(2))
            s3 = [torch.empty(c, device="cuda") for _ in range(3)]
            ws = torch.empty(zs.zs_block_norm_backward_workspace(r, c), dtype=torch.uint8,
                             device="cuda")
            more = dict(post_gain=post_gain.cuda(), post_rstd=post_rstd.cuda(),
                        dpost_gain=s3[2]) if post else {}
            zs.zs_block_norm_backward(dy.cuda(), h.cuda(), rstd.cuda(), gain.cuda(), dx, dr, s3[0],
                                      ws, x=x.cuda(), gate=gate.cuda(), dgate=s3[1],
                                      dres=dres.cuda(), branch_scale=0.5,
                                      dropout=(0.5, SEED, OFFSET), **more)
            w, mag = ref.block_grad(dbl(dy), dbl(h), dbl(rstd), dbl(gain), dbl(dres), dbl(x),
                                    dbl(post_rstd), dbl(post_gain) if post else None, dbl(gate),
                                    1.0, 0.5, dbl(mask.cpu()))
            # a mean's chain: 16 elements of a thread, 6 levels of lanes, 16 waves; ten roundings
            chain = (16 + 6 + 16 + 10) * 2.0 ** -24
            for k, got in (("dx", dx), ("dresidual", dr)):
                inner = (2 if k == "dx" else 1) * chain * mag[k]
                close(got, w[k], U[dtype] * (w[k].abs() + inner) + inner + TINY[dtype], k)
            for k, got in zip(("dgain", "dgate", "dpost_gain"), s3):
                if k in w:   # a share's three rows, 8 of 32 shares at a time, 32 runs
                    close(got, w[k], ((3 + 32 + 32 + 3) * 2.0 ** -24 + chain) * mag[k] + TINY[FP32], k)
