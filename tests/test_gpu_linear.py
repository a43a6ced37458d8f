"""The product with bias, activation and residual, and the gradient of that
epilogue, on the GPU against their 64-bit plain forms.

Tolerances, fixed before the first run. U: half a step of a type, relative. A
sum over k has one fp32 rounding per step of 64 elements and pass over A (two
for 8 bits), two for joining and one for the bias, each 2^-24 of the sum of
magnitudes. An activation's exponent w is off by 2^-22 |w|, and its
instructions by 4 units of 2^-22 together.
"""
import math
import zlib

import pytest
import torch

import linear_reference as ref
import ops_reference as ops
from gpu_util import announce

pytestmark = pytest.mark.gpu
BF16, FP16, F64 = torch.bfloat16, torch.float16, torch.float64
U = {t: torch.finfo(t).eps / 2 for t in (BF16, FP16)}
TINY = {BF16: 2.0 ** -134, FP16: 2.0 ** -25}


@pytest.fixture(scope="module")
def zs(hip_built):
    from sharded_mixed_precision_zs_amd import zeroshard
    return zeroshard


def gen(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def act_of(zs, act):
    return {"none": zs.ZS_ACT_NONE, "relu": zs.ZS_ACT_RELU, "gelu": zs.ZS_ACT_GELU,
            "silu": zs.ZS_ACT_SILU}[act]


def cu(t):
    return None if t is None else t.cuda()


def guarded(rows, cols, dtype, ld=None):
    """rows of cols, `ld` apart, in a buffer of a known value, and a check that nothing else was
    written."""
    ld = ld or cols
    raw = torch.full((rows * ld + 32,), 7.0, dtype=dtype, device="cuda")
    out = raw[16:16 + rows * ld].view(rows, ld)[:, :cols]

    def whole():
        mask = torch.ones_like(raw, dtype=torch.bool)
        mask[16:16 + rows * ld].view(rows, ld)[:, :cols] = False
        return bool((raw[mask] == 7.0).all())

    return out, whole


def check(got, want, tol, what):
    got, want, tol = got.double().cpu(), want.double(), torch.as_tensor(tol).double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN positions differ"
    ok = torch.isfinite(want)
    err, tol = (got - want).abs()[ok], tol.expand(want.shape)[ok]
    assert bool((err <= tol).all()), (
        f"{what}: {int((err > tol).sum())} of {err.numel()} off; worst "
        f"{float((err / tol.clamp(min=1e-300)).max()):.3g} times the tolerance")


def operands(m, n, k, afmt):
    g = gen("l", m, n, k)
    randn = lambda *s: torch.randn(*s, generator=g)
    ac, asc, a = ops.mx_quantize((randn(m, k) * torch.exp(0.5 * randn(m, 1))).double(), afmt)
    bc, bsc, b = ops.mx_quantize((randn(n, k) * (1.5 / math.sqrt(max(k, 1)))).double(), "e2m1")
    return [t.cuda() for t in (ac, asc, bc, bsc)], a, b, randn


def expected(a, b, bias, act, res, afmt, dtype):
    """(c, its tolerance, pre, its tolerance)."""
    pre, mag = a @ b.t(), a.abs() @ b.abs().t()
    if bias is not None:
        pre, mag = pre + bias.double(), mag + bias.double().abs()
    steps = a.shape[1] / 64 * (2 if afmt == "e4m3" else 1) + 3
    acc = steps * 2.0 ** -24 * mag
    c = ref.activate(pre, act)
    inner = 1.13 * acc + 2.0 ** -24 * c.abs()
    if act in ("gelu", "silu"):
        w = ref.logistic_argument(pre, act)[0].abs() * math.log2(math.e)
        inner = inner + c.abs() * (w + 4) * 2.0 ** -22
    if res is not None:
        c = c + res.double()
        inner = inner + 2.0 ** -24 * c.abs()
    return (c, U[dtype] * (c.abs() + inner) + inner + TINY[dtype],
            pre, U[dtype] * (pre.abs() + acc) + acc + TINY[dtype])


SHAPES = [(1, 1, 1), (1, 70, 200), (2, 500, 640), (5, 33, 4096), (16, 257, 384), (17, 100, 129),
          (32, 130, 256), (33, 31, 2000), (65, 130, 700), (77, 161, 6400), (129, 255, 1024),
          (300, 520, 384)]


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=str)
@pytest.mark.parametrize("afmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("act,bias,res,pre", [("none", True, True, False), ("gelu", True, False, True),
                                              ("silu", False, True, True), ("relu", True, True, True)])
def test_linear_against_64_bits(zs, dtype, afmt, act, bias, res, pre):
    fmt = zs.ZS_MX_E4M3 if afmt == "e4m3" else zs.ZS_MX_E2M1
    for m, n, k in SHAPES:
        announce(f"linear {dtype} {afmt} {act} {m}x{n}x{k}")
        dev, a, b, randn = operands(m, n, k, afmt)
        v = (0.5 * randn(n)).to(dtype) if bias else None
        r = (2 * randn(m, n)).to(dtype) if res else None
        c, tol, p, ptol = expected(a, b, v, act, r, afmt, dtype)
        for ws in (torch.empty(32 << 20, dtype=torch.uint8, device="cuda"), None):
            out, whole = guarded(m, n, dtype)
            pout, pwhole = guarded(m, n, dtype) if pre else (None, lambda: True)
            zs.zs_mx_linear(dev[0], dev[1], fmt, dev[2], dev[3], out, k, bias=cu(v),
                            activation=act_of(zs, act), residual=cu(r), pre=pout, workspace=ws)
            check(out, c, tol, f"c {m}x{n}x{k}")
            if pre:
                check(pout, p, ptol, f"pre {m}x{n}x{k}")
            assert whole() and pwhole()


@pytest.mark.parametrize("afmt,m,n,k", [("e4m3", 1000, 20001, 130), ("e2m1", 2100, 9000, 256)])
def test_linear_of_many_tiles_is_the_product_and_its_epilogue(zs, afmt, m, n, k):
    """The large tiles: pre has the product's own bits where there is no bias, and c follows
    from sums between pre's neighbours."""
    dev, a, b, randn = operands(m, n, k, afmt)
    fmt = zs.ZS_MX_E4M3 if afmt == "e4m3" else zs.ZS_MX_E2M1
    want = torch.empty(m, n, dtype=BF16, device="cuda")
    zs.zs_mx_matmul(dev[0], dev[1], fmt, dev[2], dev[3], want, k)
    out, whole = guarded(m, n, BF16)
    pre = torch.empty_like(want)
    res = randn(m, n).to(BF16).cuda()
    zs.zs_mx_linear(dev[0], dev[1], fmt, dev[2], dev[3], out, k, activation=zs.ZS_ACT_SILU,
                    residual=res, pre=pre)
    assert torch.equal(pre, want) and whole()
    # half a step of pre moves silu by at most 1.1 of it; then c's own rounding
    c = torch.nn.functional.silu(pre.double()) + res.double()
    tol = 1.1 * U[BF16] * pre.double().abs() + 2.0 ** -18 + U[BF16] * 1.01 * c.abs()
    assert bool(((out.double() - c).abs() <= tol).all())


def test_linear_strides_and_in_place(zs):
    for m in (3, 40, 150):
        n, k = 161, 320
        dev, a, b, randn = operands(m, n, k, "e4m3")
        v, r = (0.5 * randn(n)).to(BF16), (2 * randn(m, n)).to(BF16)
        c, tol, _, _ = expected(a, b, v, "gelu", r, "e4m3", BF16)
        for ldc, ldr in ((164, 161), (163, 170), (168, 168)):
            announce(f"linear strided {m} {ldc} {ldr}")
            out, whole = guarded(m, n, BF16, ldc)
            rr, _ = guarded(m, n, BF16, ldr)
            rr.copy_(r)
            zs.zs_mx_linear(dev[0], dev[1], zs.ZS_MX_E4M3, dev[2], dev[3], out, k, bias=v.cuda(),
                            activation=zs.ZS_ACT_GELU, residual=rr)
            check(out, c, tol, "strided")
            assert whole()
            zs.zs_mx_linear(dev[0], dev[1], zs.ZS_MX_E4M3, dev[2], dev[3], rr, k, bias=v.cuda(),
                            activation=zs.ZS_ACT_GELU, residual=rr)
            assert torch.equal(rr, out)


def test_linear_without_k_and_with_nan(zs):
    e, f = torch.empty(5, 0, dtype=torch.uint8).cuda(), torch.empty(40, 0, dtype=torch.uint8).cuda()
    bias, res = torch.randn(40).to(BF16), torch.randn(5, 40).to(BF16)
    out = torch.empty(5, 40, dtype=BF16, device="cuda")
    zs.zs_mx_linear(e, e, zs.ZS_MX_E4M3, f, f, out, 0, bias=bias.cuda(), activation=zs.ZS_ACT_RELU,
                    residual=res.cuda())
    assert torch.equal(out.cpu(), (res.float() + bias.float().clamp(min=0)).to(BF16))
    g = gen("nan")
    for m in (2, 70):
        x, y = torch.randn(m, 192, generator=g).double(), torch.randn(90, 192, generator=g).double()
        x[m // 2, 100] = math.inf
        ac, asc, _ = ops.mx_quantize(x, "e4m3")
        bc, bsc, _ = ops.mx_quantize(y, "e2m1")
        for act in ("relu", "gelu", "silu"):
            c = torch.empty(m, 90, dtype=BF16, device="cuda")
            zs.zs_mx_linear(ac.cuda(), asc.cuda(), zs.ZS_MX_E4M3, bc.cuda(), bsc.cuda(), c, 192,
                            activation=act_of(zs, act))
            nan = torch.isnan(c.cpu())
            assert nan[m // 2].all() and not nan[[i for i in range(m) if i != m // 2]].any()


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=str)
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
def test_activation_backward_against_64_bits(zs, dtype, act):
    for r, c in [(1, 1), (2, 7), (5, 100), (300, 130), (9, 2049), (1000, 520), (77, 4099), (3000, 24),
                 (40, 12000)]:
        announce(f"activation backward {dtype} {act} {r}x{c}")
        g = gen("ab", r, c)
        dc = torch.randn(r, c, generator=g).to(dtype)
        pre = (2 * torch.randn(r, c, generator=g)).to(dtype)
        pre[0, 0], pre[-1, -1] = 0.0, -50.0
        s, bound = ref.slope(pre.double(), act)
        w = ref.logistic_argument(pre.double(), act)[0].abs() * math.log2(math.e)
        inner = dc.double().abs() * ((bound * (w.clamp(max=160) + 6) * 2.0 ** -22
                                      if act in ("gelu", "silu") else 0) + 2.0 ** -24 * s.abs())
        inner = inner + 2.0 ** -126
        want = dc.double() * s
        dpre, whole = guarded(r, c, dtype)
        dbias = torch.empty(c, device="cuda")
        ws = torch.empty(zs.zs_activation_backward_workspace(r, c), dtype=torch.uint8, device="cuda")
        p = None if act == "none" else pre.cuda()
        zs.zs_activation_backward(dc.cuda(), p, act_of(zs, act), dpre, dbias=dbias, workspace=ws)
        check(dpre, want, U[dtype] * (want.abs() + inner) + inner + TINY[dtype], "dpre")
        # a share has at most r / 32 rows and 8 more, 32 shares a run at most, 32 runs
        chain = (r / 32 + 8 + 32 + 32) * 2.0 ** -24
        check(dbias, want.sum(0), chain * want.abs().sum(0) + inner.sum(0) + 1e-40, "dbias")
        assert whole()
        # each output alone, and in place
        alone, sums = torch.empty_like(dpre), torch.empty_like(dbias)
        zs.zs_activation_backward(dc.cuda(), p, act_of(zs, act), alone)
        zs.zs_activation_backward(dc.cuda(), p, act_of(zs, act), None, dbias=sums, workspace=ws)
        assert torch.equal(alone, dpre) and torch.equal(sums, dbias)
        for i, t in enumerate((dc.cuda(), None if p is None else p.clone())):
            if t is not None:
                zs.zs_activation_backward(t if i == 0 else dc.cuda(), t if i == 1 else p,
                                          act_of(zs, act), t)
                assert torch.equal(t, dpre)


def test_activation_backward_ends(zs):
    """Far values, infinities and NaN of pre; no rows."""
    pre = torch.tensor([[-3e38, -1e13, -100.0, 100.0, 1e13, 3e38, math.inf, -math.inf, math.nan]]).to(BF16)
    dc = torch.ones_like(pre)
    for act in ("relu", "gelu", "silu"):
        out = torch.empty_like(pre).cuda()
        zs.zs_activation_backward(dc.cuda(), pre.cuda(), act_of(zs, act), out)
        got = out.cpu().float()[0]
        assert got[:2].abs().max() < 1e-30 and torch.equal(got[3:7], torch.ones(4))
        assert abs(float(got[7])) < 1e-30 and torch.isnan(got[8])
        assert abs(float(got[2])) < 1e-38
    dbias = torch.ones(9, device="cuda")
    none = torch.empty(0, 9, dtype=BF16, device="cuda")
    zs.zs_activation_backward(none, none, zs.ZS_ACT_GELU, none, dbias=dbias)
    assert not dbias.any()


def test_more_than_32_bits_of_elements(zs):
    """pre and c of more than 2^32 elements, and rows that are 2^31 apart."""
    m, n, k = 65600, 65544, 64
    g = gen("large")
    # codes of +-1, and scales of 1: every sum is a whole number that bf16 has
    a = torch.randint(0, 2, (m, k), generator=g) * 2.0 - 1
    b = torch.randint(0, 2, (n, k), generator=g) * 2.0 - 1
    a8, b4 = zs.mx_empty(m, k, zs.ZS_MX_E4M3), zs.mx_empty(n, k, zs.ZS_MX_E2M1)
    zs.zs_mx_quantize(a.to(BF16).cuda(), zs.ZS_MX_E4M3, *a8)
    zs.zs_mx_quantize(b.to(BF16).cuda(), zs.ZS_MX_E2M1, *b4)
    out, pre = (torch.empty(m, n, dtype=BF16, device="cuda") for _ in range(2))
    zs.zs_mx_linear(*a8, zs.ZS_MX_E4M3, *b4, out, k, activation=zs.ZS_ACT_RELU, pre=pre)
    for rows in (slice(0, 3), slice(32767, 32770), slice(m - 65, m)):
        want = a[rows] @ b.t()
        assert torch.equal(pre[rows].float().cpu(), want)
        assert torch.equal(out[rows].float().cpu(), want.clamp(min=0))
    del out
    dpre, dbias = torch.empty_like(pre), torch.empty(n, device="cuda")
    ws = torch.empty(zs.zs_activation_backward_workspace(m, n), dtype=torch.uint8, device="cuda")
    zs.zs_activation_backward(pre, pre, zs.ZS_ACT_RELU, dpre, dbias, ws)
    assert torch.equal(dpre[-65:].float().cpu(), (a[-65:] @ b.t()).clamp(min=0))
    del pre, dpre
    ld, few = 1 << 31, 3
    raw = torch.empty(2 * (few - 1) * ld + 2 * n, dtype=BF16, device="cuda")
    out, res = (raw[i * n:].as_strided((few, n), (2 * ld, 1)) for i in range(2))
    res.fill_(4.0)
    a8 = zs.mx_empty(few, k, zs.ZS_MX_E4M3)
    zs.zs_mx_quantize(a[:few].to(BF16).cuda(), zs.ZS_MX_E4M3, *a8)
    with pytest.raises(zs.ZsError):     # the extents cross each other
        zs.zs_mx_linear(*a8, zs.ZS_MX_E4M3, *b4, out, k, residual=res)
    zs.zs_mx_linear(*a8, zs.ZS_MX_E4M3, *b4, res, k, residual=res)
    assert torch.equal(res.float().cpu(), a[:few] @ b.t() + 4)


def test_tensors_of_another_device_are_refused(zs, monkeypatch):
    """Every entry point looks at its tensors' device before it queues anything."""
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    v, r = x[0].clone(), torch.zeros(4, device="cuda")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    a8, b4 = zs.mx_empty(4, 64, zs.ZS_MX_E4M3), zs.mx_empty(64, 64, zs.ZS_MX_E2M1)
    out = [torch.full_like(x, 7.0) for _ in range(3)]
    calls = {
        "dropout": lambda: zs.zs_dropout(x, out[0], (0.5, 1, 2)),
        "block": lambda: zs.zs_block_norm_forward(x, x, v, 1e-5, out[0], y=out[1]),
        "block back": lambda: zs.zs_block_norm_backward(x, x, r, v, out[0], out[1],
                                                        torch.zeros(64, device="cuda"), ws),
        "linear": lambda: zs.zs_mx_linear(*a8, zs.ZS_MX_E4M3, *b4, out[0], 64),
        "act": lambda: zs.zs_activation_backward(x, x, zs.ZS_ACT_GELU, out[0]),
        "logprob": lambda: zs.zs_logprob(x, ids, torch.empty_like(r), workspace=ws),
        "policy": lambda: zs.zs_policy(x, ids, r, torch.empty_like(r), grad=out[0], workspace=ws),
        "preference": lambda: zs.zs_preference(x, ids, ids[:3], 0.1, r[:1].clone(), grad=out[0],
                                               workspace=ws),
    }
    monkeypatch.setattr(zs._t(), "device", lambda: 1)
    for name, call in calls.items():
        with pytest.raises(ValueError, match="current device is 1"):
            call()
    torch.cuda.synchronize()
    assert all(bool((o == 7).all()) for o in out)


@pytest.mark.parametrize("dtype,act,r,c", [(BF16, "gelu", 70000, 264), (FP16, "silu", 33000, 513),
                                           (BF16, "none", 2100000, 8), (FP16, "relu", 70001, 257)],
                         ids=str)
def test_activation_backward_rows_walked(zs, dtype, act, r, c):
    """So many rows that a block takes several turns of them."""
    announce(f"activation backward walk {dtype} {act} {r}x{c}")
    g = gen("aw", r, c)
    dc = torch.randn(r, c, generator=g).to(dtype)
    pre = (2 * torch.randn(r, c, generator=g)).to(dtype)
    s, bound = ref.slope(pre.double(), act)
    w = ref.logistic_argument(pre.double(), act)[0].abs() * math.log2(math.e)
    inner = dc.double().abs() * ((bound * (w.clamp(max=160) + 6) * 2.0 ** -22
                                  if act in ("gelu", "silu") else 0) + 2.0 ** -24 * s.abs())
    # the exponential gives 0 below 2^-126, and so p, which is off by as much: the slope p (1 +
    # x q w') by |1 + x q w'| times that (of gelu's at -10 some 200 times)
    p = torch.sigmoid(ref.logistic_argument(pre.double(), act)[0])
    inner = inner + 2.0 ** -126 * (1 + dc.double().abs() * (bound / p.clamp(min=1e-300)
                                                            if act in ("gelu", "silu") else 0))
    want = dc.double() * s
    dpre = torch.empty_like(dc).cuda()
    dbias = torch.empty(c, device="cuda")
    ws = torch.empty(zs.zs_activation_backward_workspace(r, c), dtype=torch.uint8, device="cuda")
    zs.zs_activation_backward(dc.cuda(), None if act == "none" else pre.cuda(), act_of(zs, act), dpre,
                              dbias=dbias, workspace=ws)
    check(dpre, want, U[dtype] * (want.abs() + inner) + inner + TINY[dtype], "dpre")
    # a thread takes four rows a turn, two turns here; a block's rows join in at most ten halvings,
    # 1024 shares in 32 runs of 32
    chain = (8 + 10 + 32 + 32) * 2.0 ** -24
    check(dbias, want.sum(0), chain * want.abs().sum(0) + inner.sum(0) + 1e-40, "dbias")
