"""The output end's operators on the GPU against their 64-bit plain forms.

Tolerances, fixed before the first run. A rounding to a type t is off by at
most half a step, relative eps(t)/2 (U below), or half its smallest
subnormal. An fp32 sum of n magnitudes adding up to M is off by at most
n * 2^-24 * M, n the length of its longest chain of additions.
"""
import math
import zlib

import pytest
import torch

import ops_reference as ref
from gpu_util import announce

pytestmark = pytest.mark.gpu
BF16, FP16, FP32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
U = {t: torch.finfo(t).eps / 2 for t in (BF16, FP16, FP32)}
TINY = {BF16: 2.0 ** -134, FP16: 2.0 ** -25, FP32: 2.0 ** -126}
SENTINEL = 0xA5


@pytest.fixture(scope="module")
def zs(hip_built):
    from sharded_mixed_precision_zs_amd import zeroshard
    return zeroshard


def gen(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def randn(g, *shape):
    return torch.randn(*shape, generator=g, dtype=FP32)


def fmt_of(zs, name):
    return zs.ZS_MX_E2M1 if name == "e2m1" else zs.ZS_MX_E4M3


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


# ---- quantisation --------------------------------------------------------------

QUANT = [(1, 1), (1, 31), (3, 32), (5, 33), (2, 128), (7, 129), (33, 200), (64, 256), (130, 96),
         (257, 1000), (1, 4099)]


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16], ids=str)
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("columns", [False, True])
def test_quantize_matches_exactly(zs, dtype, fmt, columns):
    for r, c in QUANT:
        announce(f"quantize {dtype} {fmt} columns={columns} {r}x{c}")
        g = gen("q", r, c)
        x = (randn(g, r, c) * torch.exp(randn(g, r, 1) * 2)).to(dtype)
        x[0, 0] = 0.0
        if dtype == FP32 and c > 40:
            x[0, :33] = torch.linspace(-8, 8, 33)          # ties between the codes
            x[-1, -1] = 1e-41                              # subnormal
        v = x.double().t().contiguous() if columns else x.double()
        codes, byte, val = ref.mx_quantize(v, fmt)
        cs, ss = zs.mx_shapes(*v.shape, fmt_of(zs, fmt))
        dc, ok1 = guarded(cs, torch.uint8)
        ds, ok2 = guarded(ss, torch.uint8)
        dv, ok3 = guarded((r, c), BF16)
        zs.zs_mx_quantize(x.cuda(), fmt_of(zs, fmt), dc, ds, columns=columns, values=dv)
        assert torch.equal(ds.cpu(), byte)
        assert torch.equal(dc.cpu(), codes)
        want = (val.t() if columns else val).to(BF16)
        assert torch.equal(dv.cpu().view(torch.int16), want.contiguous().view(torch.int16))
        assert ok1() and ok2() and ok3()


@pytest.mark.parametrize("columns", [False, True])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_quantize_blocks_that_are_not_finite(zs, fmt, columns):
    x = torch.randn(96, 160, generator=gen("nf"))
    x[0, 5], x[40, 40], x[70, 159], x[3, 33] = math.inf, math.nan, -math.inf, 3e38
    x[64:, 64:96] = 0.0
    v = x.double().t().contiguous() if columns else x.double()
    codes, byte, val = ref.mx_quantize(v, fmt)
    dc, ds = zs.mx_empty(*v.shape, fmt_of(zs, fmt))
    dv = torch.empty(96, 160, dtype=BF16, device="cuda")
    zs.zs_mx_quantize(x.cuda(), fmt_of(zs, fmt), dc, ds, columns=columns, values=dv)
    assert torch.equal(ds.cpu(), byte) and torch.equal(dc.cpu(), codes)
    want = (val.t() if columns else val).to(BF16)
    assert torch.equal(torch.isnan(dv.cpu()), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(dv.cpu()), torch.nan_to_num(want))


@pytest.mark.parametrize("columns", [False, True])
def test_quantize_strided_and_unaligned_source(zs, columns):
    base = randn(gen("st"), 70, 301).to(BF16)
    for off, width in ((0, 64), (1, 64), (3, 200), (8, 256)):
        announce(f"quantize strided offset {off} width {width}")
        x = base[:, off:off + width]
        v = x.double().t().contiguous() if columns else x.double()
        codes, byte, _ = ref.mx_quantize(v, "e2m1")
        dc, ds = zs.mx_empty(*v.shape, zs.ZS_MX_E2M1)
        zs.zs_mx_quantize(base.cuda()[:, off:off + width], zs.ZS_MX_E2M1, dc, ds, columns=columns)
        assert torch.equal(ds.cpu(), byte) and torch.equal(dc.cpu(), codes)


def test_quantize_rows_past_32_bits(zs):
    """Rows 2^31 elements apart."""
    big = torch.empty(2 * (1 << 31) + 128, dtype=BF16, device="cuda")
    x = randn(gen("big"), 3, 128).to(BF16)
    view = big.as_strided((3, 128), (1 << 31, 1))
    view.copy_(x)
    codes, byte, _ = ref.mx_quantize(x.double(), "e4m3")
    dc, ds = zs.mx_empty(3, 128, zs.ZS_MX_E4M3)
    zs.zs_mx_quantize(view, zs.ZS_MX_E4M3, dc, ds)
    assert torch.equal(ds.cpu(), byte) and torch.equal(dc.cpu(), codes)


# ---- product -------------------------------------------------------------------

PRODUCT = [(1, 1, 1), (1, 64, 128), (1, 33, 4096), (2, 500, 640), (15, 16, 96), (16, 257, 384),
           (17, 100, 129), (33, 31, 2000), (64, 128, 256), (65, 130, 700), (77, 513, 768),
           (128, 128, 512), (129, 255, 1024), (200, 300, 4224), (256, 256, 256), (300, 520, 384),
           (1, 2048, 8192), (5, 96, 16384)]


def product_tolerance(a, b, want, afmt, dtype):
    """Half a step of the result, and the sums': one fp32 rounding per step of
    64 elements of K for 4-bit operands; with an 8-bit one the matrix unit drops
    what lies 13 bits below the largest of eight neighbouring products, which for
    quantised normal data stays below 2^-16 of the sum of magnitudes."""
    mag = a.abs() @ b.abs().t()
    steps = a.shape[1] / 64 + 2
    acc = steps * 2.0 ** -24 * mag + (2.0 ** -16 * mag if afmt == "e4m3" else 0)
    return U[dtype] * (want.abs() + acc) + acc + TINY[dtype]


@pytest.mark.parametrize("afmt,dtype", [("e4m3", BF16), ("e4m3", FP16), ("e2m1", BF16),
                                        ("e2m1", FP16), ("e2m1", FP32)], ids=str)
def test_product_against_64_bits(zs, afmt, dtype):
    for m, n, k in PRODUCT:
        announce(f"product {afmt} {dtype} {m}x{n}x{k}")
        g = gen("p", m, n, k)
        ac, asc, a = ref.mx_quantize((randn(g, m, k) * torch.exp(randn(g, m, 1))).double(), afmt)
        bc, bsc, b = ref.mx_quantize((randn(g, n, k) * 0.05).double(), "e2m1")
        want = a @ b.t()
        out, whole = guarded((m, n), dtype)
        ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
        for w in (ws, None):
            zs.zs_mx_matmul(ac.cuda(), asc.cuda(), fmt_of(zs, afmt), bc.cuda(), bsc.cuda(), out, k,
                            workspace=w)
            close(out, want, product_tolerance(a, b, want, afmt, dtype), f"{m}x{n}x{k}")
            assert whole()


@pytest.mark.parametrize("afmt,m,n,k", [("e4m3", 1000, 20001, 900), ("e2m1", 2100, 9000, 640),
                                        ("e2m1", 1030, 17000, 1152)])
def test_product_of_many_tiles(zs, afmt, m, n, k):
    """Enough tiles for every kernel variant, every code, ragged edges."""
    g = gen("pl", m, n, k)
    p = ref.padded(k)
    ops = []
    for rows, fmt in ((m, afmt), (n, "e2m1")):
        c = torch.randint(0, 256, (rows, p // 2 if fmt == "e2m1" else p), generator=g,
                          dtype=torch.uint8)
        if fmt == "e4m3":
            c[(c & 127) == 127] = 1                        # not NaN
        c[:, (k if fmt == "e4m3" else k // 2):] = 0        # the padding is zeros
        s = torch.randint(118, 130, (rows, p // 32), generator=g, dtype=torch.uint8)
        ops += [c, s, ref.mx_values(c, s, fmt, k)]
    ac, asc, bc, bsc = (ops[i].cuda() for i in (0, 1, 3, 4))
    out, whole = guarded((m, n), BF16)
    zs.zs_mx_matmul(ac, asc, fmt_of(zs, afmt), bc, bsc, out, k)
    assert whole()
    # every tile adds up along k in the same order: a part of C alone has the same bits
    for r0, c0 in ((0, 0), (m - 300, n - 700), (256, 4096)):
        part = torch.empty(300, 700, dtype=BF16, device="cuda")
        zs.zs_mx_matmul(ac[r0:r0 + 300], asc[r0:r0 + 300], fmt_of(zs, afmt),
                        bc[c0:c0 + 700], bsc[c0:c0 + 700], part, k)
        assert torch.equal(part, out[r0:r0 + 300, c0:c0 + 700])
    if afmt == "e2m1":
        a, b = ops[2].cuda(), ops[5].cuda()
        want, mag = (a @ b.t()).cpu(), (a.abs() @ b.abs().t()).cpu()
        acc = (k / 64 + 2) * 2.0 ** -24 * mag
        close(out, want, U[BF16] * (want.abs() + acc) + acc + TINY[BF16], "C")


@pytest.mark.parametrize("m", [3, 40, 130])
def test_product_of_odd_and_strided_results(zs, m):
    """Rows of C further apart than n, at odd offsets: nothing between them is written."""
    g = gen("ps", m)
    n, k = 161, 320
    ac, asc, a = ref.mx_quantize(randn(g, m, k).double(), "e4m3")
    bc, bsc, b = ref.mx_quantize(randn(g, n, k).double(), "e2m1")
    want = a @ b.t()
    for ld, off in ((164, 0), (163, 1), (168, 4)):
        raw = torch.full((m * ld + 16,), 7.0, dtype=BF16, device="cuda")
        out = raw[off:off + m * ld].view(m, ld)[:, :n]
        zs.zs_mx_matmul(ac.cuda(), asc.cuda(), zs.ZS_MX_E4M3, bc.cuda(), bsc.cuda(), out, k)
        close(out, want, product_tolerance(a, b, want, "e4m3", BF16), f"ld {ld} offset {off}")
        keep = torch.ones_like(raw, dtype=torch.bool)
        keep[off:off + m * ld].view(m, ld)[:, :n] = False
        assert bool((raw[keep] == 7.0).all())


@pytest.mark.parametrize("m,n", [(1, 70), (40, 70), (200, 300)])
def test_product_carries_nan_blocks_and_empty_k(zs, m, n):
    g = gen("pn", m)
    x, y = randn(g, m, 192).double(), randn(g, n, 192).double()
    x[m // 2, 100], y[n - 2, 3] = math.inf, math.nan
    ac, asc, a = ref.mx_quantize(x, "e4m3")
    bc, bsc, b = ref.mx_quantize(y, "e2m1")
    out = torch.empty(m, n, dtype=BF16, device="cuda")
    zs.zs_mx_matmul(ac.cuda(), asc.cuda(), zs.ZS_MX_E4M3, bc.cuda(), bsc.cuda(), out, 192)
    want = a @ b.t()
    close(out, want, product_tolerance(torch.nan_to_num(a), torch.nan_to_num(b),
                                       torch.nan_to_num(want), "e4m3", BF16), "NaN blocks")
    e = torch.empty(m, 0, dtype=torch.uint8, device="cuda")
    f = torch.empty(n, 0, dtype=torch.uint8, device="cuda")
    zs.zs_mx_matmul(e, e, zs.ZS_MX_E4M3, f, f, out, 0)
    assert not out.any()


def test_product_repeats_its_bits(zs):
    g = gen("rep")
    for m, n, k in ((1, 512, 4096), (100, 300, 8192), (300, 300, 2048)):
        ac, asc, _ = ref.mx_quantize(randn(g, m, k).double(), "e4m3")
        bc, bsc, _ = ref.mx_quantize(randn(g, n, k).double(), "e2m1")
        ops = [t.cuda() for t in (ac, asc, bc, bsc)]
        ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
        outs = [torch.empty(m, n, dtype=BF16, device="cuda") for _ in range(3)]
        for o in outs:
            zs.zs_mx_matmul(ops[0], ops[1], zs.ZS_MX_E4M3, ops[2], ops[3], o, k, workspace=ws)
        assert all(torch.equal(outs[0].view(torch.int16), o.view(torch.int16)) for o in outs)


# ---- norm ----------------------------------------------------------------------

NORM = [(1, 1), (1, 31), (3, 64), (2, 100), (5, 768), (4, 1000), (7, 1600), (1100, 520), (1030, 4096),
        (2, 4104), (3, 9001), (2, 16384), (1, 40000), (1, 65536)]


def norm_inputs(zs, r, c, dt, residual):
    g = gen("n", r, c)
    x = randn(g, r, c).to(dt)
    res = (randn(g, r, c) * 2).to(dt) if residual else None
    gain = (1 + 0.2 * randn(g, c)).to(dt)
    # h as defined: the fp32 sum rounded once
    h = (x.float() + res.float()).to(dt) if residual else x
    return x, res, gain, h


@pytest.mark.parametrize("dt", [BF16, FP16], ids=str)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_forward(zs, dt, residual):
    for r, c in NORM:
        announce(f"norm forward {dt} residual={residual} {r}x{c}")
        x, res, gain, h = norm_inputs(zs, r, c, dt, residual)
        y, rstd = ref.rmsnorm(h.double(), gain.double(), 1e-5)
        cs, ss = zs.mx_shapes(r, c, zs.ZS_MX_E4M3)
        (dh, k1), (dy, k2) = guarded((r, c), dt), guarded((r, c), dt)
        (dc, k3), (ds, k4), (dr, k5) = (guarded(cs, torch.uint8), guarded(ss, torch.uint8),
                                        guarded((r,), FP32))
        zs.zs_rmsnorm_forward(x.cuda(), gain.cuda(), 1e-5, h=dh, rstd=dr, y=dy, codes=dc, scales=ds,
                              residual=None if res is None else res.cuda())
        assert k1() and k2() and k3() and k4() and k5()
        assert torch.equal(dh.cpu().view(torch.int16), h.contiguous().view(torch.int16))
        # chains: at most 64 squares per thread, 6 steps in a wave, 16 waves; half of that in the root
        rel = (64 + 6 + 16 + 6) * 2.0 ** -24
        close(dr, rstd, rel * rstd, "rstd")
        rel += 4 * 2.0 ** -24
        close(dy, y, U[dt] * y.abs() * (1 + rel) + rel * y.abs() + TINY[dt], "y")
        # 8 bits: half a step of a normal or subnormal code, or what saturates
        codes, byte = dc.cpu(), ds.cpu()
        val = ref.mx_values(codes, byte, "e4m3", c)
        s = ref.pow2(byte.long() - 127).repeat_interleave(32, 1)[:, :c]
        tol = torch.maximum(y.abs() * 2.0 ** -4, s * 2.0 ** -10)
        tol = torch.where(y.abs() > 448 * s, torch.maximum(tol, y.abs() - 448 * s), tol)
        close(val, y, tol + rel * y.abs(), "8-bit y")
        # the scale is that of the block's largest, up to the sum's rounding
        lo, hi = ref.mx_quantize(y * (1 - rel), "e4m3")[1], ref.mx_quantize(y * (1 + rel), "e4m3")[1]
        assert bool(((byte >= lo) & (byte <= hi)).all())
        assert not codes[:, c:].any()


def test_norm_forward_in_place_and_partial_outputs(zs):
    x, res, gain, h = norm_inputs(zs, 5, 776, BF16, True)
    want = torch.empty(5, 776, dtype=BF16, device="cuda")
    zs.zs_rmsnorm_forward(x.cuda(), gain.cuda(), 1e-5, h=torch.empty_like(want), residual=res.cuda(),
                          y=want)
    for place in ("x", "res"):
        dx, dres = x.cuda(), res.cuda()
        y = torch.empty_like(want)
        zs.zs_rmsnorm_forward(dx, gain.cuda(), 1e-5, h=dx if place == "x" else dres, residual=dres,
                              y=y)
        got = dx if place == "x" else dres
        assert torch.equal(got.cpu().view(torch.int16), h.view(torch.int16))
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))


def test_norm_forward_rows_that_are_zero_or_not_finite(zs):
    x = randn(gen("nz"), 6, 256).to(BF16)
    x[0] = 0.0
    x[1, 3] = math.inf
    x[2, 200] = math.nan
    gain = torch.ones(256, dtype=BF16)
    gain[7] = 0.0
    c, s = zs.mx_empty(6, 256, zs.ZS_MX_E4M3)
    y = torch.empty(6, 256, dtype=BF16, device="cuda")
    zs.zs_rmsnorm_forward(x.cuda(), gain.cuda(), 0.0, y=y, codes=c, scales=s)
    val = ref.mx_values(c.cpu(), s.cpu(), "e4m3", 256)
    assert torch.isnan(val[2]).all() and torch.isnan(y[2]).all()
    # inf * 0 in the row's own place, 0 elsewhere; a zero row with eps = 0 is 0 * inf
    assert torch.isnan(y[1, 3]) and torch.isnan(val[1, :32]).all() and not val[1, 32:].any()
    assert torch.isnan(y[0]).all()
    assert torch.isfinite(val[3:]).all() and not val[3:, 7].any()


@pytest.mark.parametrize("dt", [BF16, FP16], ids=str)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_backward(zs, dt, residual):
    for r, c in NORM + [(2500, 96), (1500, 33)]:
        announce(f"norm backward {dt} residual={residual} {r}x{c}")
        g = gen("nb", r, c)
        h = randn(g, r, c).to(dt)
        gain = (1 + 0.2 * randn(g, c)).to(dt)
        dy, dres = (randn(g, r, c) * 0.1).to(dt), (randn(g, r, c) * 0.1).to(dt) if residual else None
        rstd = (h.double().square().mean(1) + 1e-5).rsqrt().float()
        dx, dgain, mag, gmag = ref.rmsnorm_grad(dy.double(), h.double(), rstd.double(), gain.double(),
                                                None if dres is None else dres.double())
        ws = torch.empty(max(4, zs.zs_rmsnorm_backward_workspace(r, c)), dtype=torch.uint8,
                         device="cuda")
        (ox, k1), (og, k2) = guarded((r, c), dt), guarded((c,), FP32)
        zs.zs_rmsnorm_backward(dy.cuda(), h.cuda(), rstd.cuda(), gain.cuda(), ox, og, ws,
                               dres=None if dres is None else dres.cuda())
        assert k1() and k2()
        # the row's sum: at most 64 + 6 + 16 additions, and a handful of products
        acc = (64 + 6 + 16 + 8) * 2.0 ** -24 * mag
        close(ox, dx, U[dt] * (dx.abs() + acc) + acc + TINY[dt], "dx")
        # the gain's: r rows in some order of at most r + 32 additions
        close(og, dgain, (r + 32) * 2.0 ** -24 * gmag + 1e-37, "dgain")


def test_norm_backward_in_place_and_no_rows(zs):
    g = gen("nbi")
    h, dy, dres = (randn(g, 9, 520).to(BF16) for _ in range(3))
    gain, rstd = torch.ones(520, dtype=BF16).cuda(), torch.rand(9, generator=g).cuda() + 0.5
    ws = torch.empty(zs.zs_rmsnorm_backward_workspace(9, 520), dtype=torch.uint8, device="cuda")
    want, wg = torch.empty(9, 520, dtype=BF16, device="cuda"), torch.empty(520, device="cuda")
    zs.zs_rmsnorm_backward(dy.cuda(), h.cuda(), rstd, gain, want, wg, ws, dres=dres.cuda())
    for place in range(3):
        t = [dy.cuda(), h.cuda(), dres.cuda()]
        og = torch.empty(520, device="cuda")
        zs.zs_rmsnorm_backward(t[0], t[1], rstd, gain, t[place], og, ws, dres=t[2])
        assert torch.equal(t[place].view(torch.int16), want.view(torch.int16))
        assert torch.equal(og, wg)
    og.fill_(3.0)
    e = torch.empty(0, 520, dtype=BF16, device="cuda")
    zs.zs_rmsnorm_backward(e, e, rstd[:0], gain, e, og, None)
    assert not og.any()


# ---- distillation --------------------------------------------------------------

# (rows, vocabulary, slots)
DISTILL = [(1, 1, 1), (2, 7, 3), (3, 100, 0), (3, 1000, 5), (5, 1001, 64), (40, 2048, 32),
           (130, 4099, 7), (1, 50257, 32), (4, 50257, 100), (2, 131073, 20), (1, 200000, 300),
           (1100, 640, 9), (1030, 9001, 4)]


def distill_inputs(r, v, k, dt, tail, tau, seed=0):
    g = gen("d", r, v, k, seed)
    z = (randn(g, r, v) * 3).to(dt)
    ids = torch.randint(-1, v + 1, (r, k), generator=g, dtype=torch.int32)
    t = (randn(g, r, k) * 2).to(dt)
    if k > 3:
        ids[0, 1], ids[0, 2] = ids[0, 0], -5           # a token twice, an empty slot
        t[0, 3] = -math.inf
    if r > 2:
        ids[2] = -1                                    # a row without slots
    w = torch.rand(r, generator=g) + 0.1
    if r > 3:
        w[3] = 0.0
    lse = None
    if tail:
        kept = torch.where((ids >= 0) & (ids < v), t.double() / tau, -math.inf)
        kept = torch.cat([kept, torch.zeros(r, 1, dtype=F64)], 1)
        lse = (torch.logsumexp(kept, 1) + 0.2).float()
    return z, ids, t, w, lse


def distill_tolerance(z, bound, grad, dt, tau, q_scale=1.0):
    """exp's argument (z - max) / tau carries two roundings of 2^-24 of its
    size, and the exp, the sum (a chain of at most 200 terms per thread) and
    the products some 2^-21 together; a probability that small (beyond 60
    units below the top) no longer counts beside the smallest value."""
    arg = ((z.double().amax(1, keepdim=True) - z.double()) / tau).clamp(max=90)
    acc = bound * (arg * 2.0 ** -22 + 2.0 ** -19) * q_scale
    return U[dt] * (grad.abs() + acc) + acc + TINY[dt]


@pytest.mark.parametrize("dt", [BF16, FP16, FP32], ids=str)
@pytest.mark.parametrize("tail", [False, True])
def test_distill(zs, dt, tail):
    for r, v, k in DISTILL:
        tau = 1.0 if v % 2 else 2.0
        announce(f"distill {dt} tail={tail} {r}x{v} slots {k}")
        z, ids, t, w, lse = distill_inputs(r, v, k, dt, tail, tau)
        loss, grad, bound = ref.distill(z, ids, t, tau, lse, w, scale=64.0)
        ws = torch.empty(max(16, zs.zs_distill_workspace(r, v, k, zs._float_code(z, "z", True))),
                         dtype=torch.uint8, device="cuda")
        (ol, k1), (og, k2) = guarded((r,), FP32), guarded((r, v), dt)
        args = [x.cuda() for x in (z, ids, t)]
        more = dict(teacher_lse=None if lse is None else lse.cuda(), row_weight=w.cuda(),
                    loss_scale=64.0, workspace=ws)
        zs.zs_distill(*args, tau, ol, grad=og, **more)
        assert k1() and k2()
        # off the slots the tail's factor 1 - pr/qr can be large: its own size scales the error
        amp = 1.0
        if tail:
            amp = (grad.abs() / bound.clamp(min=1e-300)).amax(1, keepdim=True).clamp(min=1.0) * 4
        close(og, grad, distill_tolerance(z, bound, grad, dt, tau, amp), "grad")
        # the loss: terms of the size of the logits' spread, weighted by p
        size = ((z.double().amax(1) - z.double().amin(1)) / tau + 20) * w.double() * tau * tau
        close(ol, loss, size * 2.0 ** -20, "loss")
        only, k3 = guarded((r,), FP32)
        zs.zs_distill(*args, tau, only, **more)            # forward alone
        assert k3() and torch.equal(only, ol)
        inplace = args[0].clone()
        zs.zs_distill(inplace, *args[1:], tau, only, grad=inplace, **more)
        assert torch.equal(only, ol)
        i = torch.int32 if dt == FP32 else torch.int16
        assert torch.equal(inplace.view(i), og.contiguous().view(i))


@pytest.mark.parametrize("dt", [BF16, FP32], ids=str)
@pytest.mark.parametrize("tail", [False, True])
def test_distill_more_slots_than_threads(zs, dt, tail):
    """The shortest rows' blocks have 64 threads; the others of a row's slots come later."""
    for r, v, k in ((3, 900, 300), (70, 1000, 65), (2, 5000, 1024)):
        announce(f"distill {dt} tail={tail} {r}x{v} slots {k}")
        z, ids, t, w, lse = distill_inputs(r, v, k, dt, tail, 1.0)
        loss, grad, bound = ref.distill(z, ids, t, 1.0, lse, w, scale=64.0)
        ol, og = torch.empty(r, device="cuda"), torch.empty(r, v, dtype=dt, device="cuda")
        zs.zs_distill(z.cuda(), ids.cuda(), t.cuda(), 1.0, ol, grad=og, row_weight=w.cuda(),
                      teacher_lse=None if lse is None else lse.cuda(), loss_scale=64.0,
                      workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
        amp = 1.0
        if tail:
            amp = (grad.abs() / bound.clamp(min=1e-300)).amax(1, keepdim=True).clamp(min=1.0) * 4
        close(og, grad, distill_tolerance(z, bound, grad, dt, 1.0, amp), "grad")
        size = ((z.double().amax(1) - z.double().amin(1)) + 20) * w.double()
        close(ol, loss, size * 2.0 ** -20, "loss")


@pytest.mark.parametrize("dt,r,v,k,piece", [(BF16, 9000, 700, 5, 1000), (BF16, 2500, 16001, 130, 500),
                                            (FP32, 1200, 13000, 3, 250), (BF16, 700, 70003, 20, 100)],
                         ids=str)
@pytest.mark.parametrize("tail", [False, True])
def test_distill_more_rows_than_blocks(zs, dt, r, v, k, piece, tail):
    """Blocks that go on to further rows give the bits of calls with a row to a block."""
    announce(f"distill {dt} tail={tail} {r}x{v} slots {k}")
    g = gen("rows", r, v, k)
    z = torch.randn(r, v, device="cuda", generator=torch.Generator("cuda").manual_seed(7)).to(dt)
    ids = torch.randint(-1, v, (r, k), generator=g, dtype=torch.int32).cuda()
    t = randn(g, r, k).to(dt).cuda()
    w = torch.randint(0, 4, (r,), generator=g).float().cuda()   # a quarter of the rows is skipped
    lse = (torch.logsumexp(t.float(), 1) + 0.2) if tail else None
    i = torch.int32 if dt == FP32 else torch.int16
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def run(z, ids, t, w, lse, grad):
        loss = torch.empty(z.shape[0], device="cuda")
        zs.zs_distill(z, ids, t, 1.0, loss, grad=grad, teacher_lse=lse, row_weight=w, workspace=ws)
        return loss

    grad = torch.full_like(z, 7.0)
    loss = run(z, ids, t, w, lse, grad)
    assert torch.equal(run(z, ids, t, w, lse, None), loss)
    whole = torch.full_like(z, 7.0)   # a gradient aligned unlike its logits takes another kernel
    for a in range(0, r, piece):
        b = min(a + piece, r)
        part = whole[a:b]
        ol = run(z[a:b], ids[a:b], t[a:b], w[a:b], None if lse is None else lse[a:b], part)
        assert torch.equal(ol, loss[a:b]), a
        assert torch.equal(part.view(i), grad[a:b].view(i)), a
    inplace = z.clone()
    assert torch.equal(run(inplace, ids, t, w, lse, inplace), loss)
    assert torch.equal(inplace.view(i), grad.view(i))
    assert bool(torch.isfinite(loss).all()) and not bool(grad[w == 0].any())


@pytest.mark.parametrize("dt", [BF16, FP32], ids=str)
def test_distill_strided_rows(zs, dt):
    """Logits and gradient in wider buffers, at offsets of their own."""
    for r, v, ld, off, gld, goff in ((3, 1000, 1008, 8, 1008, 8), (5, 999, 1003, 1, 1003, 1),
                                     (4, 640, 701, 3, 650, 2)):
        z, ids, t, w, _ = distill_inputs(r, v, 6, dt, False, 1.0)
        loss, grad, bound = ref.distill(z, ids, t, 1.0, None, w, scale=4.0)
        zraw = torch.full((r * ld + 16,), math.nan, dtype=dt, device="cuda")
        graw = torch.full((r * gld + 16,), 7.0, dtype=dt, device="cuda")
        zv = zraw[off:off + r * ld].view(r, ld)[:, :v]
        gv = graw[goff:goff + r * gld].view(r, gld)[:, :v]
        zv.copy_(z)
        ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        ol = torch.empty(r, device="cuda")
        zs.zs_distill(zv, ids.cuda(), t.cuda(), 1.0, ol, grad=gv, row_weight=w.cuda(),
                      loss_scale=4.0, workspace=ws)
        close(gv, grad, distill_tolerance(z, bound, grad, dt, 1.0), f"ld {ld}")
        keep = torch.ones_like(graw, dtype=torch.bool)
        keep[goff:goff + r * gld].view(r, gld)[:, :v] = False
        assert bool((graw[keep] == 7.0).all())


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("v", [700, 40000])
def test_distill_masked_and_non_finite_logits(zs, tail, v):
    r, k = 9, 4
    z, ids, t, w, lse = distill_inputs(r, v, k, FP32, tail, 1.0)
    w[:] = 1.0
    ids[:] = torch.tensor([1, 5, 9, 600])
    t[:] = torch.tensor([1.0, 0.5, -1.0, 0.0])
    if tail:
        lse[:] = torch.logsumexp(t[0], 0) + 0.3
    low = torch.finfo(FP32).min
    z[0, 100:] = -math.inf
    z[0, 600] = 0.0                                    # a masked vocabulary
    z[1, 5] = -math.inf                                # the teacher's token is masked
    z[2, 50] = math.nan
    z[3, 50] = math.inf
    z[4] = -math.inf
    z[5, 100:] = low
    z[5, 600] = 0.0
    z[6] = math.nan
    w[6] = 0.0                                         # weight 0: nothing of it comes through
    t[7] = -math.inf                                   # no mass on the slots
    z[8, 9], t[8, 2] = -math.inf, -math.inf            # masked, and without mass: no contribution
    ol, og = torch.empty(r, device="cuda"), torch.empty(r, v, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    zs.zs_distill(z.cuda(), ids.cuda(), t.cuda(), 1.0, ol, grad=og, row_weight=w.cuda(),
                  teacher_lse=None if lse is None else lse.cuda(), workspace=ws)
    loss, grad, bound = ref.distill(z, ids, t, 1.0, lse, w)
    ol, og = ol.cpu(), og.cpu()
    assert torch.isnan(og[2]).all() and torch.isnan(og[3]).all() and torch.isnan(og[4]).all()
    assert torch.isnan(ol[2]) and torch.isnan(ol[3]) and torch.isnan(ol[4])
    assert ol[6] == 0 and not og[6].any()
    assert ol[1] == math.inf and torch.isfinite(og[1]).all()
    if not tail:
        assert ol[7] == 0 and not og[7].any()
    fine = [0, 1, 5, 7, 8]
    amp = 1.0
    if tail:
        amp = (grad.abs() / bound.clamp(min=1e-300)).amax(1, keepdim=True).clamp(min=1.0)[fine] * 4
    zf = torch.where(z[fine] < -1e30, -90.0, z[fine].double())
    close(og[fine], grad[fine], distill_tolerance(zf, bound[fine], grad[fine], FP32, 1.0, amp), "grad")
    close(ol[fine], loss[fine], 120 * 2.0 ** -20, "loss")
    # a masked token gets the gradient 0, not NaN
    assert not og[0, 100:600].any() and not og[5, 100:600].any()


def test_distill_all_mass_on_the_slots(zs):
    """The tail's mass vanishes on either side."""
    v = 300
    z = torch.full((3, v), -200.0)
    ids = torch.tensor([[3, 8]] * 3, dtype=torch.int32)
    z[:, 3], z[:, 8] = 1.0, 2.0
    z[2] = 0.0
    t = torch.tensor([[1.0, 2.0]] * 3)
    lse = torch.logsumexp(t, 1) + torch.tensor([0.0, 0.5, 0.0])
    ol, og = torch.empty(3, device="cuda"), torch.empty(3, v, device="cuda")
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    zs.zs_distill(z.cuda(), ids.cuda(), t.cuda(), 1.0, ol, grad=og, teacher_lse=lse.cuda(),
                  workspace=ws)
    assert abs(float(ol[0])) < 1e-5 and float(ol[1]) == math.inf
    assert not torch.isnan(og).any() and float(og[:2].abs()[:, 10:].max()) == 0.0
    want = ref.distill(z, ids, t, 1.0, lse)
    close(ol[2:], want[0][2:], 1e-5, "loss")


def test_distill_scale_from_the_device(zs):
    """The device scaler's scale, and a gradient that overflows: data, not an error."""
    z, ids, t, w, _ = distill_inputs(4, 500, 5, FP16, False, 1.0)
    z, ids, t = z.cuda(), ids.cuda(), t.cuda()
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    ol = torch.empty(4, device="cuda")
    out = {}
    for scale in (512.0, 2.0 ** 40):
        image = zs.zs_device_scaler_make(zs.zs_loss_scaler(scale=scale, dynamic=1), 0.9, 0.999)
        dev = zs.device_scaler_upload(image)
        a, b = torch.empty_like(z), torch.empty_like(z)
        zs.zs_distill(z, ids, t, 1.0, ol, grad=a, dev_scaler=dev, workspace=ws)
        zs.zs_distill(z, ids, t, 1.0, ol, grad=b, loss_scale=scale, workspace=ws)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        out[scale] = a
    assert torch.isfinite(out[512.0]).all() and torch.isinf(out[2.0 ** 40]).any()


@pytest.mark.parametrize("tail", [False, True])
def test_distill_gradient_against_differences(zs, tail):
    """The kernel's own loss, in central differences of 2^-6: their own error
    is below 2^-12 / 6 of the third derivative (at most 1 here), and 2^-20 of
    the loss (at most 8) over the difference."""
    r, v, k, d = 1, 40, 6, 2.0 ** -6
    z, ids, t, _, lse = distill_inputs(r, v, k, FP32, tail, 1.0, seed=1)
    zz = z.repeat(2 * v, 1)
    for j in range(v):
        zz[2 * j, j] += d
        zz[2 * j + 1, j] -= d
    many = [x.repeat(2 * v, 1).cuda() for x in (ids, t)]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    ol, og, o1 = torch.empty(2 * v, device="cuda"), torch.empty(1, v, device="cuda"), torch.empty(
        1, device="cuda")
    zs.zs_distill(zz.cuda(), *many, 1.0, ol, workspace=ws,
                  teacher_lse=None if lse is None else lse.repeat(2 * v).cuda())
    zs.zs_distill(z.cuda(), ids.cuda(), t.cuda(), 1.0, o1, grad=og, workspace=ws,
                  teacher_lse=None if lse is None else lse.cuda())
    diff = (ol[0::2] - ol[1::2]).double().cpu() / (zz[0::2].diagonal() - zz[1::2].diagonal()).double()
    close(og[0], diff, 2.0 ** -12 / 6 + 2 * 8 * 2.0 ** -20 / (2 * d), "differences")


def test_distill_rows_past_32_bits(zs):
    big = torch.empty(2 * (1 << 31) + 64, dtype=BF16, device="cuda")
    z, ids, t, w, _ = distill_inputs(3, 64, 4, BF16, False, 1.0)
    ids[2] = ids[1]
    view = big.as_strided((3, 64), (1 << 31, 1))
    view.copy_(z)
    loss, grad, bound = ref.distill(z, ids, t, 1.0)
    ol = torch.empty(3, device="cuda")
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    zs.zs_distill(view, ids.cuda(), t.cuda(), 1.0, ol, grad=view, workspace=ws)
    close(view, grad, distill_tolerance(z, bound, grad, BF16, 1.0), "grad")


# ---- streams and graphs ----------------------------------------------------------

def all_operators(zs, g, rows=70, width=320, vocab=515):
    """Buffers of one head's pass, and a function that queues all of it on a stream."""
    dev = dict(device="cuda")
    x, res = ((torch.randn(rows, width, generator=g)).to(BF16).cuda() for _ in range(2))
    gain, weight = torch.ones(width, dtype=BF16, **dev), torch.randn(vocab, width, generator=g).cuda()
    ids = torch.randint(0, vocab, (rows, 8), generator=g, dtype=torch.int32).cuda()
    t = torch.randn(rows, 8, generator=g).to(BF16).cuda()
    out = {"h": torch.empty_like(x), "rstd": torch.empty(rows, **dev),
           "logits": torch.empty(rows, vocab, dtype=BF16, **dev), "loss": torch.empty(rows, **dev),
           "dlogits": torch.empty(rows, vocab, dtype=BF16, **dev), "dy": torch.empty_like(x),
           "dw": torch.empty(vocab, width, dtype=BF16, **dev), "dx": torch.empty_like(x),
           "dgain": torch.empty(width, **dev)}
    E2, E4 = zs.ZS_MX_E2M1, zs.ZS_MX_E4M3
    y, w, wt = (zs.mx_empty(rows, width, E4), zs.mx_empty(vocab, width, E2),
                zs.mx_empty(width, vocab, E2))
    d, dt, xt = (zs.mx_empty(rows, vocab, E4), zs.mx_empty(vocab, rows, E4),
                 zs.mx_empty(width, rows, E2))
    ws = torch.empty(32 << 20, dtype=torch.uint8, **dev)

    def queue(stream=None):
        s = dict(stream=stream)
        zs.zs_rmsnorm_forward(x, gain, 1e-5, h=out["h"], rstd=out["rstd"], residual=res, codes=y[0],
                              scales=y[1], **s)
        zs.zs_mx_quantize(weight, E2, *w, **s)
        zs.zs_mx_matmul(*y, E4, *w, out["logits"], width, workspace=ws, **s)
        zs.zs_distill(out["logits"], ids, t, 2.0, out["loss"], grad=out["dlogits"],
                      loss_scale=256.0, workspace=ws, **s)
        zs.zs_mx_quantize(out["dlogits"], E4, *d, **s)
        zs.zs_mx_quantize(weight, E2, *wt, columns=True, **s)
        zs.zs_mx_matmul(*d, E4, *wt, out["dy"], vocab, workspace=ws, **s)
        zs.zs_mx_quantize(out["dlogits"], E4, *dt, columns=True, **s)
        zs.zs_mx_quantize(out["h"], E2, *xt, columns=True, **s)
        zs.zs_mx_matmul(*dt, E4, *xt, out["dw"], rows, workspace=ws, **s)
        zs.zs_rmsnorm_backward(out["dy"], out["h"], out["rstd"], gain, out["dx"], out["dgain"], ws,
                               **s)

    return (x, weight), out, queue


def same(a, b):
    return all(torch.equal(a[k], b[k]) for k in a)


def test_operators_on_another_stream(zs):
    _, out, queue = all_operators(zs, gen("streams"))
    queue()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in out.items()}
    for v in out.values():
        v.fill_(1.0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    queue(side)
    side.synchronize()
    assert same(out, want)
    assert all(torch.isfinite(v.float()).all() for v in want.values())


def test_operators_in_a_graph(zs):
    """Replays, with eager work between them and new inputs in the same buffers."""
    (x, weight), out, queue = all_operators(zs, gen("graph"))
    queue()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            queue()
    torch.cuda.current_stream().wait_stream(side)
    for i in range(4):
        x.add_(0.25 * i)
        weight.mul_(1.5)
        queue()
        torch.cuda.synchronize()
        want = {k: v.clone() for k, v in out.items()}
        for v in out.values():
            v.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want), f"replay {i}"


@pytest.mark.parametrize("dt", [BF16, FP16, FP32], ids=str)
def test_distill_small_temperatures_and_large_logits(zs, dt):
    """Exponents far beyond 2^24 units: the largest logit's neighbours have nothing, but of fp32
    some, and ties share. A term's exponent is off by 2^-24 of itself, and of 128 where its whole
    number is as far away: 2^-15 of the terms that matter; below 2^-126 they are 0."""
    sizes = [(1e-6, 1), (1e-8, 1), (1e-9, 1), (1e-12, 1), (1e-18, 1)]
    if dt is not FP16:
        sizes += [(1.0, 3e7), (1.0, 1e9), (1.0, 1e13), (1.0, 1e17)]
    for r, v in ((5, 1000), (3, 70000), (2, 140001)):
        for tau, size in sizes:
            announce(f"distill cold {dt} {tau} {size} {r}x{v}")
            g = gen("cold", r, v, tau, size)
            z = (2 * size * torch.randn(r, v, generator=g)).to(dt)
            if dt is FP32:
                z[1, torch.randint(0, v, (3,), generator=g)] = torch.nextafter(
                    z[1].max(), torch.tensor(-math.inf))
            ids = torch.stack([torch.randperm(v, generator=g)[:5] for _ in range(r)]).int()
            ids[0, 2], ids[1, 0] = int(z[0].float().argmax()), int(z[1].float().argmax())
            t = torch.stack([torch.randperm(8, generator=g)[:5] * 0.5 for _ in range(r)]).to(dt)
            tau32, scale = float(torch.tensor(tau)), 64.0 / float(torch.tensor(tau))
            loss, grad, bound = ref.distill(z, ids, t, tau32, None, None, scale=scale)
            ol, og = torch.full((r,), 9.0, device="cuda"), torch.full_like(z, 7.0).cuda()
            ws = torch.empty(max(16, zs.zs_distill_workspace(r, v, 5, zs._float_code(z, "z", True))),
                             dtype=torch.uint8, device="cuda")
            zs.zs_distill(z.cuda(), ids.cuda(), t.cuda(), tau, ol, grad=og, loss_scale=scale,
                          workspace=ws)
            close(og, grad, U[dt] * grad.abs() + 2.0 ** -14 * bound + 64 * 2.0 ** -125, "grad")
            close(ol, loss, 2.0 ** -18 * loss.abs() + tau32 ** 2 * 2.0 ** -13, "loss")
