"""The output end's operators on the CPU: argument errors return before
anything is enqueued, and the plain 64-bit forms that the GPU tests compare
with agree with themselves, with torch and with differences. No GPU work."""
import ctypes as C
import math

import pytest
import torch

import ops_reference as ref

FAKE = 0x7F0000000000
P = C.c_void_p


@pytest.fixture(scope="module")
def zs(hip_built):
    from sharded_mixed_precision_zs_amd import zeroshard
    return zeroshard


def far(i, off=0):
    """Address i of several that lie 2^40 bytes apart."""
    return P(FAKE + (i << 40) + off)


def calls(zs):
    """One valid argument list per entry point, with zero rows where that
    enqueues nothing, and positions by name."""
    lib = zs._lib
    return {
        "quantize": (lib.zs_mx_quantize, dict(
            src=far(0), dtype=0, rows=8, cols=64, ld=64, fmt=0, columns=0, codes=far(1),
            scales=far(2), values=far(3), vdt=0, stream=None)),
        "matmul": (lib.zs_mx_matmul, dict(
            a=far(0), as_=far(1), fmt=1, b=far(2), bs=far(3), m=8, n=8, k=64, c=far(4), cdt=0,
            ldc=8, ws=None, wsb=0, stream=None)),
        "forward": (lib.zs_rmsnorm_forward, dict(
            x=far(0), res=far(1), gain=far(2), dtype=0, rows=8, cols=64, eps=1e-5, h=far(3),
            rstd=far(4), codes=far(5), scales=far(6), y=far(7), stream=None)),
        "backward": (lib.zs_rmsnorm_backward, dict(
            dy=far(0), h=far(1), rstd=far(2), gain=far(3), dres=far(4), dtype=0, rows=8, cols=64,
            dx=far(5), dgain=far(6), ws=far(7), wsb=1 << 20, stream=None)),
        "distill": (lib.zs_distill, dict(
            z=far(0), dtype=0, rows=8, vocab=100, ld=100, ids=far(1), teacher=far(2), slots=4,
            tau=1.0, lse=None, weight=None, scale=1.0, dev=None, loss=far(3), grad=far(4),
            gld=100, ws=far(5), wsb=1 << 20, stream=None)),
    }


INVALID, UNSUPPORTED, ALIAS = 1, 2, 3
BAD = [
    ("quantize", dict(src=None), INVALID), ("quantize", dict(codes=None), INVALID),
    ("quantize", dict(scales=None), INVALID), ("quantize", dict(dtype=3), INVALID),
    ("quantize", dict(dtype=-1), INVALID), ("quantize", dict(vdt=2), INVALID),
    ("quantize", dict(fmt=2), INVALID), ("quantize", dict(ld=63), INVALID),
    ("quantize", dict(codes=far(1, 8)), UNSUPPORTED), ("quantize", dict(scales=far(2, 2)), UNSUPPORTED),
    ("quantize", dict(rows=1 << 49), UNSUPPORTED), ("quantize", dict(rows=1 << 30, ld=1 << 30), UNSUPPORTED),
    ("quantize", dict(rows=1 << 24, columns=1, values=None), UNSUPPORTED),
    ("quantize", dict(src=far(0, 1)), UNSUPPORTED), ("quantize", dict(values=far(3, 1)), UNSUPPORTED),
    ("quantize", dict(src=far(0, 2), dtype=2), UNSUPPORTED),
    ("quantize", dict(codes=far(0, 512)), ALIAS), ("quantize", dict(values=far(0)), ALIAS),
    ("quantize", dict(values=far(1, 16)), ALIAS),
    ("matmul", dict(a=None), INVALID), ("matmul", dict(bs=None), INVALID),
    ("matmul", dict(c=None), INVALID), ("matmul", dict(fmt=7), INVALID),
    ("matmul", dict(cdt=5), INVALID), ("matmul", dict(ldc=7), INVALID),
    ("matmul", dict(cdt=2), UNSUPPORTED), ("matmul", dict(m=1 << 31), UNSUPPORTED),
    ("matmul", dict(n=1 << 31, ldc=1 << 31), UNSUPPORTED), ("matmul", dict(k=1 << 31), UNSUPPORTED),
    ("matmul", dict(a=far(0, 8)), UNSUPPORTED), ("matmul", dict(b=far(2, 4)), UNSUPPORTED),
    ("matmul", dict(as_=far(1, 1)), UNSUPPORTED), ("matmul", dict(c=far(4, 1)), UNSUPPORTED),
    ("matmul", dict(c=far(0)), ALIAS), ("matmul", dict(c=far(3)), ALIAS),
    ("matmul", dict(ws=far(4), wsb=64), ALIAS), ("matmul", dict(ws=far(5, 8), wsb=64), UNSUPPORTED),
    ("forward", dict(x=None), INVALID), ("forward", dict(gain=None), INVALID),
    ("forward", dict(h=None), INVALID), ("forward", dict(codes=None), INVALID),
    ("forward", dict(scales=None), INVALID), ("forward", dict(codes=None, scales=None, y=None), INVALID),
    ("forward", dict(dtype=2), INVALID), ("forward", dict(eps=-1.0), INVALID),
    ("forward", dict(eps=math.nan), INVALID), ("forward", dict(eps=math.inf), INVALID),
    ("forward", dict(cols=65537), UNSUPPORTED), ("forward", dict(rows=1 << 49), UNSUPPORTED),
    ("forward", dict(codes=far(5, 8)), UNSUPPORTED),
    ("forward", dict(x=far(0, 1)), UNSUPPORTED), ("forward", dict(res=far(1, 1)), UNSUPPORTED),
    ("forward", dict(gain=far(2, 1)), UNSUPPORTED), ("forward", dict(h=far(3, 1)), UNSUPPORTED),
    ("forward", dict(rstd=far(4, 2)), UNSUPPORTED), ("forward", dict(y=far(7, 1)), UNSUPPORTED),
    ("forward", dict(y=far(0)), ALIAS), ("forward", dict(h=far(0, 64)), ALIAS),
    ("forward", dict(rstd=far(2)), ALIAS), ("forward", dict(codes=far(7)), ALIAS),
    ("backward", dict(dy=None), INVALID), ("backward", dict(h=None), INVALID),
    ("backward", dict(rstd=None), INVALID), ("backward", dict(gain=None), INVALID),
    ("backward", dict(dx=None), INVALID), ("backward", dict(dgain=None), INVALID),
    ("backward", dict(ws=None), INVALID), ("backward", dict(wsb=8 * 64 * 4 - 1), INVALID),
    ("backward", dict(dtype=2), INVALID), ("backward", dict(cols=65537), UNSUPPORTED),
    ("backward", dict(ws=far(7, 2)), UNSUPPORTED),
    ("backward", dict(dy=far(0, 1)), UNSUPPORTED), ("backward", dict(dres=far(4, 1)), UNSUPPORTED),
    ("backward", dict(rstd=far(2, 2)), UNSUPPORTED), ("backward", dict(dgain=far(6, 2)), UNSUPPORTED),
    ("backward", dict(dx=far(0, 16)), ALIAS), ("backward", dict(dgain=far(5)), ALIAS),
    ("backward", dict(ws=far(1)), ALIAS), ("backward", dict(dgain=far(3)), ALIAS),
    ("distill", dict(z=None), INVALID), ("distill", dict(ids=None), INVALID),
    ("distill", dict(teacher=None), INVALID), ("distill", dict(loss=None), INVALID),
    ("distill", dict(dtype=3), INVALID), ("distill", dict(tau=0.0), INVALID),
    ("distill", dict(tau=math.inf), INVALID), ("distill", dict(tau=math.nan), INVALID),
    ("distill", dict(scale=0.0), INVALID), ("distill", dict(scale=math.inf), INVALID),
    ("distill", dict(vocab=0), INVALID), ("distill", dict(ld=99), INVALID),
    ("distill", dict(gld=99), INVALID), ("distill", dict(vocab=1 << 31, ld=1 << 31, gld=1 << 31), INVALID),
    ("distill", dict(slots=1025), UNSUPPORTED), ("distill", dict(rows=1 << 49), UNSUPPORTED),
    ("distill", dict(z=far(0, 1)), UNSUPPORTED), ("distill", dict(grad=far(4, 1)), UNSUPPORTED),
    ("distill", dict(dev=far(6, 4)), UNSUPPORTED),
    ("distill", dict(ids=far(1, 2)), UNSUPPORTED), ("distill", dict(teacher=far(2, 1)), UNSUPPORTED),
    ("distill", dict(loss=far(3, 2)), UNSUPPORTED), ("distill", dict(lse=far(6, 2)), UNSUPPORTED),
    ("distill", dict(weight=far(6, 2)), UNSUPPORTED),
    ("distill", dict(grad=far(0, 2)), ALIAS), ("distill", dict(grad=far(0), gld=101), ALIAS),
    ("distill", dict(loss=far(0)), ALIAS), ("distill", dict(grad=far(2)), ALIAS),
    ("distill", dict(loss=far(4)), ALIAS),
]


@pytest.mark.parametrize("name,change,status", BAD,
                         ids=[f"{n}-{'-'.join(c)}-{i}" for i, (n, c, _) in enumerate(BAD)])
def test_bad_arguments_are_refused(zs, name, change, status):
    fn, args = calls(zs)[name]
    assert set(change) <= set(args)
    assert fn(*{**args, **change}.values()) == status
    assert zs.zs_last_error()


@pytest.mark.parametrize("name,change", [
    ("quantize", dict(rows=1 << 27, cols=1024, ld=1024, values=None)),
    ("matmul", dict(m=1, n=1 << 29, ldc=1 << 29)),
    ("matmul", dict(m=1 << 26, n=1 << 13, ldc=1 << 13)),
    ("forward", dict(rows=1 << 27)),
    ("distill", dict(rows=1 << 31, vocab=16, ld=16, gld=16, wsb=1 << 36)),
    ("distill", dict(rows=1 << 26, vocab=5, ld=5, gld=5, wsb=1 << 36)),
])
def test_more_threads_than_a_launch_has_are_refused(zs, name, change):
    fn, args = calls(zs)[name]
    assert fn(*{**args, **change}.values()) == UNSUPPORTED


def test_a_workspace_too_small_is_refused(zs):
    need = zs.zs_distill_workspace(8, 1 << 20, 4, zs.ZS_FP32)
    assert need > 0
    fn, args = calls(zs)["distill"]
    big = dict(args, dtype=2, vocab=1 << 20, ld=1 << 20, gld=1 << 20)
    assert fn(*{**big, "wsb": need - 1}.values()) == zs.ZS_ERR_INVALID_ARG
    assert fn(*{**big, "ws": None, "wsb": 0}.values()) == zs.ZS_ERR_INVALID_ARG
    assert fn(*{**big, "ws": far(5, 8), "wsb": need}.values()) == zs.ZS_ERR_UNSUPPORTED
    assert fn(*{**big, "ws": far(4, 64), "wsb": need}.values()) == zs.ZS_ERR_ALIAS


def test_workspaces_by_size(zs):
    assert zs.zs_mx_matmul_workspace(1, 32000, 4096) == 0          # the thin kernel
    assert zs.zs_mx_matmul_workspace(8192, 8192, 8192) == 0        # tiles enough
    assert zs.zs_mx_matmul_workspace(768, 768, 512) == 0           # nothing to split
    assert zs.zs_mx_matmul_workspace(768, 768, 8192) == 6 * 768 * 768 * 4   # 64 groups in pieces of 12
    assert zs.zs_mx_matmul_workspace(0, 5, 8192) == 0
    assert zs.zs_rmsnorm_backward_workspace(10, 100) == 10 * 100 * 4
    assert zs.zs_rmsnorm_backward_workspace(1 << 30, 100) == 1024 * 100 * 4
    assert zs.zs_distill_workspace(0, 100, 4, zs.ZS_BF16) == 0


@pytest.mark.parametrize("name,change", [
    ("quantize", dict(rows=0)), ("quantize", dict(cols=0)), ("matmul", dict(m=0)),
    ("matmul", dict(n=0)), ("forward", dict(rows=0)), ("forward", dict(cols=0)),
    ("backward", dict(cols=0)), ("distill", dict(rows=0))])
def test_empty_calls_do_nothing(zs, name, change):
    fn, args = calls(zs)[name]
    assert fn(*{**args, **change}.values()) == zs.ZS_OK


def test_binding_checks_its_tensors(zs):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        zs.zs_mx_quantize(x, zs.ZS_MX_E2M1, x, x)
    with pytest.raises(ValueError):
        zs.zs_rmsnorm_forward(x.bfloat16(), x[0].bfloat16(), 1e-5, y=x.bfloat16())
    assert zs.mx_shapes(5, 130, zs.ZS_MX_E2M1) == ((5, 128), (5, 8))
    assert zs.mx_shapes(5, 128, zs.ZS_MX_E4M3) == ((5, 128), (5, 4))


# ---- the plain forms themselves ------------------------------------------------

@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_reference_codes_stand_for_the_nearest_values(fmt):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(7, 200, generator=g, dtype=torch.float64) * torch.exp(
        torch.randn(7, 1, generator=g, dtype=torch.float64) * 5)
    codes, byte, val = ref.mx_quantize(x, fmt)
    assert torch.equal(ref.mx_values(codes, byte, fmt, 200), val)
    if fmt == "e4m3":
        assert torch.equal(codes.view(torch.float8_e4m3fn).double()[:, :200]
                           * ref.pow2(byte.long() - 127).repeat_interleave(32, 1)[:, :200], val)
    # nearest: no other code of the block's scale is closer
    s = ref.pow2(byte.long() - 127).repeat_interleave(32, 1)[:, :200]
    every = torch.arange(127 if fmt == "e4m3" else 8)
    grid = every.to(torch.uint8).view(torch.float8_e4m3fn).double() if fmt == "e4m3" else ref.GRID
    best = (x.abs().unsqueeze(2) - grid * s.unsqueeze(2)).abs().amin(2)
    assert torch.equal((val.abs() - x.abs()).abs(), best)


def test_reference_blocks_that_are_not_finite():
    x = torch.ones(3, 64, dtype=torch.float64)
    x[0, 3], x[1, 40], x[2] = math.inf, math.nan, 0.0
    codes, byte, val = ref.mx_quantize(x, "e4m3")
    assert byte.tolist() == [[255, 119, 1, 1], [119, 255, 1, 1], [1, 1, 1, 1]]
    assert torch.isnan(val[0, :32]).all() and torch.isnan(val[1, 32:]).all()
    assert not codes[0, :32].any() and not val[2].any()


def test_reference_norm_gradient_against_differences():
    g = torch.Generator().manual_seed(5)
    h, dy, gain = (torch.randn(*s, generator=g, dtype=torch.float64)
                   for s in ((3, 10), (3, 10), (10,)))
    dres, eps, d = torch.randn(3, 10, generator=g, dtype=torch.float64), 1e-5, 1e-6

    def f(h, gain):
        return (ref.rmsnorm(h, gain, eps)[0] * dy).sum() + (h * dres).sum()

    dx, dgain, _, _ = ref.rmsnorm_grad(dy, h, ref.rmsnorm(h, gain, eps)[1], gain, dres)
    for i in range(3):
        for j in range(10):
            e = torch.zeros(3, 10, dtype=torch.float64)
            e[i, j] = d
            assert abs(float(f(h + e, gain) - f(h - e, gain)) / (2 * d) - float(dx[i, j])) < 1e-7
    for j in range(10):
        e = torch.zeros(10, dtype=torch.float64)
        e[j] = d
        assert abs(float(f(h, gain + e) - f(h, gain - e)) / (2 * d) - float(dgain[j])) < 1e-7


@pytest.mark.parametrize("tail", [False, True])
def test_reference_distill_gradient_against_differences(tail):
    g = torch.Generator().manual_seed(6)
    z = torch.randn(2, 12, generator=g, dtype=torch.float64)
    ids = torch.tensor([[3, 7, -1, 3], [0, 11, 5, 12]])
    t = torch.randn(2, 4, generator=g, dtype=torch.float64)
    tau, d = 1.7, 1e-6
    lse = torch.logsumexp(t / tau, 1) + 0.4 if tail else None
    w = torch.tensor([0.5, 2.0])
    loss, grad, _ = ref.distill(z, ids, t, tau, lse, w, scale=8.0)
    assert (loss > -1e-12).all() or tail
    for i in range(2):
        for j in range(12):
            e = torch.zeros_like(z)
            e[i, j] = d
            up, dn = (ref.distill(z + s * e, ids, t, tau, lse, w)[0].sum() for s in (1, -1))
            # the loss carries temperature^2 and its gradient by z one temperature less
            assert abs(float(up - dn) / (2 * d) * 8.0 - float(grad[i, j])) < 1e-6


def test_reference_distill_full_vocabulary_is_kl():
    g = torch.Generator().manual_seed(7)
    z, t = (torch.randn(3, 20, generator=g, dtype=torch.float64) for _ in range(2))
    ids = torch.arange(20).expand(3, 20)
    loss, grad, _ = ref.distill(z, ids, t, 2.0)
    want = torch.nn.functional.kl_div(torch.log_softmax(z / 2, 1), torch.log_softmax(t / 2, 1),
                                      reduction="none", log_target=True).sum(1) * 4
    assert torch.allclose(loss, want, rtol=1e-12)
    assert torch.allclose(grad, 2 * (torch.softmax(z / 2, 1) - torch.softmax(t / 2, 1)), atol=1e-14)
