"""The product with an epilogue on the CPU: argument errors return before anything
is enqueued, and the plain 64-bit forms that the GPU tests compare with against
torch, autograd and differences. No GPU work."""
import ctypes as C
import math

import pytest
import torch

import linear_reference as ref

FAKE = 0x7F0000000000
P = C.c_void_p
F64 = torch.float64
INVALID, UNSUPPORTED, ALIAS = 1, 2, 3


@pytest.fixture(scope="module")
def zs(hip_built):
    from sharded_mixed_precision_zs_amd import zeroshard
    return zeroshard


def far(i, off=0):
    """Address i of several that lie 2^40 bytes apart."""
    return P(FAKE + (i << 40) + off)


def calls(zs):
    """One argument list per entry point that only its changes make invalid."""
    lib = zs._lib
    return {
        "linear": (lib.zs_mx_linear, dict(
            a=far(0), as_=far(1), fmt=1, b=far(2), bs=far(3), m=8, n=8, k=64, bias=far(4), act=2,
            res=far(5), ldr=8, pre=far(6), c=far(7), cdt=0, ldc=8, ws=None, wsb=0, stream=None)),
        "backward": (lib.zs_activation_backward, dict(
            dc=far(0), pre=far(1), act=2, dtype=0, rows=8, cols=64, dpre=far(2), dbias=far(3),
            ws=far(4), wsb=1 << 20, stream=None)),
    }


BAD = [
    ("linear", dict(a=None), INVALID), ("linear", dict(as_=None), INVALID),
    ("linear", dict(b=None), INVALID), ("linear", dict(bs=None), INVALID),
    ("linear", dict(c=None), INVALID), ("linear", dict(fmt=2), INVALID),
    ("linear", dict(act=4), INVALID), ("linear", dict(act=-1), INVALID),
    ("linear", dict(cdt=2), INVALID), ("linear", dict(ldc=7), INVALID),
    ("linear", dict(ldr=7), INVALID), ("linear", dict(m=1 << 31), UNSUPPORTED),
    ("linear", dict(k=(1 << 22) + 1), UNSUPPORTED),
    ("linear", dict(n=1 << 31, ldc=1 << 31, ldr=1 << 31), UNSUPPORTED),
    ("linear", dict(a=far(0, 8)), UNSUPPORTED), ("linear", dict(bs=far(3, 1)), UNSUPPORTED),
    ("linear", dict(bias=far(4, 1)), UNSUPPORTED), ("linear", dict(res=far(5, 1)), UNSUPPORTED),
    ("linear", dict(pre=far(6, 1)), UNSUPPORTED), ("linear", dict(c=far(7, 1)), UNSUPPORTED),
    ("linear", dict(ws=far(8, 8), wsb=64), UNSUPPORTED),
    ("linear", dict(c=far(0)), ALIAS), ("linear", dict(pre=far(2)), ALIAS),
    ("linear", dict(c=far(5, 2)), ALIAS), ("linear", dict(c=far(5), ldc=9), ALIAS),
    ("linear", dict(pre=far(5)), ALIAS), ("linear", dict(pre=far(7)), ALIAS),
    ("linear", dict(c=far(4)), ALIAS), ("linear", dict(ws=far(7), wsb=64), ALIAS),
    ("linear", dict(ws=far(6), wsb=64), ALIAS), ("linear", dict(ws=far(4), wsb=64), ALIAS),
    ("backward", dict(dc=None), INVALID), ("backward", dict(pre=None), INVALID),
    ("backward", dict(dpre=None, dbias=None), INVALID), ("backward", dict(act=9), INVALID),
    ("backward", dict(dtype=2), INVALID), ("backward", dict(ws=None), INVALID),
    ("backward", dict(wsb=16), INVALID), ("backward", dict(cols=1 << 31), UNSUPPORTED),
    ("backward", dict(rows=1 << 49), UNSUPPORTED), ("backward", dict(dc=far(0, 1)), UNSUPPORTED),
    ("backward", dict(pre=far(1, 1)), UNSUPPORTED), ("backward", dict(dpre=far(2, 1)), UNSUPPORTED),
    ("backward", dict(dbias=far(3, 2)), UNSUPPORTED), ("backward", dict(ws=far(4, 2)), UNSUPPORTED),
    ("backward", dict(dpre=far(0, 2)), ALIAS), ("backward", dict(dbias=far(1)), ALIAS),
    ("backward", dict(dbias=far(2)), ALIAS), ("backward", dict(ws=far(0)), ALIAS),
]


@pytest.mark.parametrize("name,change,status", BAD,
                         ids=[f"{n}-{'-'.join(c)}-{i}" for i, (n, c, _) in enumerate(BAD)])
def test_bad_arguments_are_refused(zs, name, change, status):
    fn, args = calls(zs)[name]
    assert set(change) <= set(args)
    assert fn(*{**args, **change}.values()) == status
    assert zs.zs_last_error()


def test_nothing_to_do_is_fine(zs):
    for name, change in (("linear", dict(m=0)), ("linear", dict(n=0)), ("backward", dict(cols=0)),
                         ("backward", dict(rows=0, dbias=None))):
        fn, args = calls(zs)[name]
        assert fn(*{**args, **change}.values()) == 0


def test_workspace(zs):
    for rows, cols in ((1, 1), (7, 100), (8192, 16384), (1 << 20, 8), (3, 1 << 20), (100000, 1600)):
        parts, rest = divmod(zs.zs_activation_backward_workspace(rows, cols), cols * 4)
        assert rest == 0 and 1 <= parts <= min(rows, 1024)
    assert zs.zs_activation_backward_workspace(0, 8) == 0
    assert zs.zs_activation_backward_workspace(8, 1 << 31) == 0


def test_too_large_is_said_by_its_name(zs):
    """A product of more tiles than a launch takes is refused, in the entry point's own words."""
    fn, args = calls(zs)["linear"]
    size, apart = 1 << 20, {k: P((i + 1) << 48) for i, k in enumerate(("a", "as_", "b", "bs", "c"))}
    args = {**args, **apart, "m": size, "n": size, "ldc": size, "bias": None, "res": None, "pre": None}
    assert fn(*args.values()) == UNSUPPORTED
    assert zs.zs_last_error().startswith("zs_mx_linear: too large")


def test_python_checks(zs):
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        zs.zs_activation_backward(x, x, zs.ZS_ACT_GELU, x)      # not on the GPU
    with pytest.raises(ValueError):
        zs.zs_activation_backward(x[0], x[0], zs.ZS_ACT_GELU, x[0])


def test_device_of_tensors_and_stream(zs, monkeypatch):
    class Stub:
        def __init__(self, index):
            self.device, self.device_index, self.cuda_stream = f"cuda:{index}", index, 5

        def get_device(self):
            return self.device_index

    monkeypatch.setattr(zs._t(), "device", lambda: 1)
    assert zs._here(Stub(1), Stub(1), None, Stub(1)) == 5 and zs._here(3, Stub(1)) == 3
    for stream, tensors in ((3, (Stub(1), Stub(0))), (Stub(0), (Stub(1),))):
        with pytest.raises(ValueError, match="device"):
            zs._here(stream, *tensors)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
def test_activations_against_torch_and_differences(act):
    x = torch.cat([torch.linspace(-9, 9, 400, dtype=F64), torch.tensor([-40.0, 40.0, 0.3], dtype=F64)])
    f = {"none": lambda t: t * 1.0, "relu": torch.relu, "silu": torch.nn.functional.silu,
         "gelu": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[act]
    assert torch.allclose(ref.activate(x, act), f(x), rtol=1e-12, atol=1e-14)
    leaf = x.clone().requires_grad_(True)
    want, = torch.autograd.grad(f(leaf).sum(), leaf)
    got, bound = ref.slope(x, act)
    assert torch.allclose(got, want, rtol=1e-10, atol=1e-13) and bool((bound >= got.abs() - 1e-15).all())
    h = 1e-5
    diff = (ref.activate(x + h, act) - ref.activate(x - h, act)) / (2 * h)
    assert bool(((diff - got).abs() < 1e-8)[x.abs() > h].all())
