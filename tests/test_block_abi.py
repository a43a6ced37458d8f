"""The last block's operators on the CPU: argument errors return before anything
is enqueued; the generator against its published answers; and the plain 64-bit
forms that the GPU tests compare with against autograd and differences. No GPU
work."""
import ctypes as C
import math

import pytest
import torch

import block_reference as ref

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


def rule(zs, p=0.1, seed=1, offset=2, dev=None):
    return C.byref(zs.zs_dropout_rule(p, seed, offset, dev))


def calls(zs):
    """One argument list per entry point that only its changes make invalid."""
    lib = zs._lib
    return {
        "dropout": (lib.zs_dropout, dict(
            x=far(0), res=far(1), dtype=0, rows=8, cols=64, rule=rule(zs), out=far(2),
            stream=None)),
        "forward": (lib.zs_block_norm_forward, dict(
            x=far(0), res=far(1), post=far(2), gate=far(3), gain=far(4), dtype=0, rows=8, cols=64,
            eps=1e-5, rs=1.0, bs=1.0, rule=rule(zs), h=far(5), prstd=far(6), rstd=far(7),
            codes=far(8), scales=far(9), y=far(10), stream=None)),
        "backward": (lib.zs_block_norm_backward, dict(
            dy=far(0), h=far(1), rstd=far(2), gain=far(3), dres=far(4), x=far(5), prstd=far(6),
            post=far(7), gate=far(8), dtype=0, rows=8, cols=64, rs=1.0, bs=1.0, rule=rule(zs),
            dx=far(9), dresidual=far(10), dgain=far(11), dpost=far(12), dgate=far(13), ws=far(14),
            wsb=1 << 20, stream=None)),
    }


def bad(zs):
    r = lambda **k: rule(zs, **k)
    return [
        ("dropout", dict(x=None), INVALID), ("dropout", dict(out=None), INVALID),
        ("dropout", dict(rule=None), INVALID), ("dropout", dict(dtype=3), INVALID),
        ("dropout", dict(rule=r(p=-0.1)), INVALID), ("dropout", dict(rule=r(p=1.01)), INVALID),
        ("dropout", dict(rule=r(p=math.nan)), INVALID),
        ("dropout", dict(rule=r(dev=FAKE + (9 << 40) + 4)), UNSUPPORTED),
        ("dropout", dict(x=far(0, 1)), UNSUPPORTED), ("dropout", dict(res=far(1, 1)), UNSUPPORTED),
        ("dropout", dict(out=far(2, 2), dtype=2), UNSUPPORTED),
        ("dropout", dict(rows=1 << 49), UNSUPPORTED), ("dropout", dict(rows=1 << 32, cols=1), UNSUPPORTED),
        ("dropout", dict(rows=1 << 20, cols=1 << 16), UNSUPPORTED),
        ("dropout", dict(rows=1, cols=1 << 40), UNSUPPORTED),
        ("dropout", dict(out=far(0, 16)), ALIAS), ("dropout", dict(out=far(1, 2)), ALIAS),
        ("dropout", dict(rule=r(dev=FAKE + (2 << 40) + 8)), ALIAS),
        ("forward", dict(x=None), INVALID), ("forward", dict(res=None), INVALID),
        ("forward", dict(gain=None), INVALID), ("forward", dict(h=None), INVALID),
        ("forward", dict(codes=None), INVALID), ("forward", dict(scales=None), INVALID),
        ("forward", dict(codes=None, scales=None, y=None), INVALID),
        ("forward", dict(post=None), INVALID), ("forward", dict(dtype=2), INVALID),
        ("forward", dict(eps=-1.0), INVALID), ("forward", dict(eps=math.nan), INVALID),
        ("forward", dict(rs=math.inf), INVALID), ("forward", dict(bs=math.nan), INVALID),
        ("forward", dict(rule=r(p=2.0)), INVALID),
        ("forward", dict(cols=65537), UNSUPPORTED), ("forward", dict(rows=1 << 49), UNSUPPORTED),
        ("forward", dict(rows=1 << 33, cols=8), UNSUPPORTED),
        ("forward", dict(codes=far(8, 8)), UNSUPPORTED), ("forward", dict(scales=far(9, 2)), UNSUPPORTED),
        ("forward", dict(gate=far(3, 1)), UNSUPPORTED), ("forward", dict(prstd=far(6, 2)), UNSUPPORTED),
        ("forward", dict(post=far(2, 1)), UNSUPPORTED), ("forward", dict(y=far(10, 1)), UNSUPPORTED),
        ("forward", dict(h=far(0, 64)), ALIAS), ("forward", dict(y=far(0)), ALIAS),
        ("forward", dict(h=far(3)), ALIAS), ("forward", dict(rstd=far(6)), ALIAS),
        ("forward", dict(y=far(5)), ALIAS), ("forward", dict(codes=far(1)), ALIAS),
        ("forward", dict(rule=r(dev=FAKE + (5 << 40))), ALIAS),
        ("backward", dict(dy=None), INVALID), ("backward", dict(h=None), INVALID),
        ("backward", dict(rstd=None), INVALID), ("backward", dict(gain=None), INVALID),
        ("backward", dict(x=None), INVALID), ("backward", dict(prstd=None), INVALID),
        ("backward", dict(dx=None), INVALID), ("backward", dict(dresidual=None), INVALID),
        ("backward", dict(dgain=None), INVALID), ("backward", dict(dpost=None), INVALID),
        ("backward", dict(dgate=None), INVALID), ("backward", dict(gate=None), INVALID),
        ("backward", dict(post=None), INVALID), ("backward", dict(ws=None), INVALID),
        ("backward", dict(wsb=8 * 64 * 8 - 1), INVALID), ("backward", dict(dtype=2), INVALID),
        ("backward", dict(rs=math.nan), INVALID), ("backward", dict(rule=r(p=-1.0)), INVALID),
        ("backward", dict(cols=65537), UNSUPPORTED), ("backward", dict(rows=1 << 32, cols=8), UNSUPPORTED),
        ("backward", dict(ws=far(14, 2)), UNSUPPORTED), ("backward", dict(x=far(5, 1)), UNSUPPORTED),
        ("backward", dict(dgate=far(13, 2)), UNSUPPORTED), ("backward", dict(dx=far(9, 1)), UNSUPPORTED),
        ("backward", dict(dx=far(0, 16)), ALIAS), ("backward", dict(dresidual=far(5, 2)), ALIAS),
        ("backward", dict(dx=far(10)), ALIAS), ("backward", dict(dgain=far(12)), ALIAS),
        ("backward", dict(dgate=far(8)), ALIAS), ("backward", dict(ws=far(1)), ALIAS),
        ("backward", dict(rule=r(dev=FAKE + (11 << 40))), ALIAS),
    ]


def test_bad_arguments_are_refused(zs):
    for name, change, status in bad(zs):
        fn, args = calls(zs)[name]
        assert set(change) <= set(args)
        assert fn(*{**args, **change}.values()) == status, (name, change)
        assert zs.zs_last_error()


def test_nothing_to_do_is_fine(zs):
    for name, change in (("dropout", dict(rows=0)), ("dropout", dict(cols=0, x=None)),
                         ("forward", dict(rows=0)), ("forward", dict(cols=0)),
                         ("backward", dict(cols=0))):
        fn, args = calls(zs)[name]
        assert fn(*{**args, **change}.values()) == 0


def test_python_checks(zs):
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        zs.zs_dropout(x, x, (0.1, 0, 0))            # not on the GPU
    with pytest.raises(ValueError):
        zs.zs_dropout(x.view(-1), x, (0.1, 0, 0))
    with pytest.raises(ValueError):
        zs.zs_block_norm_forward(x, x, x[0], 1e-5, x, codes=x)
    with pytest.raises(ValueError):
        zs._rule((0.1, 0, 0, torch.zeros(1, dtype=torch.int64)))


def test_workspace_grows_with_the_shares(zs):
    assert zs.zs_block_norm_backward_workspace(0, 64) == 0
    assert zs.zs_block_norm_backward_workspace(3, 64) == 3 * 64 * 8
    assert zs.zs_block_norm_backward_workspace(1 << 20, 64) == 1024 * 64 * 8
    assert zs.zs_block_norm_backward_workspace(8, 65537) == 0


def test_generator_against_its_published_answers():
    """The authors' known answers for Philox4x32 with seven and with ten rounds."""
    ones, pi = 0xffffffff, (0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344, 0xa4093822, 0x299f31d0)
    for rounds, counter, key, want in (
            (7, (0,) * 4, (0,) * 2, "5f6fb709 0d893f64 4f121f81 4f730a48"),
            (7, (ones,) * 4, (ones,) * 2, "5207ddc2 45165e59 4d8ee751 8c52f662"),
            (7, pi[:4], pi[4:], "4dfccaba 190a87f0 c47362ba b6b5242a"),
            (10, (0,) * 4, (0,) * 2, "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
            (10, (ones,) * 4, (ones,) * 2, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
            (10, pi[:4], pi[4:], "d16cfe09 94fdcceb 5001e420 24126ea1")):
        assert " ".join("%08x" % w for w in ref.philox(counter, key, rounds)) == want


def test_kept_share_is_what_p_says():
    """Binomial: four standard deviations of 40960 elements."""
    for p in (0.0, 0.1, 0.5, 1.0):
        f = ref.keep_factor(40, 1024, p, 7, 1 << 40)
        assert abs(float((f == 0).double().mean()) - p) <= 4 * math.sqrt(p * (1 - p) / 40960)


def test_rounding_is_to_nearest_even():
    g = torch.Generator().manual_seed(0)
    for dtype in (torch.bfloat16, torch.float16):
        a = torch.randn(1000, generator=g, dtype=F64).to(dtype).to(F64)
        up = torch.nextafter(a.to(dtype), torch.full((1000,), math.inf, dtype=dtype)).to(F64)
        mid = (a + up) / 2
        even = torch.where(a.to(dtype).view(torch.int16) % 2 == 0, a, up)
        assert torch.equal(ref.rounded(mid, dtype), even)
        assert torch.equal(ref.rounded(mid + 1e-9 * (up - a), dtype), up)
        assert torch.equal(ref.rounded(mid - 1e-9 * (up - a), dtype), a)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [False, True])
def test_gradients_against_autograd_and_differences(post, gate):
    g = torch.Generator().manual_seed(3)
    rows, cols, eps, rs, bs = 5, 11, 1e-5, 0.75, 0.5

    def randn(*s):
        return torch.randn(*s, generator=g, dtype=F64)

    leaves = {"x": randn(rows, cols), "res": randn(rows, cols), "gain": 1 + 0.1 * randn(cols)}
    if post:
        leaves["post_gain"] = 1 + 0.1 * randn(cols)
    if gate:
        leaves["gate"] = randn(cols)
    factor = ref.keep_factor(rows, cols, 0.3, 5, 6)
    dy, dres = randn(rows, cols), randn(rows, cols)

    def value(v):
        """The formula without its rounding, whose gradient is taken to pass through."""
        n = v["x"]
        if post:
            n = n / torch.sqrt((n * n).mean(1, keepdim=True) + eps) * v["post_gain"]
        if gate:
            n = n * v["gate"]
        h = rs * v["res"] + bs * n * factor
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * v["gain"]
        return (dy * y).sum() + (dres * h).sum(), h

    for t in leaves.values():
        t.requires_grad_(True)
    total, h = value(leaves)
    want = dict(zip(leaves, torch.autograd.grad(total, list(leaves.values()))))
    v = {k: t.detach() for k, t in leaves.items()}
    h = h.detach()
    rstd = 1 / torch.sqrt((h * h).mean(1) + eps)
    post_rstd = 1 / torch.sqrt((v["x"] ** 2).mean(1) + eps) if post else None
    got, _ = ref.block_grad(dy, h, rstd, v["gain"], dres, v["x"], post_rstd, v.get("post_gain"),
                            v.get("gate"), rs, bs, factor)
    names = {"x": "dx", "res": "dresidual", "gain": "dgain", "post_gain": "dpost_gain",
             "gate": "dgate"}
    for k, t in v.items():
        assert torch.allclose(got[names[k]], want[k], rtol=1e-11, atol=1e-13)
        # central differences: the third derivative's term stays below 1e-8 of values near 1
        step = 1e-4
        for i in range(0, t.numel(), 7):
            d = torch.zeros_like(t).view(-1)
            d[i] = step
            d = d.view(t.shape)
            diff = (value({**v, k: t + d})[0] - value({**v, k: t - d})[0]) / (2 * step)
            assert abs(float(diff - got[names[k]].view(-1)[i])) < 1e-5
