"""The losses on given tokens on the CPU: argument errors return before anything
is enqueued; the rules of the host side that a result depends on; and the plain
64-bit forms that the GPU tests compare with against autograd and differences.
No GPU work."""
import ctypes as C
import math

import pytest
import torch

import token_reference as ref

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
    common = dict(z=far(0), dtype=0, rows=8, vocab=100, ld=100, ids=far(1))
    ws = dict(ws=far(20), wsb=1 << 20, stream=None)
    return {
        "logprob": (lib.zs_logprob, dict(**common, tau=1.0, logp=far(2), **ws)),
        "policy": (lib.zs_policy, dict(
            **common, tau=1.0, adv=far(2), old=far(3), ref=far(4), low=0.2, high=0.2, kl=0.1,
            weight=far(5), scale=1.0, dev=None, logp=far(6), loss=far(7), grad=far(8), gld=100,
            **ws)),
        "preference": (lib.zs_preference, dict(
            **common, starts=far(2), pairs=2, tau=1.0, ref=far(3), kind=0, beta=0.1, smooth=0.0,
            mean=0, weight=far(4), scale=1.0, dev=None, seq=far(5), loss=far(6), grad=far(7),
            gld=100, clear=0, **ws)),
    }


COMMON = [
    (dict(z=None), INVALID), (dict(ids=None), INVALID), (dict(ws=None), INVALID),
    (dict(wsb=8), INVALID), (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID),
    (dict(vocab=0), INVALID), (dict(ld=99), INVALID), (dict(vocab=1 << 31, ld=1 << 31), INVALID),
    (dict(tau=0.0), INVALID), (dict(tau=2.0 ** -127), INVALID), (dict(tau=math.inf), INVALID),
    (dict(tau=math.nan), INVALID), (dict(rows=1 << 49), UNSUPPORTED),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(z=far(0, 1)), UNSUPPORTED),
    (dict(z=far(0, 2), dtype=2), UNSUPPORTED), (dict(ids=far(1, 2)), UNSUPPORTED),
    (dict(ws=far(20, 8)), UNSUPPORTED), (dict(ws=far(0)), ALIAS),
]
BAD = [(name, *c) for name in ("logprob", "policy", "preference") for c in COMMON] + [
    ("logprob", dict(logp=None), INVALID), ("logprob", dict(logp=far(2, 2)), UNSUPPORTED),
    ("logprob", dict(logp=far(0)), ALIAS), ("logprob", dict(logp=far(20)), ALIAS),
    ("policy", dict(adv=None), INVALID), ("policy", dict(loss=None), INVALID),
    ("policy", dict(low=-0.1), INVALID), ("policy", dict(low=1.1), INVALID),
    ("policy", dict(high=-0.1), INVALID), ("policy", dict(high=math.inf), INVALID),
    ("policy", dict(low=math.nan), INVALID), ("policy", dict(kl=math.nan), INVALID),
    ("policy", dict(scale=0.0), INVALID), ("policy", dict(scale=math.inf), INVALID),
    ("policy", dict(gld=99), INVALID), ("policy", dict(grad=far(8, 1)), UNSUPPORTED),
    ("policy", dict(adv=far(2, 2)), UNSUPPORTED), ("policy", dict(old=far(3, 1)), UNSUPPORTED),
    ("policy", dict(ref=far(4, 2)), UNSUPPORTED), ("policy", dict(weight=far(5, 2)), UNSUPPORTED),
    ("policy", dict(dev=far(9, 4)), UNSUPPORTED), ("policy", dict(loss=far(7, 2)), UNSUPPORTED),
    ("policy", dict(grad=far(0, 2)), ALIAS), ("policy", dict(grad=far(0), gld=101), ALIAS),
    ("policy", dict(loss=far(6)), ALIAS), ("policy", dict(logp=far(3)), ALIAS),
    ("policy", dict(loss=far(2)), ALIAS), ("policy", dict(logp=far(8)), ALIAS),
    ("preference", dict(starts=None), INVALID), ("preference", dict(loss=None), INVALID),
    ("preference", dict(kind=3), INVALID), ("preference", dict(kind=-1), INVALID),
    ("preference", dict(beta=0.0), INVALID), ("preference", dict(beta=math.nan), INVALID),
    ("preference", dict(smooth=1.5), INVALID), ("preference", dict(smooth=0.1, kind=1), INVALID),
    ("preference", dict(smooth=math.nan), INVALID), ("preference", dict(scale=-1.0), INVALID),
    ("preference", dict(gld=99), INVALID), ("preference", dict(pairs=1 << 22), UNSUPPORTED),
    ("preference", dict(starts=far(2, 2)), UNSUPPORTED), ("preference", dict(ref=far(3, 2)), UNSUPPORTED),
    ("preference", dict(weight=far(4, 1)), UNSUPPORTED), ("preference", dict(seq=far(5, 2)), UNSUPPORTED),
    ("preference", dict(loss=far(6, 2)), UNSUPPORTED), ("preference", dict(grad=far(7, 1)), UNSUPPORTED),
    ("preference", dict(dev=far(9, 4)), UNSUPPORTED),
    ("preference", dict(grad=far(0, 2)), ALIAS), ("preference", dict(seq=far(6)), ALIAS),
    ("preference", dict(loss=far(2)), ALIAS), ("preference", dict(seq=far(7, 16)), ALIAS),
    ("preference", dict(grad=far(3)), ALIAS),
]


@pytest.mark.parametrize("name,change,status", BAD,
                         ids=[f"{n}-{'-'.join(c)}-{i}" for i, (n, c, _) in enumerate(BAD)])
def test_bad_arguments_are_refused(zs, name, change, status):
    fn, args = calls(zs)[name]
    assert set(change) <= set(args)
    assert fn(*{**args, **change}.values()) == status
    assert zs.zs_last_error()


def test_nothing_to_do_is_fine(zs):
    for name, change in (("logprob", dict(rows=0)), ("policy", dict(rows=0)),
                         ("preference", dict(pairs=0))):
        fn, args = calls(zs)[name]
        assert fn(*{**args, **change}.values()) == 0


@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_parts_of_a_row_leave_nothing_out(zs, dtype):
    """All parts but the last lie within the row's vectors, whatever its alignment (the last
    takes what comes after its first vector, at least the row's end). The workspace tells their
    number: 16 bytes each, and 20 a row."""
    esz = 4 if dtype == zs.ZS_FP32 else 2
    ve = 16 // esz
    for rows in (1, 2, 3, 5, 13, 100, 512, 1000, 1024, 5000):
        for vocab in (1, 3, 8, 15, 100, 1000, 4095, 32000, 50257, 65537, 128000, 152064, 200003):
            parts, rest = divmod(zs.zs_policy_workspace(rows, vocab, dtype) // rows - 20, 16)
            assert rest == 0 and parts >= 1
            vecs = vocab * esz // 16
            each = -(-vecs // parts) if vecs else 1
            for head in range(min(ve, vocab)):
                have = (vocab - head) // ve
                assert (parts - 1) * each <= have <= parts * each or parts == 1


def test_python_checks(zs):
    z = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        zs.zs_logprob(z, z, z)
    with pytest.raises(ValueError):
        zs._grad_rows(z.half(), z, 4, 8)


@pytest.mark.parametrize("old,refs", [(True, True), (False, True), (True, False)])
def test_policy_gradient_against_autograd_and_differences(old, refs):
    g = torch.Generator().manual_seed(1)
    z = 2 * torch.randn(9, 13, generator=g, dtype=F64)
    ids = torch.tensor([0, 5, 12, -1, 13, 3, 3, 7, 1])
    adv = torch.randn(9, generator=g, dtype=F64)
    logp = ref.logprob(z, ids, 0.7)[0]
    drift = torch.tensor([0.05, 0.4, -0.4, 0, 0, 0.4, -0.4, 0.1, 0.3], dtype=F64)
    o = logp - drift if old else None
    r = logp + 0.3 * torch.randn(9, generator=g, dtype=F64) if refs else None
    w = torch.rand(9, generator=g, dtype=F64)
    w[8] = 0

    def total(zz):
        lp, _, live = ref.logprob(zz, ids, 0.7)
        ratio = torch.exp(lp - (o if old else lp.detach()))
        loss = -torch.minimum(ratio * adv, ratio.clamp(0.8, 1.28) * adv)
        if refs:
            loss = loss + 0.05 * (torch.exp(r - lp) - 1 - (r - lp))
        return torch.where(live, w * loss, 0.0)

    zz = z.clone().requires_grad_(True)
    want, = torch.autograd.grad(total(zz).sum() * 8, zz)
    lp, loss, got, _ = ref.policy(z, ids, 0.7, adv, o, r, 0.2, 0.28, 0.05, w, 8.0)
    assert torch.allclose(got, want, rtol=1e-11, atol=1e-13)
    assert torch.allclose(loss, total(z).detach(), rtol=1e-12, atol=1e-14)
    if old:   # without old_logp the ratio is 1 for every logits: no difference to take
        for i, j in ((0, 0), (1, 5), (2, 4), (5, 3), (7, 7)):
            d = torch.zeros_like(z)
            d[i, j] = 1e-5
            diff = float((total(z + d) - total(z - d)).sum()) / 2e-5 * 8
            assert abs(diff - float(got[i, j])) < 1e-7


@pytest.mark.parametrize("kind,smoothing,mean", [("sigmoid", 0.0, False), ("sigmoid", 0.2, True),
                                                 ("hinge", 0.0, False), ("square", 0.0, True)])
def test_preference_gradient_against_autograd_and_differences(kind, smoothing, mean):
    g = torch.Generator().manual_seed(2)
    z = 2 * torch.randn(20, 11, generator=g, dtype=F64)
    ids = torch.randint(0, 11, (20,), generator=g)
    ids[[2, 9]] = -1
    starts, refs = [1, 6, 6, 11, 18], torch.randn(4, generator=g, dtype=F64)
    w = torch.tensor([0.7, 1.3], dtype=F64)

    def losses(zz):
        lp, _, live = ref.logprob(zz, ids, 2.0)
        out = []
        for p in (0, 1):
            seq = []
            for s in (2 * p, 2 * p + 1):
                n = max(1, int(live[starts[s]:starts[s + 1]].sum())) if mean else 1
                seq.append(lp[starts[s]:starts[s + 1]].sum() / n - refs[s])
            d = seq[0] - seq[1]
            if kind == "sigmoid":
                soft = torch.nn.functional.softplus
                out.append((1 - smoothing) * soft(-0.5 * d) + smoothing * soft(0.5 * d))
            elif kind == "hinge":
                out.append(torch.relu(1 - 0.5 * d))
            else:
                out.append((d - 1.0) ** 2)
        return w * torch.stack(out)

    zz = z.clone().requires_grad_(True)
    want, = torch.autograd.grad(losses(zz).sum() * 4, zz)
    loss, seq, got, _, inside = ref.preference(z, ids, starts, 2.0, refs, kind, 0.5, smoothing,
                                               mean, w, 4.0)
    assert torch.allclose(loss, losses(z).detach(), rtol=1e-12)
    assert torch.allclose(got, want, rtol=1e-11, atol=1e-13)
    assert seq[1] == 0 and inside.tolist() == [1 <= i < 18 for i in range(20)]
    for i, j in ((1, 0), (4, 3), (12, 10), (17, 5), (0, 0), (2, 1)):
        d = torch.zeros_like(z)
        d[i, j] = 1e-5
        diff = float((losses(z + d) - losses(z - d)).sum()) / 2e-5 * 4
        assert abs(diff - float(got[i, j])) < 1e-7
