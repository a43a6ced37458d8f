"""The losses on given tokens' log-probabilities on the GPU against their 64-bit
plain forms.

Tolerances, fixed before the first run. U: half a step of a type, relative. A
term 2^(z c - I) has the rounding of its exponent, of c (relative to the row's
largest) and of the instruction: with D the row's spread of z / tau, relative
(2 D + 6) 2^-24. A thread adds at most 32 terms in fp32, everything beyond in
binary64. So a sum is off by delta = (2 D + 38) 2^-24 of itself, a
log-probability by 2 delta, or by that much of itself where it is small.
"""
import math
import zlib

import pytest
import torch

import token_reference as ref
from gpu_util import announce

pytestmark = pytest.mark.gpu
BF16, FP16, FP32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
U = {t: torch.finfo(t).eps / 2 for t in (BF16, FP16, FP32)}
TINY = {BF16: 2.0 ** -134, FP16: 2.0 ** -25, FP32: 2.0 ** -126}
SHAPES = [(1, 1), (2, 3), (3, 9), (5, 15), (4, 100), (6, 1000), (7, 4099), (3, 50257), (2, 66000),
          (2, 140001), (1100, 520), (1030, 2001)]


@pytest.fixture(scope="module")
def zs(hip_built):
    from sharded_mixed_precision_zs_amd import zeroshard
    return zeroshard


def gen(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def code(zs, dtype):
    return {BF16: zs.ZS_BF16, FP16: zs.ZS_FP16, FP32: zs.ZS_FP32}[dtype]


def f32(t):
    return None if t is None else t.float()


def cu(t):
    return None if t is None else t.cuda()


def problem(rows, vocab, dtype):
    """Logits; tokens, some of which are none, one of which is nearly certain, one unlikely."""
    g = gen("z", rows, vocab)
    z = 2 * torch.randn(rows, vocab, generator=g)
    ids = torch.randint(0, vocab, (rows,), generator=g)
    z[torch.arange(rows), ids] += 3
    z[0, ids[0]] += 25
    if rows > 3:
        z[1, ids[1]] -= 30
        ids[2], ids[3] = -1, vocab
    return z.to(dtype), ids.int(), g


def spread(z, tau):
    zz = z.double() / tau
    return zz.amax(1) - zz.masked_fill(torch.isinf(zz), 0).amin(1)


def errors(z, tau, logp):
    delta = (2 * spread(z, tau) + 38) * 2.0 ** -24
    return delta, 2 * delta * (2 * logp.abs()).clamp(max=1) + 2.0 ** -23 * logp.abs()


def check(got, want, tol, what):
    got, want, tol = got.double().cpu(), want.double(), torch.as_tensor(tol).double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN positions differ"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    ok = ~inf & ~torch.isnan(want)
    err, tol = (got - want).abs()[ok], tol.expand(want.shape)[ok]
    assert bool((err <= tol).all()), (
        f"{what}: {int((err > tol).sum())} of {err.numel()} off; worst "
        f"{float((err / tol.clamp(min=1e-300)).max()):.3g} times the tolerance")


def check_grad(got, want, z, ids, tau, delta, dslope, dtype, what):
    """dslope: error of the slope times scale / tau, per row."""
    q = torch.softmax(z.double() / tau, 1)
    live = (ids >= 0) & (ids < z.shape[1])
    at = torch.arange(z.shape[0])[live]
    share = q.clone()
    others = q.clone()
    others[at, ids[live].long()] = 0
    share[at, ids[live].long()] = others[live].sum(1)
    inner = want.abs() * (3 * delta.unsqueeze(1) + 2.0 ** -22) + share * dslope.unsqueeze(1)
    check(got, want, U[dtype] * (want.abs() + inner) + inner + TINY[dtype], what)


def guarded_like(z, ld=None):
    """An output of z's shape in a buffer of a known value, rows `ld` apart, and a check that
    nothing else was written."""
    rows, vocab = z.shape
    ld = ld or vocab
    raw = torch.full((rows * ld + 32,), 7.0, dtype=z.dtype, device="cuda")
    out = raw[16:16 + rows * ld].view(rows, ld)[:, :vocab]

    def whole():
        mask = torch.ones_like(raw, dtype=torch.bool)
        mask[16:16 + rows * ld].view(rows, ld)[:, :vocab] = False
        return bool((raw[mask] == 7.0).all())

    return out, whole


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=str)
@pytest.mark.parametrize("tau", [1.0, 0.7])
def test_logprob_against_64_bits(zs, dtype, tau):
    for rows, vocab in SHAPES:
        announce(f"logprob {dtype} {tau} {rows}x{vocab}")
        z, ids, _ = problem(rows, vocab, dtype)
        want, _, _ = ref.logprob(z.double(), ids, float(torch.tensor(tau)))
        out = torch.full((rows,), 9.0, device="cuda")
        ws = torch.empty(zs.zs_logprob_workspace(rows, vocab, code(zs, dtype)), dtype=torch.uint8,
                         device="cuda")
        zs.zs_logprob(z.cuda(), ids.cuda(), out, temperature=tau, workspace=ws)
        check(out, want, errors(z, tau, want)[1] + 1e-45, "logp")


def run_policy(zs, z, ids, tau, adv, old, refs, weight, scale, grad, kl=0.05, **more):
    rows, vocab = z.shape
    logp, loss = torch.full((rows,), 9.0, device="cuda"), torch.full((rows,), 9.0, device="cuda")
    need = zs.zs_policy_workspace(rows, vocab, code(zs, z.dtype))
    zs.zs_policy(z, cu(ids), cu(adv), loss, temperature=tau, old_logp=cu(old), ref_logp=cu(refs),
                 clip_low=0.2, clip_high=0.28, kl_weight=kl, row_weight=cu(weight),
                 loss_scale=scale, logp=logp, grad=grad,
                 workspace=torch.empty(need, dtype=torch.uint8, device="cuda"), **more)
    return logp, loss


def policy_inputs(z, ids, g, tau, old, refs, weighted):
    rows = z.shape[0]
    logp = ref.logprob(z.double(), ids, tau)[0]
    adv = torch.randn(rows, generator=g)
    # clipped on either side, or not; never within 1e-3 of an end
    drift = torch.tensor([0.05, 0.4, -0.4, 0.1, -0.1, 0.3, -0.3])[torch.arange(rows) % 7]
    o = (logp - drift.double()).float() if old else None
    r = (logp + 0.3 * torch.randn(rows, generator=g)).float() if refs else None
    w = torch.rand(rows, generator=g) if weighted else None
    if weighted:
        w[rows // 2] = 0
    return adv, o, r, w


def check_policy(z, ids, tau, adv, o, r, w, scale, logp, loss, grad, what):
    tau = float(torch.tensor(tau))
    dbl = lambda t: None if t is None else t.double()
    low, high, kl = (float(torch.tensor(v)) for v in (0.2, 0.28, 0.05))
    lp, want, g, mag = ref.policy(z.double(), ids, tau, adv.double(), dbl(o), dbl(r), low, high, kl,
                                  dbl(w), scale)
    delta, dlogp = errors(z, tau, lp)
    check(logp, lp, dlogp + 1e-45, what + " logp")
    # ratio and KL follow the log-probability; exp, products and sums beside it
    check(loss, want, (mag * tau / scale + want.abs()) * (2 * dlogp + 2.0 ** -20) + 1e-45,
          what + " loss")
    if grad is not None:
        check_grad(grad, g, z, ids, tau, delta, mag * (2 * dlogp + 2.0 ** -20), z.dtype, what)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=str)
@pytest.mark.parametrize("old,refs,weighted", [(True, True, True), (False, True, False),
                                               (True, False, False)])
def test_policy_against_64_bits(zs, dtype, old, refs, weighted):
    for rows, vocab in SHAPES:
        announce(f"policy {dtype} {old} {refs} {rows}x{vocab}")
        tau = 1.0 if old else 2.0
        z, ids, g = problem(rows, vocab, dtype)
        adv, o, r, w = policy_inputs(z, ids, g, tau, old, refs, weighted)
        grad, whole = guarded_like(z)
        logp, loss = run_policy(zs, z.cuda(), ids, tau, adv, o, r, w, 256.0, grad)
        check_policy(z, ids, tau, adv, o, r, w, 256.0, logp, loss, grad, f"{rows}x{vocab}")
        assert whole()
        # without a gradient, and in the logits' place
        l2, s2 = run_policy(zs, z.cuda(), ids, tau, adv, o, r, w, 256.0, None)
        inplace = z.cuda()
        l3, s3 = run_policy(zs, inplace, ids, tau, adv, o, r, w, 256.0, inplace)
        assert torch.equal(l3, logp) and torch.equal(s3, loss) and torch.equal(inplace, grad)
        check_policy(z, ids, tau, adv, o, r, w, 256.0, l2, s2, None, "loss alone")


def test_policy_strided_and_unaligned(zs):
    for dtype, off, vocab, ld, gld in ((BF16, 3, 1001, 1016, 1001), (FP16, 1, 9000, 9003, 9010),
                                       (FP32, 1, 501, 777, 501), (BF16, 0, 20000, 20008, 20016)):
        announce(f"policy strided {dtype} {vocab}")
        z, ids, g = problem(6, vocab, dtype)
        base = torch.zeros(6 * ld + 16, dtype=dtype, device="cuda")
        view = base[off:off + 6 * ld].view(6, ld)[:, :vocab]
        view.copy_(z)
        adv, o, r, w = policy_inputs(z, ids, g, 1.0, True, True, False)
        grad, whole = guarded_like(z, gld)
        logp, loss = run_policy(zs, view, ids, 1.0, adv, o, r, w, 64.0, grad)
        check_policy(z, ids, 1.0, adv, o, r, w, 64.0, logp, loss, grad, f"{vocab}")
        assert whole()


def test_policy_rows_that_are_not_finite(zs):
    """-inf logits cannot be chosen; NaN, +inf and rows of -inf spoil their own row alone; rows
    without a token or weight are not looked at."""
    for dtype in (BF16, FP32):
        z, ids, g = problem(12, 1000, dtype)
        adv, o, r, w = policy_inputs(z, ids, g, 1.0, True, True, True)
        ids[4:] = torch.arange(4, 12)
        lp = ref.logprob(z.double(), ids, 1.0)[0]
        o, r = (lp - 0.1).float(), (lp + 0.1).float()
        z[4, 100:900] = -math.inf
        z[5, 7] = math.nan
        z[7, 8] = math.inf
        z[8] = -math.inf
        z[2] = math.nan                 # no token
        z[6] = math.nan                 # no weight
        w[6] = 0
        z[9, 9] = -math.inf             # the token itself cannot be chosen
        r[9] = -5
        grad = torch.full_like(z, 3.0).cuda()
        logp, loss = run_policy(zs, z.cuda(), ids, 1.0, adv, o, r, w, 16.0, grad)
        bad = [5, 7, 8]
        assert torch.isnan(logp[bad]).all() and torch.isnan(grad[bad].float()).all(1).all()
        for row in (2, 3, 6):
            assert logp[row] == 0 and loss[row] == 0 and not grad[row].any()
        assert logp[9] == -math.inf and loss[9] == math.inf
        keep = [0, 1, 4, 10, 11]
        check_policy(z[keep], ids[keep], 1.0, adv[keep], o[keep], r[keep], w[keep], 16.0,
                     logp[keep], loss[keep], grad[keep], "the others")


def test_policy_sure_and_far_apart(zs):
    """A token that has all but 2^-40 of the mass keeps its gradient and log-probability; logits
    beyond the exponents' range do not overflow."""
    z = torch.full((4, 300), -28.0)
    z[0, 5] = 0.0
    z[1] = torch.linspace(-3e4, 3e4, 300)
    z[2] = torch.linspace(-3e38, 3e38, 300, dtype=F64).float()
    z[3, :10] = 3e38
    ids, adv = torch.tensor([5, 298, 299, 3], dtype=torch.int32), torch.ones(4)
    grad = torch.empty(4, 300, device="cuda")
    logp, loss = run_policy(zs, z.cuda(), ids, 1.0, adv, None, None, None, 1.0, grad, kl=0.0)
    lp, q, _ = ref.logprob(z.double(), ids, 1.0)
    g = ref.logit_grad(q, ids, torch.full((4,), -1.0, dtype=F64))
    assert abs(float(logp[0]) / float(lp[0]) - 1) < 1e-5
    assert abs(float(grad[0, 5]) / float(g[0, 5]) - 1) < 1e-5
    assert torch.isfinite(grad).all()
    # row 1: neighbours 200 apart; the token one below the top has none of the mass
    assert abs(float(logp[1]) - float(lp[1])) < 1e-3 * 200 and logp[2] == 0 and not grad[2].any()
    assert abs(float(logp[3]) + math.log(10)) < 1e-5


def test_policy_scale_from_the_device(zs):
    z, ids, g = problem(9, 777, BF16)
    adv, o, r, w = policy_inputs(z, ids, g, 1.0, True, True, True)
    scaler = zs.zs_loss_scaler(scale=512.0, clean_steps=0, growth_interval=0, dynamic=0, step_t=0,
                               skipped=0)
    dev = zs.device_scaler_upload(zs.zs_device_scaler_make(scaler, 0.9, 0.999))
    a, b = torch.empty_like(z).cuda(), torch.empty_like(z).cuda()
    run_policy(zs, z.cuda(), ids, 1.0, adv, o, r, w, 512.0, a)
    run_policy(zs, z.cuda(), ids, 1.0, adv, o, r, w, 1.0, b, dev_scaler=dev)
    assert torch.equal(a, b)


# ---- pairs ---------------------------------------------------------------------

def run_preference(zs, z, ids, starts, grad, refs=None, weight=None, **how):
    pairs = (len(starts) - 1) // 2
    loss, seq = torch.full((pairs,), 9.0, device="cuda"), torch.full((2 * pairs,), 9.0, device="cuda")
    need = zs.zs_preference_workspace(*z.shape, code(zs, z.dtype))
    zs.zs_preference(z, cu(ids), torch.tensor(starts, dtype=torch.int32).cuda(), how.pop("beta"),
                     loss, ref_logp=cu(refs), pair_weight=cu(weight), seq_logp=seq, grad=grad,
                     workspace=torch.empty(max(16, need), dtype=torch.uint8, device="cuda"), **how)
    return loss, seq


PAIRS = [((1, 1), [0, 1, 1]), ((2, 9), [0, 1, 2]), ((9, 100), [0, 2, 5, 7, 9]),
         ((14, 1000), [2, 5, 9, 9, 12]), ((11, 4099), [0, 4, 11]), ((5, 50257), [0, 3, 5]),
         ((3, 140001), [0, 1, 3]), ((1100, 520), [0, 300, 600, 700, 1100]),
         ((1040, 2001), [3, 500, 501, 800, 1039])]
KINDS = [("sigmoid", 0.0, False), ("sigmoid", 0.2, True), ("hinge", 0.0, False), ("square", 0.0, True)]


def kind_of(zs, kind):
    return {"sigmoid": zs.ZS_PREFERENCE_SIGMOID, "hinge": zs.ZS_PREFERENCE_HINGE,
            "square": zs.ZS_PREFERENCE_SQUARE}[kind]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=str)
@pytest.mark.parametrize("kind,smoothing,mean", KINDS)
def test_preference_against_64_bits(zs, dtype, kind, smoothing, mean):
    beta = 0.25
    for (rows, vocab), starts in PAIRS:
        announce(f"preference {dtype} {kind} {rows}x{vocab}")
        z, ids, g = problem(rows, vocab, dtype)
        pairs = (len(starts) - 1) // 2
        own = ref.preference(z.double(), ids, starts, 1.0, None, kind, beta, smoothing, mean, None,
                             1.0)[1]
        refs = (own + torch.randn(2 * pairs, generator=g)).float()
        weight = 0.5 + torch.rand(pairs, generator=g)
        grad, whole = guarded_like(z)
        loss, seq = run_preference(zs, z.cuda(), ids, starts, grad, refs, weight, beta=beta,
                                   kind=kind_of(zs, kind), smoothing=smoothing, mean=mean,
                                   loss_scale=64.0)
        wl, ws, wg, slope, inside = ref.preference(z.double(), ids, starts, 1.0, refs.double(), kind,
                                                   beta, float(torch.tensor(smoothing)), mean,
                                                   weight.double(), 64.0)
        lp = ref.logprob(z.double(), ids, 1.0)[0]
        delta, dlogp = errors(z, 1.0, lp)
        count = torch.ones(2 * pairs, dtype=F64)
        dl = torch.zeros(2 * pairs, dtype=F64)
        drow = torch.zeros(rows, dtype=F64)
        for s in range(2 * pairs):
            live = (ids[starts[s]:starts[s + 1]] >= 0) & (ids[starts[s]:starts[s + 1]] < vocab)
            count[s] = max(1, int(live.sum())) if mean else 1
            dl[s] = dlogp[starts[s]:starts[s + 1]].sum() / count[s]
        check(seq, ws, dl + 2.0 ** -24 * ws.abs() + 1e-45, "seq_logp")
        dd = dl[0::2] + dl[1::2]
        bend = 2.0 if kind == "square" else beta * beta
        steep = torch.stack([torch.as_tensor(ref.pair_loss(float(x), kind, beta, smoothing)[1])
                             for x in (ws - refs.double())[0::2] - (ws - refs.double())[1::2]]).double()
        check(loss, wl, weight.double() * (steep.abs() * dd + bend * dd * dd) + 2.0 ** -22 * wl + 1e-45,
              "loss")
        for s in range(2 * pairs):
            drow[starts[s]:starts[s + 1]] = 64 * weight[s // 2] * bend * dd[s // 2] / count[s]
        drow = drow + 2.0 ** -22 * slope
        check_grad(grad[inside.cuda()], wg[inside], z[inside], ids[inside], 1.0, delta[inside],
                   drow[inside], dtype, "grad")
        assert bool((grad[~inside.cuda()] == 7.0).all()) and whole()
        inplace = z.cuda()
        l2, s2 = run_preference(zs, inplace, ids, starts, inplace, refs, weight, beta=beta,
                                kind=kind_of(zs, kind), smoothing=smoothing, mean=mean,
                                loss_scale=64.0)
        assert torch.equal(l2, loss) and torch.equal(s2, seq)
        assert torch.equal(inplace[inside.cuda()], grad[inside.cuda()])
        assert torch.equal(inplace[~inside.cuda()].cpu(), z[~inside])
        cleared = torch.full_like(inplace, 7.0)
        run_preference(zs, z.cuda(), ids, starts, cleared, refs, weight, beta=beta,
                       kind=kind_of(zs, kind), smoothing=smoothing, mean=mean, loss_scale=64.0,
                       clear=True)
        assert torch.equal(cleared[inside.cuda()], grad[inside.cuda()])
        assert not cleared[~inside.cuda()].any()
        l3, s3 = run_preference(zs, z.cuda(), ids, starts, None, refs, weight, beta=beta,
                                kind=kind_of(zs, kind), smoothing=smoothing, mean=mean)
        assert torch.equal(l3, loss) and torch.equal(s3, seq)


def test_preference_masks_weights_and_nan(zs):
    """A pair without weight, sequences without a token, a NaN in one pair: the others stay."""
    z, ids, _ = problem(40, 600, BF16)
    ids = (torch.arange(40, dtype=torch.int32) * 13) % 600
    starts = [0, 5, 10, 15, 20, 25, 30, 35, 40]
    ids[10:15] = -1                          # pair 1 prefers an answer without tokens
    clean = torch.empty_like(z).cuda()
    w = torch.tensor([1.0, 1.0, 0.0, 2.0])
    l0, s0 = run_preference(zs, z.cuda(), ids, starts, clean, None, w, beta=0.1)
    bad = z.clone()
    bad[21, 5] = math.nan                    # pair 2 has no weight
    bad[12] = math.nan                       # not a token's row
    g1 = torch.empty_like(z).cuda()
    l1, s1 = run_preference(zs, bad.cuda(), ids, starts, g1, None, w, beta=0.1)
    assert torch.equal(l1, l0) and torch.equal(g1, clean)
    assert not g1[10:15].any() and not g1[20:30].any() and l1[2] == 0
    assert float(s1[2]) == 0 and torch.isnan(s1[4])
    bad[36, 7] = math.nan
    for kind in ("sigmoid", "hinge", "square"):
        l2, _ = run_preference(zs, bad.cuda(), ids, starts, g1, None, w, beta=0.1,
                               kind=kind_of(zs, kind))
        assert torch.isnan(l2[3]) and torch.isfinite(l2[:3]).all()
        assert torch.isnan(g1[30:].float()).any(1).all() and torch.isfinite(g1[:30].float()).all()


def test_preference_starts_out_of_range_stay_inside(zs):
    """Starts below 0 and past the rows are taken as the ends; nothing else is written."""
    z, ids, _ = problem(20, 300, FP16)
    ids = ids.clamp(0, 299)
    grad, whole = guarded_like(z)
    loss, seq = run_preference(zs, z.cuda(), ids, [-5, 8, 1 << 30], grad, beta=0.1)
    l2, s2 = run_preference(zs, z.cuda(), ids, [0, 8, 20], torch.empty_like(z).cuda(), beta=0.1)
    assert torch.equal(loss, l2) and torch.equal(seq, s2) and whole()


def test_preference_without_pairs_clears(zs):
    z, ids, _ = problem(7, 90, BF16)
    grad = torch.full_like(z, 7.0).cuda()
    run_preference(zs, z.cuda(), ids, [3], grad, beta=0.1)
    assert bool((grad == 7.0).all())
    run_preference(zs, z.cuda(), ids, [3], grad, beta=0.1, clear=True)
    assert not grad.any()


def test_preference_without_rows(zs):
    z = torch.empty(0, 50, device="cuda")
    loss, seq = run_preference(zs, z, torch.empty(0, dtype=torch.int32), [0, 0, 0], z, beta=0.1)
    assert abs(float(loss) - math.log(2)) < 1e-6 and not seq.any()


def test_token_losses_captured_and_replayed(zs):
    """Replays with new logits in the same buffers, eager work between them."""
    for rows, vocab in ((40, 3000), (1100, 700)):
        z, ids, g = problem(rows, vocab, BF16)
        adv, o, r, w = (cu(t) for t in policy_inputs(z, ids, g, 1.0, True, True, True))
        dz, di = z.cuda(), ids.cuda()
        starts = torch.tensor([0, rows // 4, rows // 2, rows], dtype=torch.int32).cuda()
        starts = torch.cat([starts, starts[-1:]])       # an empty last sequence
        ws = torch.empty(max(zs.zs_policy_workspace(rows, vocab, zs.ZS_BF16),
                             zs.zs_preference_workspace(rows, vocab, zs.ZS_BF16)),
                         dtype=torch.uint8, device="cuda")
        outs = [torch.empty_like(dz), torch.empty_like(dz), torch.empty(rows, device="cuda"),
                torch.empty(rows, device="cuda"), torch.empty(2, device="cuda")]

        def both(outs):
            zs.zs_policy(dz, di, adv, outs[2], old_logp=o, ref_logp=r, kl_weight=0.1, row_weight=w,
                         logp=outs[3], grad=outs[0], workspace=ws)
            zs.zs_preference(dz, di, starts, 0.1, outs[4], grad=outs[1], workspace=ws)

        both(outs)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            both(outs)
        for i in range(3):
            dz.copy_(torch.randn(rows, vocab, generator=g).to(BF16))
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in outs]
            both(outs)
            torch.cuda.synchronize()
            for a, b in zip(got, outs):
                assert torch.equal(a, b)


def test_rows_past_32_bits(zs):
    """Rows 2^31 elements apart."""
    ld, vocab = 1 << 31, 1000
    base = torch.empty(2 * ld + vocab, dtype=BF16, device="cuda")
    view = base.as_strided((3, vocab), (ld, 1))
    z, ids, _ = problem(3, vocab, BF16)
    view.copy_(z)
    adv = torch.tensor([1.0, -1.0, 0.5])
    want, got = torch.empty_like(z).cuda(), torch.empty_like(z).cuda()
    l0, s0 = run_policy(zs, z.cuda(), ids, 1.0, adv, None, None, None, 8.0, want)
    l1, s1 = run_policy(zs, view, ids, 1.0, adv, None, None, None, 8.0, got)
    assert torch.equal(l0, l1) and torch.equal(s0, s1) and torch.equal(got, want)
    run_policy(zs, view, ids, 1.0, adv, None, None, None, 8.0, view)
    assert torch.equal(view, want)
    view.copy_(z)
    a, _ = run_preference(zs, z.cuda(), ids, [0, 1, 3], want, beta=0.1)
    b, _ = run_preference(zs, view, ids, [0, 1, 3], view, beta=0.1)
    assert torch.equal(a, b) and torch.equal(view, want)


def test_two_streams_at_once(zs):
    """Calls side by side, each with a workspace of its own, give what they give alone."""
    jobs = []
    for k, (rows, vocab) in enumerate(((300, 9000), (40, 50257))):
        z, ids, g = problem(rows, vocab, BF16)
        adv, o, r, w = (cu(t) for t in policy_inputs(z, ids, g, 1.0, True, True, False))
        starts = torch.tensor([0, rows // 3, rows], dtype=torch.int32).cuda()
        out = [torch.empty_like(z).cuda() for _ in range(2)] + [torch.empty(rows, device="cuda"),
                                                                torch.empty(1, device="cuda")]
        need = max(zs.zs_policy_workspace(rows, vocab, zs.ZS_BF16),
                   zs.zs_preference_workspace(rows, vocab, zs.ZS_BF16))
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        jobs.append((z.cuda(), ids.cuda(), adv, o, r, starts, out, ws, torch.cuda.Stream()))

    def run(z, ids, adv, o, r, starts, out, ws, stream):
        zs.zs_policy(z, ids, adv, out[2], old_logp=o, ref_logp=r, kl_weight=0.1, grad=out[0],
                     workspace=ws, stream=stream)
        zs.zs_preference(z, ids, starts, 0.1, out[3], grad=out[1], workspace=ws, stream=stream)

    want = []
    for job in jobs:
        torch.cuda.synchronize()
        run(*job)
        torch.cuda.synchronize()
        want.append([t.clone() for t in job[6]])
        for t in job[6]:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for job in jobs:
            run(*job)
    torch.cuda.synchronize()
    for job, w in zip(jobs, want):
        for a, b in zip(job[6], w):
            assert torch.equal(a, b)


def test_one_token_and_many_equal_ones(zs):
    """A vocabulary of one, every logit alike, the same token in every row."""
    for vocab in (1, 2, 700, 20000):
        z = torch.full((5, vocab), 3.0).to(BF16)
        ids = torch.full((5,), vocab - 1, dtype=torch.int32)
        grad = torch.empty_like(z).cuda()
        logp, loss = run_policy(zs, z.cuda(), ids, 1.0, torch.ones(5), None, None, None, 1.0, grad)
        want = ref.logprob(z.double(), ids, 1.0)[0]
        assert bool(((logp.cpu().double() - want).abs() <= 2.0 ** -20 * want.abs()).all())
        q = torch.full((5, vocab), 1.0 / vocab, dtype=F64)
        g = ref.logit_grad(q, ids, torch.full((5,), -1.0, dtype=F64))
        check(grad, g, U[BF16] * g.abs() * 1.001 + 2.0 ** -20 * g.abs(), "grad")


# ---- rows that a block walks -----------------------------------------------------

def gpu_close(got, want, tol, what):
    """As check, of finite values, where they lie."""
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {err.numel()} off; rows " \
        f"{torch.nonzero(bad)[:4].tolist()}"


# rows, vocabulary, type, threads of a block, rows of 64 threads that a CU holds
WALKS = [(600, 66000, BF16, 512, 8), (1100, 35001, FP16, 512, 16), (2100, 9001, FP32, 256, 16),
         (4200, 8301, BF16, 128, 16), (8300, 4200, BF16, 64, 16), (8300, 2049, FP16, 64, 16)]


@pytest.mark.parametrize("rows,vocab,dtype,threads,held", WALKS,
                         ids=[f"{w[0]}x{w[1]}" for w in WALKS])
def test_policy_rows_walked(zs, rows, vocab, dtype, threads, held):
    """Blocks that take a third row and more, whose second has a token, none, or no weight: a
    row without a token passes no barrier between the sums of those around it. Some tokens have
    less than e^-41 of the mass, so that their row is summed again. The 64-bit forms run on the
    GPU: products, exponentials and sums alone."""
    announce(f"policy walk {dtype} {rows}x{vocab}")
    blocks = torch.cuda.get_device_properties(0).multi_processor_count * held * 64 // threads
    z, ids, g = problem(rows, vocab, dtype)
    at = torch.arange(rows)
    ids = (ids % vocab).int()
    ids[(at // blocks % 2 == 1) & (at % 4 == 0)] = -1
    weight = torch.rand(rows, generator=g) + 0.5
    weight[(at // blocks % 2 == 1) & (at % 4 == 1)] = 0
    z, ids, weight = z.cuda(), ids.cuda(), weight.cuda()
    for first in (0, 1, 2, 3):           # of the first and the third turn, and one of the second
        rare = torch.arange(first, rows, 2 * blocks)[:4].cuda()
        z[rare, ids[rare].clamp(min=0).long()] = -60
    z[blocks + 2, ids[blocks + 2].long()] = -60
    adv = torch.randn(rows, generator=g).cuda()
    lp = ref.logprob(z.double(), ids, 1.0)[0]
    drift = torch.tensor([0.05, 0.4, -0.4, 0.1, -0.1, 0.3, -0.3])[at % 7].cuda()
    old, refs = (lp - drift.double()).float(), (lp + 0.3 * torch.randn(rows, generator=g).cuda()).float()
    logp, loss = torch.full((2, rows), 9.0, device="cuda")
    grad = torch.full_like(z, 7.0)
    ws = torch.empty(zs.zs_policy_workspace(rows, vocab, code(zs, dtype)), dtype=torch.uint8,
                     device="cuda")

    def run(z, logp, loss, grad):
        zs.zs_policy(z, ids, adv, loss, old_logp=old, ref_logp=refs, clip_low=0.2, clip_high=0.28,
                     kl_weight=0.05, row_weight=weight, loss_scale=64.0, logp=logp, grad=grad,
                     workspace=ws)

    run(z, logp, loss, grad)
    low, high, kl = (float(torch.tensor(v)) for v in (0.2, 0.28, 0.05))
    lp, want, wg, mag = ref.policy(z.double(), ids, 1.0, adv.double(), old.double(), refs.double(),
                                   low, high, kl, weight.double(), 64.0)
    delta, dlogp = errors(z, 1.0, lp)
    gpu_close(logp, lp, dlogp + 1e-45, "logp")
    gpu_close(loss, want, (mag / 64 + want.abs()) * (2 * dlogp + 2.0 ** -20) + 1e-45, "loss")
    q = torch.softmax(z.double(), 1)
    live = (ids >= 0) & (ids < vocab)
    mine = ids.clamp(0, vocab - 1).long().unsqueeze(1)
    share = q.scatter(1, mine, torch.where(live, q.scatter(1, mine, 0.0).sum(1),
                                           q.gather(1, mine).squeeze(1)).unsqueeze(1))
    inner = (wg.abs() * (3 * delta.unsqueeze(1) + 2.0 ** -22)
             + share * (mag * (2 * dlogp + 2.0 ** -20)).unsqueeze(1))
    gpu_close(grad, wg, U[dtype] * (wg.abs() + inner) + inner + TINY[dtype], "grad")
    l2, s2 = torch.full((2, rows), 9.0, device="cuda")
    run(z, l2, s2, z)
    assert torch.equal(l2, logp) and torch.equal(s2, loss) and torch.equal(z, grad)


# ---- tokens that cannot be chosen -------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=str)
@pytest.mark.parametrize("tau", [1.0, 0.7])
def test_tokens_that_cannot_be_chosen(zs, dtype, tau):
    """A token whose logit is -inf, among ordinary others, others far below and far above 0, and
    a single other one: its log-probability is -inf and the row's gradient the definition's, by
    rows, in parts, and in two passes."""
    for rows, vocab in ((5, 9), (5, 1000), (5, 20000), (6, 50257), (5, 140001), (70, 50257),
                        (70, 140001)):
        announce(f"-inf token {dtype} {rows}x{vocab}")
        z, ids, g = problem(rows, vocab, dtype)
        ids = (ids % vocab).int()
        at = torch.arange(4)
        z[1] -= 200
        z[3] += 200
        z[2] = -math.inf
        z[2, (int(ids[2]) + vocab // 2 + 1) % vocab] = -7
        z[at, ids[:4].long()] = -math.inf
        want, q, _ = ref.logprob(z.double(), ids, float(torch.tensor(tau)))
        assert bool((want[:4] == -math.inf).all()) and bool(torch.isfinite(want[4:]).all())
        finite = torch.where(torch.isfinite(want), want, 0.0)
        delta, dlogp = errors(z, tau, finite)
        out = torch.full((rows,), 9.0, device="cuda")
        ws = torch.empty(zs.zs_logprob_workspace(rows, vocab, code(zs, dtype)), dtype=torch.uint8,
                         device="cuda")
        zs.zs_logprob(z.cuda(), ids.cuda(), out, temperature=tau, workspace=ws)
        check(out, want, dlogp + 1e-45, "logp alone")
        # without the sampler's the ratio is 1, and the slope -A
        adv = torch.tensor([1.0, -0.7])[torch.arange(rows) % 2]
        grad = torch.full_like(z, 7.0).cuda()
        logp, loss = run_policy(zs, z.cuda(), ids, tau, adv, None, None, None, 64.0, grad)
        check(logp, want, dlogp + 1e-45, "logp")
        assert torch.equal(loss.cpu(), -adv)
        slope = -adv.double() * 64 / float(torch.tensor(tau))
        check_grad(grad, ref.logit_grad(q, ids, slope), z, ids, tau, delta,
                   slope.abs() * 2.0 ** -20, dtype, "grad")
        # with it the ratio is 0: clipped below for A < 0, no slope either way
        old = (finite - 0.05).float()
        logp, loss = run_policy(zs, z.cuda(), ids, tau, adv, old, None, None, 64.0, grad)
        low = 1 - float(torch.tensor(0.2))
        clipped = torch.tensor([0.0, 0.7 * low])[torch.arange(4) % 2]
        check(loss[:4], clipped, 1e-6, "loss")
        assert not grad[:4].any() and torch.isfinite(grad.float()).all()
        # a preferred sequence with such a token: its loss is inf, its slope -beta
        grad.fill_(7.0)
        l2, s2 = run_preference(zs, z.cuda(), ids, [0, 1, 1], grad, None, beta=0.25,
                                temperature=tau)
        assert s2[0] == -math.inf and s2[1] == 0 and l2[0] == math.inf
        slope = torch.full((1,), -0.25 / float(torch.tensor(tau)), dtype=F64)
        check_grad(grad[:1], ref.logit_grad(q[:1], ids[:1], slope), z[:1], ids[:1], tau, delta[:1],
                   slope.abs() * 2.0 ** -20, dtype, "pair grad")


# the values that d takes are far from 0, where exp(d) - 1 - d and exp(d) - 1 part
KL_SHAPES = [(6, 1000), (6, 140001), (70, 140001)]


def test_policy_far_from_the_reference(zs):
    """A reference that gives a token nothing, or far less than the student: the KL term's slope
    is that of exp(d) - 1, -1 in the end, and keeps its precision."""
    for rows, vocab in KL_SHAPES:
        announce(f"policy far from the reference {rows}x{vocab}")
        z, ids, g = problem(rows, vocab, FP32)
        ids = (ids % vocab).int()
        lp = ref.logprob(z.double(), ids, 1.0)[0]
        d = torch.tensor([-math.inf, -3e7, -1000.5, -20.0, -1.0, 1.0])[torch.arange(rows) % 6]
        refs = (lp + d.double()).float()
        for adv in (torch.zeros(rows), torch.full((rows,), 0.5)):
            grad = torch.full_like(z, 7.0).cuda()
            logp, loss = run_policy(zs, z.cuda(), ids, 1.0, adv, None, refs, None, 64.0, grad)
            check_policy(z, ids, 1.0, adv, None, refs, None, 64.0, logp, loss, grad,
                         f"{rows}x{vocab}")
            assert torch.isfinite(grad).all()


def test_policy_without_kl_weight_has_no_kl_term(zs):
    """A weight of 0 is no term, also where exp(d) is beyond fp32 or d is not finite."""
    for rows, vocab in KL_SHAPES:
        announce(f"policy kl 0 {rows}x{vocab}")
        z, ids, g = problem(rows, vocab, BF16)
        ids = (ids % vocab).int()
        adv, o, _, _ = policy_inputs(z, ids, g, 1.0, True, False, False)
        refs = torch.tensor([-math.inf, 100.0, 3e38, -3.0, math.inf, math.nan])[torch.arange(rows) % 6]
        a, b = torch.full((2,) + tuple(z.shape), 7.0, dtype=BF16, device="cuda")
        want = run_policy(zs, z.cuda(), ids, 1.0, adv, o, None, None, 64.0, a, kl=0.0)
        got = run_policy(zs, z.cuda(), ids, 1.0, adv, o, refs, None, 64.0, b, kl=0.0)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(a, b)
        assert torch.isfinite(got[1]).all()


def test_policy_without_advantage(zs):
    """An advantage of 0 gives a loss of 0 and no slope, also where the ratio is beyond fp32."""
    for rows, vocab in KL_SHAPES:
        announce(f"policy advantage 0 {rows}x{vocab}")
        z, ids, g = problem(rows, vocab, BF16)
        ids = (ids % vocab).int()
        lp = ref.logprob(z.double(), ids, 1.0)[0]
        adv = torch.tensor([0.0, -0.0, 0.7])[torch.arange(rows) % 3]
        old = (lp - 100).float()                       # a ratio of e^100
        grad = torch.full_like(z, 7.0).cuda()
        logp, loss = run_policy(zs, z.cuda(), ids, 1.0, adv, old, None, None, 64.0, grad)
        clipped = -(1 + float(torch.tensor(0.28))) * adv.double()
        check(loss, clipped, 2.0 ** -22 * clipped.abs(), "loss")
        assert not grad.any()
        z[0] = math.nan
        logp, loss = run_policy(zs, z.cuda(), ids, 1.0, adv, old, None, None, 64.0, grad)
        assert torch.isnan(loss[0]) and torch.isnan(grad[0].float()).all()


def test_preference_of_tokens_that_cannot_be_chosen(zs):
    """A sequence with a token that cannot be chosen, against one without: with no smoothing the
    side that it is right on costs nothing, the other one is infinite with a finite slope."""
    z, ids, _ = problem(8, 600, FP32)
    ids = (ids % 600).int()
    z[5, ids[5].long()] = -math.inf
    for starts, delta in (([0, 4, 8], math.inf), ([4, 8, 8], -math.inf)):
        for kind, smoothing in (("sigmoid", 0.0), ("sigmoid", 1.0), ("sigmoid", 0.25), ("hinge", 0.0)):
            grad = torch.full_like(z, 7.0).cuda()
            loss, seq = run_preference(zs, z.cuda(), ids, starts, grad, None, beta=0.25,
                                       kind=kind_of(zs, kind), smoothing=smoothing, loss_scale=16.0)
            good = smoothing if delta < 0 else 1 - smoothing     # weight of the term that is 0
            assert float(loss) == (0.0 if kind == "hinge" and delta > 0 or
                                   kind == "sigmoid" and good == 1 else math.inf)
            k = {"sigmoid": 0.25 * (smoothing if delta > 0 else smoothing - 1),
                 "hinge": 0.0 if delta > 0 else -0.25}[kind] * 16
            _, q, _ = ref.logprob(z.double(), ids, 1.0)
            slope = torch.zeros(8, dtype=F64)
            slope[starts[0]:starts[1]], slope[starts[1]:starts[2]] = k, -k
            wg = ref.logit_grad(q, ids, slope)
            inside = slice(starts[0], starts[2])
            check(grad[inside], wg[inside], 1e-4 * wg[inside].abs() + TINY[FP32], "grad")


def test_logits_far_below_the_others(zs):
    """Tokens whose logit is the type's lowest value, or far below the largest of a row that is
    itself beyond the exponents' range: the log-probability is their distance over tau."""
    for rows, vocab in ((6, 1000), (6, 140001), (70, 140001), (70, 50257)):
        for dtype in (BF16, FP32):
            for tau in (1.0, 1.7):
                announce(f"far logits {dtype} {tau} {rows}x{vocab}")
                z, ids, g = problem(rows, vocab, dtype)
                ids = (ids % vocab).int()
                mine = ids[:6].long()
                top = (mine + vocab // 2 + 1) % vocab
                z[0, mine[0]] = torch.finfo(dtype).min
                z[1, mine[1]], z[1, top[1]] = 1e30, 1e31
                z[2, mine[2]], z[2, top[2]] = -1e25, 1e25
                z[3, mine[3]], z[3, top[3]] = 3.0, 2e19
                z[4] = torch.finfo(dtype).min
                z[4, top[4]] = -1e30
                z[5] = torch.finfo(dtype).min
                want, q, _ = ref.logprob(z.double(), ids, float(torch.tensor(tau)))
                tol = errors(z.clamp(-60, 60), tau, want)[1] + 2.0 ** -22 * want.abs()
                out = torch.full((rows,), 9.0, device="cuda")
                ws = torch.empty(zs.zs_logprob_workspace(rows, vocab, code(zs, dtype)),
                                 dtype=torch.uint8, device="cuda")
                zs.zs_logprob(z.cuda(), ids.cuda(), out, temperature=tau, workspace=ws)
                check(out, want.float(), tol, "logp alone")
                grad = torch.full_like(z, 7.0).cuda()
                adv = torch.full((rows,), 0.5)
                logp, loss = run_policy(zs, z.cuda(), ids, tau, adv, None, None, None, 64.0, grad)
                check(logp, want.float(), tol, "logp")
                slope = torch.full((rows,), -32.0 / float(torch.tensor(tau)), dtype=F64)
                wg = ref.logit_grad(q, ids, slope)
                delta = errors(z.clamp(-60, 60), tau, want)[0]
                inner = wg.abs() * (3 * delta.unsqueeze(1) + 2.0 ** -20)
                check(grad, wg, U[dtype] * (wg.abs() + inner) + inner + TINY[dtype], "grad")


def cold_logits(rows, vocab, size, dtype, g):
    """Logits, tokens that are a row's largest in every other row, and in fp32 rows that have
    others next to the largest."""
    z = (2 * size * torch.randn(rows, vocab, generator=g)).to(dtype)
    ids = torch.randint(0, vocab, (rows,), generator=g, dtype=torch.int32)
    ids[::2] = z[::2].float().argmax(1).int()
    if dtype is FP32:
        for r in (1, 2):
            z[r, torch.randint(0, vocab, (3,), generator=g)] = torch.nextafter(
                z[r].max(), torch.tensor(-math.inf))
        ids[1] = int(z[1].argmax())
    return z, ids


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=str)
def test_small_temperatures_and_large_logits(zs, dtype):
    """Exponents far beyond 2^24 units: the largest logit's neighbours have nothing, but of fp32
    some, and ties share.

    Tolerance: an exponent e of a term has errors of 2^-24 |e| from c and from its own rounding,
    and of 2^-24 128 where it is formed by a whole number up to 128 away: with those terms that
    matter within 128 of the largest, 2^-15 of a term; a log-probability 2^-21 of itself beside
    that. An exponential below 2^-126 is 0."""
    sizes = [(1e-6, 1), (1e-7, 1), (3e-9, 1), (1e-9, 1), (1e-10, 1), (1e-13, 1), (1e-17, 1),
             (1e-18, 1), (1e-20, 1), (1e-30, 1), (2.0 ** -126, 1)]
    if dtype is not FP16:
        sizes += [(1.0, 3e7), (1.0, 1e9), (1.0, 1e13), (1.0, 1e17), (0.5, 1e30)]
    for rows, vocab in ((6, 1000), (6, 70000), (70, 20000)):
        for tau, size in sizes:
            announce(f"cold {dtype} {tau} {size} {rows}x{vocab}")
            z, ids = cold_logits(rows, vocab, size, dtype, gen("cold", rows, vocab, tau, size))
            tau32 = float(torch.tensor(tau))
            want, q, _ = ref.logprob(z.double(), ids, tau32)
            tol = 2.0 ** -15 + 2.0 ** -21 * want.abs()
            out = torch.full((rows,), 9.0, device="cuda")
            ws = torch.empty(zs.zs_logprob_workspace(rows, vocab, code(zs, dtype)),
                             dtype=torch.uint8, device="cuda")
            zs.zs_logprob(z.cuda(), ids.cuda(), out, temperature=tau, workspace=ws)
            check(out, want.float(), tol, "logp alone")
            grad = torch.full_like(z, 7.0).cuda()
            logp, loss = run_policy(zs, z.cuda(), ids, tau, torch.ones(rows), None, None, None,
                                    64 * tau32, grad)
            check(logp, want.float(), tol, "logp")
            assert bool((loss == -1).all())

            def near(got, slope, what):
                wg = ref.logit_grad(q[:len(slope)], ids[:len(slope)], slope)
                check(got, wg, (U[dtype] + 2.0 ** -14) * wg.abs() + 64 * 2.0 ** -125, what)

            near(grad, torch.full((rows,), -64.0, dtype=F64), "grad")
            if tau32 < 1e-17 or size > 1e17:
                continue
            # a pair's slope is beta's, whatever its difference of up to 1e19
            grad.fill_(7.0)
            loss, seq = run_preference(zs, z.cuda(), ids, [0, 2, 4], grad, None, beta=1e-30,
                                       kind=zs.ZS_PREFERENCE_HINGE, temperature=tau,
                                       loss_scale=64e30 * tau32)
            sums = torch.stack([want[:2].sum(), want[2:4].sum()])
            check(seq, sums, 2 * (2.0 ** -15 + 2.0 ** -21 * want[:4].abs().max()), "seq_logp")
            near(grad[:4], torch.tensor([-64.0, -64.0, 64.0, 64.0], dtype=F64), "pair grad")
