"""A student's last block and head as a user runs them: every part of a step
against its 64-bit form, given the operands that the call before it left in
memory; dropout, padding, the shard step's skip, and the example."""
import math
import os
import sys

import pytest
import torch

import block_reference as blk
import linear_reference as lin
import ops_reference as ops
import token_reference as tok
from conftest import ROOT
from gpu_util import announce

pytestmark = pytest.mark.gpu
F64, BF16 = torch.float64, torch.bfloat16
ROWS, WIDTH, HIDDEN, VOCAB = 96, 192, 320, 700
U = 2.0 ** -8                            # half a step of bfloat16


@pytest.fixture(scope="module")
def zs(hip_built):
    from sharded_mixed_precision_zs_amd import zeroshard
    return zeroshard


def problem(block, head, seed=0):
    g = torch.Generator().manual_seed(seed)
    parts = []
    for shape in block.shapes + ((WIDTH,), (VOCAB, WIDTH)):
        t = torch.randn(*shape, generator=g)
        parts.append(((1 + 0.1 * t) if shape == (WIDTH,) else 0.06 * t).flatten())
    x, res = (torch.randn(ROWS, WIDTH, generator=g).to(BF16) for _ in range(2))
    ids = torch.randint(0, VOCAB, (ROWS,), generator=g, dtype=torch.int32)
    ids[::9] = -1
    return torch.cat(parts).to(BF16), x, res, ids, g


def near(got, want, tol, what):
    err = (got.double().cpu() - want).abs()
    assert bool((err <= tol).all()), f"{what}: worst {float((err / tol.clamp(min=1e-300)).max()):.3g}"


def back(t):
    return t.cpu().double()


def product_bits(zs, out, a, b, k):
    """The product's own bits for the 64-bit form's quantisation of a and b."""
    ac, asc, _ = ops.mx_quantize(a, "e4m3")
    bc, bsc, _ = ops.mx_quantize(b, "e2m1")
    want = torch.empty_like(out)
    ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    zs.zs_mx_matmul(ac.cuda(), asc.cuda(), zs.ZS_MX_E4M3, bc.cuda(), bsc.cuda(), want, k,
                    workspace=ws)
    return torch.equal(out, want)


def parts(zs, kind):
    from sharded_mixed_precision_zs_amd.block import BlockStudent, MlpBlock
    from sharded_mixed_precision_zs_amd.head import PolicyHead, PreferenceHead
    block = MlpBlock(ROWS, WIDTH, HIDDEN, dropout=0.25, seed=77, residual_scale=0.75,
                     branch_scale=0.5)
    head = PolicyHead(ROWS, WIDTH, VOCAB, clip_high=0.28, kl_weight=0.05) if kind == "policy" else \
        PreferenceHead(ROWS, WIDTH, VOCAB, 2, 0.25, smoothing=0.1)
    return BlockStudent(block, head)


@pytest.mark.parametrize("kind", ["policy", "preference"])
def test_every_part_of_a_step_against_64_bits(zs, kind):
    announce(f"student step {kind}")
    student = parts(zs, kind)
    block, head = student.block, student.head
    params, x, res, ids, g = problem(block, head)
    scale = 512.0
    starts = [0, 20, 45, 60, 90]                       # six rows of padding behind
    adv = torch.randn(ROWS, generator=g)
    loss_args = dict(advantage=adv.cuda()) if kind == "policy" else \
        dict(starts=torch.tensor(starts, dtype=torch.int32).cuda())
    logits = student.forward(params.cuda(), x.cuda(), res.cuda(), offset=5).clone()
    logp = tok.logprob(back(logits), ids, 1.0)[0]
    if kind == "policy":
        old = (logp - 0.5 * torch.randn(ROWS, generator=g)).float()
        refs = (logp + 0.3 * torch.randn(ROWS, generator=g)).float()
        loss_args.update(old_logp=old.cuda(), ref_logp=refs.cuda())
    loss = student.step(params.cuda(), x.cuda(), res.cuda(), offset=5, ids=ids.cuda(),
                        loss_scale=scale, **loss_args)
    torch.cuda.synchronize()
    mine, heads = student.split(params.double())
    gain0, w1, b1, w2, b2, post, gate = block.split(mine)
    gain, wh = head.split(heads)
    # forward
    h0 = (x.float() + res.float()).to(BF16).double()
    assert torch.equal(back(block.h0), h0)
    y0 = blk.rounded(ops.rmsnorm(h0, gain0, 1e-5)[0], BF16)
    near(block.y0, y0, U * y0.abs() * 1.01 + 1e-30, "y0")
    y8 = ops.mx_values(block._y8[0].cpu(), block._y8[1].cpu(), "e4m3", WIDTH)
    for out, a, w, b, act, pre in ((block.a, y8, w1, b1, "gelu", block.pre),
                                   (block.o, ops.mx_quantize(back(block.a), "e4m3")[2], w2, b2,
                                    "none", None)):
        w4 = ops.mx_quantize(w, "e2m1")[2]
        p = a @ w4.t() + b
        acc = (2 * a.shape[1] / 64 + 3) * 2.0 ** -24 * (a.abs() @ w4.abs().t() + b.abs())
        c = lin.activate(p, act)
        near(out, c, U * c.abs() + 1.2 * acc + c.abs() * 2.0 ** -18, "linear")
        if pre is not None:
            near(pre, p, U * p.abs() + 1.1 * acc, "pre")
    factor = blk.keep_factor(ROWS, WIDTH, 0.25, 77, 5)
    h, _, post_rstd, rstd, y = blk.block(back(block.o), h0, post, gate, gain, float(
        torch.tensor(1e-5)), 0.75, 0.5, factor, BF16)
    assert torch.equal(back(head.h), h)
    assert torch.equal(head._y8[0].cpu(), ops.mx_quantize(y, "e4m3")[0])
    w4 = ops.mx_quantize(wh, "e2m1")[2]
    y8 = ops.mx_values(head._y8[0].cpu(), head._y8[1].cpu(), "e4m3", WIDTH)
    z = y8 @ w4.t()
    near(logits, z, U * z.abs() + (2 * WIDTH / 64 + 2) * 2.0 ** -23 * (y8.abs() @ w4.abs().t()),
         "logits")
    # the loss's gradient, in the logits' place
    z = back(logits)
    q = torch.softmax(z, 1)
    if kind == "policy":
        _, want, dz, mag = tok.policy(z, ids, 1.0, adv.double(), old.double(), refs.double(),
                                      *(float(torch.tensor(v)) for v in (0.2, 0.28, 0.05)), None,
                                      scale)
        near(loss, want, 1e-5 * (mag / scale + want.abs()) + 1e-6, "loss")
    else:
        want, _, dz, mag, inside = tok.preference(z, ids, starts, 1.0, None, "sigmoid", 0.25,
                                                  float(torch.tensor(0.1)), False, None, scale)
        assert not head.logits[~inside.cuda()].any()
        near(loss, want, 1e-4 * want.abs() + 1e-5, "loss")
    near(head.logits, dz, U * dz.abs() + 1e-4 * (q + dz.abs() / mag.clamp(min=1e-30).unsqueeze(1))
         * mag.unsqueeze(1) + 1e-30, "dlogits")
    # the products back
    dlog = back(head.logits)
    dmine, dheads = student.split(student.grads)
    _, dw1, db1, dw2, db2, dpost, dgate = block.split(dmine)
    assert product_bits(zs, head.dy, dlog, wh.t().contiguous(), VOCAB)
    assert product_bits(zs, head.split(dheads)[1], dlog.t().contiguous(),
                        back(head.y).t().contiguous(), ROWS)
    # the block norm's
    got, bound = blk.block_grad(back(head.dy), h, back(head.rstd), gain, None, back(block.o),
                                back(block.post_rstd), post, gate, 0.75, 0.5, factor)
    for name, t in (("dx", block.do), ("dresidual", block.dh0), ("dgain", head.split(dheads)[0]),
                    ("dpost_gain", dpost), ("dgate", dgate)):
        near(t, got[name], U * got[name].abs() * 1.01 + 2.0 ** -16 * bound[name] + 1e-30, name)
    do = back(block.do)
    near(db2, do.sum(0), U * do.sum(0).abs() * 1.01 + 2.0 ** -16 * do.abs().sum(0) + 1e-30, "db2")
    assert product_bits(zs, dw2, do.t().contiguous(), back(block.a).t().contiguous(), ROWS)
    da = torch.empty(ROWS, HIDDEN, dtype=BF16, device="cuda")
    ac, asc, _ = ops.mx_quantize(do, "e4m3")
    bc, bsc, _ = ops.mx_quantize(w2.t().contiguous(), "e2m1")
    zs.zs_mx_matmul(ac.cuda(), asc.cuda(), zs.ZS_MX_E4M3, bc.cuda(), bsc.cuda(), da, WIDTH,
                    workspace=torch.empty(32 << 20, dtype=torch.uint8, device="cuda"))
    s, sb = lin.slope(back(block.pre), "gelu")
    dpre = back(da) * s
    near(block.da, dpre, U * dpre.abs() * 1.01 + back(da).abs() * sb * 2.0 ** -15 + 1e-30, "dpre")
    near(db1, dpre.sum(0), U * dpre.sum(0).abs() * 1.01
         + 2.0 ** -14 * (back(da).abs() * (sb + s.abs())).sum(0) + 1e-30, "db1")
    assert product_bits(zs, block.dy0, back(block.da), w1.t().contiguous(), HIDDEN)
    assert product_bits(zs, dw1, back(block.da).t().contiguous(), back(block.y0).t().contiguous(),
                        ROWS)
    dx, dg0, xmag, gmag = ops.rmsnorm_grad(back(block.dy0), h0, back(block.rstd0), gain0,
                                           back(block.dh0))
    near(student.dx, dx, U * dx.abs() * 1.01 + 2.0 ** -17 * xmag, "dx")
    near(dmine[:WIDTH], dg0, U * dg0.abs() * 1.01 + 2.0 ** -16 * gmag, "dgain0")


def test_policy_head_and_its_logprobs(zs):
    from sharded_mixed_precision_zs_amd.head import PolicyHead
    head = PolicyHead(ROWS, WIDTH, VOCAB, clip_high=0.28)
    g = torch.Generator().manual_seed(4)
    params = torch.cat([1 + 0.1 * torch.randn(WIDTH, generator=g),
                        0.05 * torch.randn(VOCAB * WIDTH, generator=g)]).to(BF16).cuda()
    x, res = (torch.randn(ROWS, WIDTH, generator=g).to(BF16).cuda() for _ in range(2))
    ids = torch.randint(0, VOCAB, (ROWS,), generator=g, dtype=torch.int32).cuda()
    adv = torch.randn(ROWS, generator=g).cuda()
    old = head.logprobs(params, x, res, ids).clone()
    loss = head.step(params, x, res, ids, adv, old_logp=old, loss_scale=64.0)
    # the ratio is 1: the loss is the advantage's, and log-probabilities are the sampler's. The two
    # kernels add a row's terms in orders of their own: each is within 2 (2 D + 38) 2^-24 of the
    # exact one, D the row's spread, and these rows' is below 16 (7 standard deviations of 0.7
    # either way): 1.7e-5 between the two, and as much of the ratio
    assert bool(((head.logp - old).abs() <= 1.7e-5).all())
    assert bool(((loss + adv).abs() <= 2e-5 * adv.abs()).all())
    assert torch.isfinite(head.grads.float()).all() and head.grads.float().abs().max() > 0


def test_example_runs_and_has_its_gradients(zs):
    """The example: it runs, and every parameter has a finite gradient that is not zero."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import tune_student
    losses, student, st = tune_student.train(steps=2, pairs=2, length=16, width=128, hidden=160,
                                             vocab=300, report=announce)
    assert len(losses) == 2 and all(math.isfinite(v) for v in losses)
    assert st.t + int(st.scaler.skipped) == 2
    assert torch.isfinite(student.grads.float()).all()
    for t in student.block.split(student.split(student.grads)[0]):
        assert t.float().abs().max() > 0


def test_student_overflow_is_skipped(zs):
    """fp16 gradients beyond their range: the device skips the step and halves the scale."""
    from sharded_mixed_precision_zs_amd import shard
    from sharded_mixed_precision_zs_amd.block import BlockStudent, MlpBlock
    from sharded_mixed_precision_zs_amd.head import PolicyHead
    half = torch.float16
    student = BlockStudent(MlpBlock(ROWS, WIDTH, HIDDEN, dtype=half, dropout=0.1),
                           PolicyHead(ROWS, WIDTH, VOCAB, dtype=half))
    params, x, res, ids, g = problem(student.block, student.head)
    st = shard.ShardState(student.phi, 1, 0, 0, student.phi, zs.ZS_FP16, zs.ZS_FP16, shard.AdamW(),
                          loss_scale=2.0 ** 24, dynamic=True, growth_interval=1000,
                          device_commit=True)
    start = params.to(half).cuda()
    st.fill_state(lambda first, count, m0, m, v: (m0.copy_(start[first:first + count].float()),
                                                  m.zero_(), v.zero_()))
    st.params.copy_(start)
    adv = torch.randn(ROWS, generator=g).cuda()
    for i in range(2):
        student.step(st.params, x.to(half).cuda(), res.to(half).cuda(), offset=i, ids=ids.cuda(),
                     advantage=adv, dev_scaler=st.dev)
        st.step_device([student.grads])
    st.sync_scaler()
    assert int(st.scaler.skipped) == 2 and st.loss_scale == 2.0 ** 22
    assert torch.equal(st.params, start)


def test_student_step_captured_and_replayed(zs):
    """A captured step whose dropout offset lies on the device: every replay is the eager step of
    its own offset."""
    student = parts(zs, "policy")
    params, x, res, ids, g = problem(student.block, student.head)
    args = (params.cuda(), x.cuda(), res.cuda())
    adv = torch.randn(ROWS, generator=g).cuda()
    more = dict(ids=ids.cuda(), advantage=adv, loss_scale=64.0)
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    student.step(*args, offset=(10, count), **more)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        student.step(*args, offset=(10, count), **more)
        count += 1
    seen = []
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        seen.append((student.grads.clone(), student.dx.clone(), student.head.loss.clone()))
        student.step(*args, offset=10 + i, **more)
        torch.cuda.synchronize()
        for a, b in zip(seen[-1], (student.grads, student.dx, student.head.loss)):
            assert torch.equal(a, b)
    assert not torch.equal(seen[0][0], seen[1][0])


def test_block_and_head_must_match(zs):
    from sharded_mixed_precision_zs_amd.block import BlockStudent, MlpBlock
    from sharded_mixed_precision_zs_amd.head import PolicyHead
    with pytest.raises(ValueError):
        BlockStudent(MlpBlock(8, 64, 64), PolicyHead(8, 128, 100))


@pytest.mark.parametrize("kind", ["policy", "preference", "distill"])
def test_students_logprobs(zs, kind):
    """Of block and head together, without dropout or with an offset's: the 64-bit
    log-probabilities of the logits that forward() leaves."""
    from sharded_mixed_precision_zs_amd.block import BlockStudent, MlpBlock
    from sharded_mixed_precision_zs_amd.head import DistillHead
    student = parts(zs, kind) if kind != "distill" else BlockStudent(
        MlpBlock(ROWS, WIDTH, HIDDEN, dropout=0.25, seed=77), DistillHead(ROWS, WIDTH, VOCAB, 4))
    params, x, res, ids, _ = problem(student.block, student.head)
    args = (params.cuda(), x.cuda(), res.cuda())
    seen = []
    for offset in (None, 5):
        got = student.logprobs(*args, ids.cuda(), **({} if offset is None else {"offset": offset}))
        z = student.forward(*args, offset=offset).clone()
        assert torch.equal(z, student.head.logits)
        want = tok.logprob(back(z), ids, 1.0)[0]
        # each is within 2 (2 D + 38) 2^-24, D the row's spread, here below 40
        near(got, want, torch.full_like(want, 1.5e-5) + 2.0 ** -23 * want.abs(), "logp")
        assert not got.cpu()[ids < 0].any()
        seen.append(z)
    keep, student.block.dropout = student.block.dropout, 0.0
    assert torch.equal(student.forward(*args, offset=5), seen[0])
    student.block.dropout = keep
    assert not torch.equal(seen[0], seen[1])
