"""The student's output end as a user runs it: one step's parts against their
64-bit forms, training that lowers the loss
with the shard step, and a skipped step."""
import os
import sys

import pytest
import torch

import ops_reference as ref
from conftest import ROOT
from gpu_util import announce

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.fixture(scope="module")
def zs(hip_built):
    from sharded_mixed_precision_zs_amd import zeroshard
    return zeroshard


def problem(rows, width, vocab, slots, seed=0):
    g = torch.Generator().manual_seed(seed)
    x, res = (torch.randn(rows, width, generator=g).bfloat16() for _ in range(2))
    params = torch.cat([1 + 0.1 * torch.randn(width, generator=g),
                        0.05 * torch.randn(vocab * width, generator=g)]).bfloat16()
    ids = torch.stack([torch.randperm(vocab, generator=g)[:slots] for _ in range(rows)]).int()
    teacher = torch.randn(rows, slots, generator=g).bfloat16()
    return x, res, params, ids, teacher


def test_head_gradients_against_64_bits(zs):
    """Every part of the step, given the operands that the kernel before it left
    in memory."""
    from sharded_mixed_precision_zs_amd.head import DistillHead
    rows, width, vocab, slots = 96, 192, 700, 12
    announce("head step")
    x, res, params, ids, teacher = problem(rows, width, vocab, slots)
    head = DistillHead(rows, width, vocab, slots, temperature=2.0)
    head.step(params.cuda(), x.cuda(), res.cuda(), ids.cuda(), teacher.cuda(), loss_scale=1024.0)
    torch.cuda.synchronize()
    h = (x.float() + res.float()).bfloat16()
    assert torch.equal(head.h.cpu(), h)
    gain, weight = (t.double() for t in head.split(params))
    y8 = ref.mx_values(head._y8[0].cpu(), head._y8[1].cpu(), "e4m3", width)
    w4 = ref.mx_quantize(weight, "e2m1")[2]
    logits = y8 @ w4.t()
    # logits are rounded to 16 bits before the loss: their own rounding, through the softmax,
    # is 2^-9 of their size; 8-bit operands' sums and the gradient's 16 bits come on top
    loss, dlogits, bound = ref.distill(logits.bfloat16(), ids, teacher, 2.0, scale=1024.0)
    spread = float(logits.abs().max()) * 2.0 ** -8
    assert float((head.loss.cpu().double() - loss).abs().max()) < 4 * spread + 1e-4
    got = head.logits.cpu().double()
    assert bool(((got - dlogits).abs() <= bound * (2 * spread + 2.0 ** -8) + 1e-6).all())
    # the backward products: the very bits that the product gives for the 64-bit form's
    # quantisation of the gradient as it lies in memory (its own accuracy is tested apart)
    gt, yt = got.t().contiguous(), head.y.cpu().double().t().contiguous()
    for out, a, b, k in ((head.dy, got, weight.t().contiguous(), vocab),
                         (head.split(head.grads)[1], gt, yt, rows)):
        ac, asc, _ = ref.mx_quantize(a, "e4m3")
        bc, bsc, _ = ref.mx_quantize(b, "e2m1")
        want = torch.empty_like(out)
        ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
        zs.zs_mx_matmul(ac.cuda(), asc.cuda(), zs.ZS_MX_E4M3, bc.cuda(), bsc.cuda(), want, k,
                        workspace=ws)
        assert torch.equal(out, want)
    dx, dgain, xmag, gmag = ref.rmsnorm_grad(head.dy.cpu().double(), h.double(),
                                             head.rstd.cpu().double(), gain, None)
    assert bool(((head.dx.cpu().double() - dx).abs() <= 2.0 ** -8 * dx.abs() + 2.0 ** -17 * xmag).all())
    assert bool(((head.grads[:width].cpu().double() - dgain).abs()
                 <= 2.0 ** -8 * dgain.abs() + 2.0 ** -16 * gmag).all())


def test_head_training_lowers_the_loss(zs):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import distill_head
    losses, st = distill_head.train(steps=61, rows=256, width=128, vocab=1000, slots=16,
                                    report=announce)
    assert st.t == 61 and int(st.scaler.skipped) == 0
    assert losses[-1] < 0.6 * losses[0]


def test_head_overflow_is_skipped(zs):
    """A scale beyond fp16's range: the gradient overflows, the step is skipped and the
    scale halves until it fits; the parameters move only then."""
    from sharded_mixed_precision_zs_amd import shard
    from sharded_mixed_precision_zs_amd.head import DistillHead
    x, res, params, ids, teacher = problem(32, 128, 300, 8)
    half = torch.float16
    head = DistillHead(32, 128, 300, 8, dtype=half)
    st = shard.ShardState(head.phi, 1, 0, 0, head.phi, zs.ZS_FP16, zs.ZS_FP16, shard.AdamW(),
                          loss_scale=2.0 ** 24, dynamic=True, growth_interval=1000,
                          device_commit=True)
    start = params.to(half).cuda()
    st.fill_state(lambda first, count, m0, m, v: (m0.copy_(start[first:first + count].float()),
                                                  m.zero_(), v.zero_()))
    st.params.copy_(start)
    args = [t.cuda() for t in (x.to(half), res.to(half), ids, teacher.to(half))]
    for _ in range(3):
        head.step(st.params, *args, dev_scaler=st.dev)
        st.step_device([head.grads])
    st.sync_scaler()
    assert int(st.scaler.skipped) == 3 and st.loss_scale == 2.0 ** 21
    assert torch.equal(st.params, start)
    for _ in range(12):
        head.step(st.params, *args, dev_scaler=st.dev)
        st.step_device([head.grads])
    st.sync_scaler()
    assert st.t > 0 and not torch.equal(st.params, start)
    assert torch.isfinite(st.params.float()).all()
