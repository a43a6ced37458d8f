"""The output end's operators where 32 bits, or the matrix unit, could lose what
counts: against their 64-bit plain forms, at the tolerances' derivation given
with each test."""
import math

import pytest
import torch

import ops_reference as ref
from gpu_util import announce
from test_gpu_ops import BF16, FP16, FP32, F64, TINY, U, close, fmt_of, gen, randn, zs  # noqa: F401

pytestmark = pytest.mark.gpu

# (m, n, k, workspace): few rows, tiles, tiles split along k, large tiles
PRODUCT = [(1, 100, 4096, False), (16, 333, 640, False), (30, 64, 128, False),
           (100, 130, 384, False), (140, 300, 8192, True), (1300, 7000, 512, False)]


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=str)
def test_product_keeps_what_cancellation_leaves(zs, dtype):
    """Of every eight neighbouring products of an 8-bit A, two large ones cancel and
    the others remain. Terms are multiples of 2^-10, and every sum of the remaining
    ones stays below 2^13: exact in fp32, so the one rounding is the result's."""
    for m, n, k, split in PRODUCT:
        announce(f"cancellation {dtype} {m}x{n}x{k}")
        g = gen("cancel", m, n, k)
        ac = torch.randint(0, 64, (m, k), generator=g, dtype=torch.uint8)   # below 2
        ac |= torch.randint(0, 2, (m, k), generator=g, dtype=torch.uint8) << 7
        ac[:, 0::8] = ac[:, 1::8] = 0x7e                                    # 448
        code = torch.randint(0, 16, (n, k), generator=g, dtype=torch.uint8)
        code[:, 0::8], code[:, 1::8] = 7, 15                                # 6 and -6
        bc = code[:, 0::2] | code[:, 1::2] << 4
        one = [torch.full((r, k // 32), 127, dtype=torch.uint8) for r in (m, n)]
        a, b = ref.mx_values(ac, one[0], "e4m3", k), ref.mx_values(bc, one[1], "e2m1", k)
        want = (a.cuda() @ b.cuda().t()).cpu()
        assert float(want.abs().max()) < 2.0 ** 13
        out = torch.empty(m, n, dtype=dtype, device="cuda")
        ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda") if split else None
        zs.zs_mx_matmul(ac.cuda(), one[0].cuda(), zs.ZS_MX_E4M3, bc.cuda(), one[1].cuda(), out, k,
                        workspace=ws)
        assert torch.equal(out.cpu(), want.to(dtype))


@pytest.mark.parametrize("kind", ["every code", "few large"])
def test_product_of_8_bits_adds_up_in_32(zs, kind):
    """Tolerance: half a step of the result, and one fp32 rounding for each half's
    step of 64 elements of K and each piece that is joined."""
    for m, n, k, split in PRODUCT:
        announce(f"8-bit sums, {kind}, {m}x{n}x{k}")
        g = gen("sums", kind, m, n, k)
        ac = torch.randint(0, 256, (m, k), generator=g, dtype=torch.uint8)
        if kind == "few large":
            large = torch.randint(0, 32, (m, k), generator=g) == 0
            ac = torch.where(large, ac | 0x70, ac & 0x9f)
        ac[(ac & 127) == 127] = 1                                           # not NaN
        bc = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
        asc, bsc = (torch.randint(120, 128, (r, k // 32), generator=g, dtype=torch.uint8)
                    for r in (m, n))
        a, b = (ref.mx_values(c, s, f, k).cuda()
                for c, s, f in ((ac, asc, "e4m3"), (bc, bsc, "e2m1")))
        want, mag = (a @ b.t()).cpu(), (a.abs() @ b.abs().t()).cpu()
        out = torch.empty(m, n, dtype=BF16, device="cuda")
        ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda") if split else None
        zs.zs_mx_matmul(ac.cuda(), asc.cuda(), zs.ZS_MX_E4M3, bc.cuda(), bsc.cuda(), out, k,
                        workspace=ws)
        acc = (2 * k / 64 + 10) * 2.0 ** -24 * mag
        close(out, want, U[BF16] * (want.abs() + acc) + acc + TINY[BF16], f"{m}x{n}x{k}")


# ---- distillation --------------------------------------------------------------

def distill(zs, z, ids, t, tau=1.0, lse=None, w=None, scale=1.0, grad=None):
    """(loss, gradient) of the kernels, on the CPU."""
    r, v = z.shape
    loss = torch.empty(r, device="cuda")
    grad = torch.empty(r, v, dtype=z.dtype, device="cuda") if grad is None else grad
    need = zs.zs_distill_workspace(r, v, ids.shape[1], zs._float_code(z, "z", True))
    gpu = [None if x is None else x.cuda() for x in (z, ids, t, lse, w)]
    zs.zs_distill(*gpu[:3], tau, loss, grad=grad, teacher_lse=gpu[3], row_weight=gpu[4],
                  loss_scale=scale,
                  workspace=torch.empty(max(need, 16), dtype=torch.uint8, device="cuda"))
    return loss.cpu(), grad.cpu()


@pytest.mark.parametrize("rows,vocab,dt", [(3, 349189, FP32), (1, 1048585, FP32),
                                           (2, 1048585, BF16), (1, 2097165, FP16)], ids=str)
@pytest.mark.parametrize("tail", [False, True])
def test_distill_slots_at_the_end_of_a_long_row(zs, rows, vocab, dt, tail):
    """Every slot's gradient holds its p, wherever its token lies. Tolerance: U of the
    type, and 2^-19 of q + p for exponents, sums and products in fp32."""
    announce(f"distill {dt} tail={tail} {rows}x{vocab}")
    g = gen("end", rows, vocab)
    z = torch.randn(rows, vocab, generator=g).to(dt)
    ids = (vocab - 1 - torch.arange(40)).expand(rows, 40).contiguous().int()
    ids[:, 30:] = torch.randint(0, vocab // 2, (rows, 10), generator=g, dtype=torch.int32)
    t = torch.randn(rows, 40, generator=g).to(dt)
    lse = (torch.logsumexp(t.double(), 1) + 0.3).float() if tail else None
    loss, grad = distill(zs, z, ids, t, lse=lse, scale=64.0)
    want, wgrad, bound = ref.distill(z, ids, t, 1.0, lse, None, 64.0)
    at = ids.long()
    acc = 2.0 ** -19 * bound.gather(1, at)
    close(grad.gather(1, at), wgrad.gather(1, at),
          U[dt] * (wgrad.gather(1, at).abs() + acc) + acc + TINY[dt], "slots' gradients")
    # terms of the size of the logits' spread (below 20), each to 2^-20
    close(loss, want, 20 * 2.0 ** -20 + want.abs() * 2.0 ** -20, "loss")
