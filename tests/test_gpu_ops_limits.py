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


def distill_close(z, got, want, tau, dt):
    """A term's exponent carries two roundings of 2^-24 of its size, and the exp, the sums
    and the products some 2^-19: of q + p on the slots, of q + pr q / qr off them."""
    (loss, grad), (wloss, wgrad, bound) = got, want
    arg = ((z.double().amax(1, keepdim=True) - z.double()) / tau).clamp(max=90)
    acc = (wgrad.abs() + 2 * bound) * (arg * 2.0 ** -22 + 2.0 ** -19)
    close(grad, wgrad, U[dt] * (wgrad.abs() + acc) + acc + TINY[dt], "gradient")
    # the loss: terms of the size of the logits' spread, weighted by p and pr
    close(loss, wloss, (arg.amax(1) + 20) * 2.0 ** -20 * tau * tau, "loss")


@pytest.mark.parametrize("vocab", [1003, 40000, 140001])   # short and long rows, and in parts
@pytest.mark.parametrize("dt,tau,gap", [(FP32, 1.0, 20), (FP32, 1.0, 35), (FP32, 1.0, 45),
                                        (FP32, 1.0, 60), (FP32, 1.0, 80), (BF16, 0.5, 22),
                                        (FP16, 0.5, 30), (BF16, 1.0, 60)], ids=str)
def test_distill_with_little_mass_off_the_slots(zs, vocab, dt, tau, gap):
    """A student that is sure of its slots, the teacher less so: what the student has off
    them counts however little it is."""
    announce(f"gap {gap} {dt} tau {tau} vocabulary {vocab}")
    g = gen("gap", vocab, gap)
    z = torch.randn(3, vocab, generator=g) * 0.5
    ids = torch.stack([torch.randperm(vocab, generator=g)[:32] for _ in range(3)]).int()
    ids[0, :4] = torch.tensor([0, 1, vocab - 1, vocab - 2])    # the ends
    ids[0, 4:] = torch.arange(16, 44)
    ids[1, 5], ids[1, 6] = ids[1, 4], -1                       # one twice, one empty
    z.scatter_add_(1, ids.clamp(min=0).long(), torch.full((3, 32), float(gap)))
    z[1, int(ids[1, 4])] = float(gap)
    z = z.to(dt)
    t = torch.randn(3, 32, generator=g).to(dt)
    kept = torch.where(ids >= 0, t.double() / tau, -math.inf)
    lse = (torch.logsumexp(kept, 1) + 0.1).float()
    want = ref.distill(z, ids, t, tau, lse, None, 64.0)
    assert torch.isfinite(want[0]).all()
    distill_close(z, distill(zs, z, ids, t, tau, lse, None, 64.0), want, tau, dt)
    if dt == FP32:   # in place, and a gradient whose rows are aligned otherwise
        place = z.cuda()
        loss, grad = distill(zs, place, ids, t, tau, lse, None, 64.0, grad=place)
        distill_close(z, (loss, grad), want, tau, dt)
        wide = torch.empty(3, vocab + 3, device="cuda")
        distill_close(z, distill(zs, z, ids, t, tau, lse, None, 64.0, grad=wide[:, 1:vocab + 1]), want,
                      tau, dt)


@pytest.mark.parametrize("vocab", [5000, 140001])
@pytest.mark.parametrize("gap", [30, 95, 140])
def test_distill_down_to_the_smallest_mass(zs, vocab, gap):
    """Terms reach down to 2^-222 of a row's largest, e^-153."""
    announce(f"gap {gap} vocabulary {vocab}")
    g = gen("least", vocab, gap)
    z = torch.randn(2, vocab, generator=g) * 0.5
    ids = torch.stack([torch.randperm(vocab, generator=g)[:20] for _ in range(2)]).int()
    z.scatter_add_(1, ids.long(), torch.full((2, 20), float(gap)))
    t = torch.randn(2, 20, generator=g)
    lse = (torch.logsumexp(t.double(), 1) + 0.2).float()
    want = ref.distill(z, ids, t, 1.0, lse)
    got = distill(zs, z, ids, t, 1.0, lse)
    # exponents of up to 150, beyond distill_close's 90
    (loss, grad), (wloss, wgrad, bound) = got, want
    acc = (wgrad.abs() + 2 * bound) * ((gap + 10) * 2.0 ** -22 + 2.0 ** -19)
    close(grad, wgrad, U[FP32] * (wgrad.abs() + acc) + acc + TINY[FP32], "gradient")
    close(loss, wloss, (gap + 30) * 2.0 ** -20, "loss")


@pytest.mark.parametrize("vocab", [2000, 140001])
@pytest.mark.parametrize("level,tau", [(1, 1.0), (20, 1.0), (40, 1.0), (-200, 1.0), (200, 1.0),
                                       (20, 0.7), (6, 0.1)])
@pytest.mark.parametrize("dt", [BF16, FP32], ids=str)
def test_distill_of_a_teacher_with_all_its_mass_on_the_slots(zs, vocab, level, tau, dt):
    """What rounding leaves of the teacher's mass is none: a student that has none off
    the slots either gets a finite loss. The teacher's probabilities are off by the
    rounding of its logsumexp, 2^-24 of its size, and 2^-19; the loss by that of terms
    of the size of the spread, below 20."""
    rows, k = 200 if vocab == 2000 else 20, 16
    announce(f"level {level} tau {tau} {dt} {rows}x{vocab}")
    g = gen("full", vocab, level, tau)
    t = (torch.randn(rows, k, generator=g) * tau + level).to(dt)
    ids = (torch.arange(k) * 3).expand(rows, k).contiguous().int()
    z = torch.full((rows, vocab), -math.inf)
    z.scatter_(1, ids.long(), torch.randn(rows, k, generator=g) * tau)
    z = z.to(dt)
    lse = torch.logsumexp(t.double() / tau, 1)
    want, wgrad, bound = ref.distill(z, ids, t, tau, lse, None, 8.0)   # the exact one
    loss, grad = distill(zs, z, ids, t, tau, lse.float(), None, 8.0)
    off = float(lse.abs().max()) * 2.0 ** -24 + 2.0 ** -19
    close(loss, want, 20 * off * tau * tau, "loss")
    close(grad, wgrad, U[dt] * wgrad.abs() + 2 * bound * off + TINY[dt], "gradient")


# ---- norm ----------------------------------------------------------------------

@pytest.mark.parametrize("size", [1e30, 1e25, 1e19, 1e-19, 1e-25, 1e-30])
@pytest.mark.parametrize("cols", [256, 1000, 5000])
def test_norm_of_rows_whose_squares_leave_32_bits(zs, size, cols):
    """Tolerances as for other rows: y's one rounding and a few of fp32; backward a
    chain of 64 + 6 + 16 additions and a handful of products."""
    announce(f"norm of size {size:g} x {cols}")
    g = gen("size", size, cols)
    h = (randn(g, 4, cols) * size).to(BF16)
    gain, dy = (1 + 0.2 * randn(g, cols)).to(BF16), (randn(g, 4, cols) * 0.1).to(BF16)
    want, wr = ref.rmsnorm(h.double(), gain.double(), 0.0)
    y, rstd = torch.empty(4, cols, dtype=BF16, device="cuda"), torch.empty(4, device="cuda")
    codes, scales = zs.mx_empty(4, cols, zs.ZS_MX_E4M3)
    zs.zs_rmsnorm_forward(h.cuda(), gain.cuda(), 0.0, y=y, rstd=rstd, codes=codes, scales=scales)
    few = 4 * 2.0 ** -24
    close(rstd, wr, few * wr, "rstd")
    close(y, want, (U[BF16] * (1 + few) + few) * want.abs() + TINY[BF16], "y")
    got, byte = ref.mx_values(codes.cpu(), scales.cpu(), "e4m3", cols), scales.cpu()
    s = ref.pow2(byte.long() - 127).repeat_interleave(32, 1)[:, :cols]
    tol = torch.maximum(want.abs() * 2.0 ** -4, s * 2.0 ** -10)
    close(got, want, torch.where(want.abs() > 448 * s, want.abs() - 448 * s + tol, tol)
          + few * want.abs(), "8-bit y")
    dx, dgain = torch.empty_like(y), torch.empty(cols, device="cuda")
    ws = torch.empty(zs.zs_rmsnorm_backward_workspace(4, cols), dtype=torch.uint8, device="cuda")
    zs.zs_rmsnorm_backward(dy.cuda(), h.cuda(), rstd, gain.cuda(), dx, dgain, ws)
    wdx, wdg, mag, gmag = ref.rmsnorm_grad(dy.double(), h.double(), rstd.cpu().double(),
                                           gain.double(), None)
    acc = (64 + 6 + 16 + 8) * 2.0 ** -24 * mag
    close(dx, wdx, U[BF16] * (wdx.abs() + acc) + acc + TINY[BF16], "dx")
    close(dgain, wdg, 36 * 2.0 ** -24 * gmag + 1e-37, "dgain")


# ---- the head's backward products ----------------------------------------------

def test_head_backward_products_against_64_bits(zs):
    """Logits' gradients have a few large entries in a row: both products of them against
    64 bits, at the tolerance of test_product_of_8_bits_adds_up_in_32."""
    from sharded_mixed_precision_zs_amd.head import DistillHead
    rows, width, vocab, slots = 300, 256, 5000, 8
    announce("head backward products")
    g = gen("head")
    params = torch.cat([torch.ones(width), 0.05 * randn(g, vocab * width)]).to(BF16)
    ids = torch.randint(0, vocab, (rows, slots), generator=g, dtype=torch.int32)
    head = DistillHead(rows, width, vocab, slots)
    head.step(params.cuda(), randn(g, rows, width).to(BF16).cuda(),
              randn(g, rows, width).to(BF16).cuda(), ids.cuda(),
              (3 * randn(g, rows, slots)).to(BF16).cuda(), loss_scale=1024.0)
    torch.cuda.synchronize()
    grad, y = head.logits.cpu().double(), head.y.cpu().double()
    weight = head.split(params)[1].double()
    for out, a, b, k in ((head.dy, grad, weight.t().contiguous(), vocab),
                         (head.split(head.grads)[1], grad.t().contiguous(), y.t().contiguous(), rows)):
        a, b = ref.mx_quantize(a, "e4m3")[2], ref.mx_quantize(b, "e2m1")[2]
        want, mag = a @ b.t(), a.abs() @ b.abs().t()
        acc = (2 * zs.mx_padded(k) / 64 + 10) * 2.0 ** -24 * mag
        close(out, want, U[BF16] * (want.abs() + acc) + acc + TINY[BF16], f"k {k}")


@pytest.mark.parametrize("dt,rows,cols", [(BF16, 2048, 4096), (FP16, 4096, 2048), (BF16, 5000, 1001)],
                         ids=str)
def test_norm_rounds_once(zs, dt, rows, cols):
    """Every code, scale and 16-bit y of millions is the 64-bit result's: rounding to fp32
    in between would put several on the other side of a tie or a power of two."""
    announce(f"norm rounds once {dt} {rows}x{cols}")
    g = torch.Generator("cuda").manual_seed(cols)
    h = torch.randn(rows, cols, generator=g, device="cuda").to(dt)
    gain = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(dt)
    y = torch.empty(rows, cols, dtype=dt, device="cuda")
    codes, scales = zs.mx_empty(rows, cols, zs.ZS_MX_E4M3)
    eps = 2.0 ** -17                                           # the same in 32 and 64 bits
    zs.zs_rmsnorm_forward(h, gain, eps, y=y, codes=codes, scales=scales)
    want = ref.rmsnorm(h.double(), gain.double(), eps)[0].cpu()
    wrong = 0
    for first in range(0, rows, 512):
        part = slice(first, first + 512)
        c, s, _ = ref.mx_quantize(want[part], "e4m3")
        wrong += int((codes[part].cpu() != c).sum()) + int((scales[part].cpu() != s).sum())
    # torch rounds binary64 to 16 bits by way of fp32: y within half a step of the 64 bits
    step = torch.where(want == 0, 0.0, torch.ldexp(torch.ones_like(want), torch.frexp(want).exponent - 1))
    step = (step * torch.finfo(dt).eps).clamp(min=2 * TINY[dt])
    over = (y.cpu().double() - want).abs() > step / 2 * (1 + 2.0 ** -40)
    assert wrong == 0 and not bool(over.any()), (wrong, int(over.sum()))
