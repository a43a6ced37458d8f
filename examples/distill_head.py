"""Distil a teacher's top logits into a small student head on one GPU: the
low-precision forward and backward of `head.DistillHead` and the mixed-precision
shard step of `shard.ShardState`, loss scale and commit-or-skip on the device.

    python examples/distill_head.py [--steps 60] [--rows 512] [--width 256] [--vocab 4096]

Prints the mean loss as it falls. Synthetic data: a fixed teacher head over
random hidden states.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from sharded_mixed_precision_zs_amd import shard, zeroshard as zs  # noqa: E402
from sharded_mixed_precision_zs_amd.head import DistillHead  # noqa: E402


def train(steps=60, rows=512, width=256, vocab=4096, slots=32, lr=3e-3, loss_scale=65536.0,
          report=print):
    """Returns the mean loss of each reported step and the shard state."""
    g = torch.Generator(device="cuda").manual_seed(0)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")

    head = DistillHead(rows, width, vocab, slots)
    st = shard.ShardState(head.phi, 1, 0, 0, head.phi, zs.ZS_BF16, zs.ZS_BF16,
                          shard.AdamW(lr=lr, weight_decay=0.0), loss_scale=loss_scale,
                          dynamic=True, growth_interval=1000, device_commit=True,
                          state_layout="grouped")
    start = torch.cat([torch.ones(width, device="cuda"), randn(vocab * width) * 0.02])

    def fill(first, count, master, m, v):
        master.copy_(start[first:first + count])
        m.zero_()
        v.zero_()

    st.fill_state(fill)
    st.params.copy_(start)
    teacher_head = randn(vocab, width) * 0.2
    weight = torch.full((rows,), 1.0 / rows, device="cuda")
    losses = []
    for i in range(steps):
        x, res = randn(rows, width).bfloat16(), randn(rows, width).bfloat16()
        h = (x.float() + res.float())
        logits = (h * h.square().mean(1, keepdim=True).rsqrt()) @ teacher_head.t()
        top, ids = logits.topk(slots, 1)
        head.step(st.params, x, res, ids.int(), top.bfloat16(), dev_scaler=st.dev,
                  teacher_lse=logits.logsumexp(1), row_weight=weight)
        st.step_device([head.grads])
        if i % 10 == 0 or i == steps - 1:
            losses.append(float(head.loss.sum()))
            report(f"step {i:4d}  loss {losses[-1]:.4f}")
    st.sync_scaler()
    report(f"{st.t} steps committed, {int(st.scaler.skipped)} skipped, scale {st.loss_scale:g}")
    return losses, st


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("steps", 60), ("rows", 512), ("width", 256), ("vocab", 4096)):
        p.add_argument(f"--{name}", type=int, default=default)
    train(**vars(p.parse_args()))
