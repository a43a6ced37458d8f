"""Tune a small student's last block and head on pairs of answers, one GPU: the
low-precision forward and backward of `block.BlockStudent` with dropout, a
frozen reference's log-probabilities, and the mixed-precision shard step of
`shard.ShardState`, loss scale and commit-or-skip on the device.

    python examples/tune_student.py [--steps 40] [--pairs 8] [--length 32] [--width 256]

Prints the mean loss. Synthetic data: random hidden states and answers.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from sharded_mixed_precision_zs_amd import shard, zeroshard as zs  # noqa: E402
from sharded_mixed_precision_zs_amd.block import BlockStudent, MlpBlock  # noqa: E402
from sharded_mixed_precision_zs_amd.head import PreferenceHead  # noqa: E402


def train(steps=40, pairs=8, length=32, width=256, hidden=512, vocab=1000, lr=1e-3, dropout=0.1,
          loss_scale=4096.0, report=print):
    """Returns the mean loss of each reported step, the student and the shard state."""
    g = torch.Generator(device="cuda").manual_seed(0)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")

    rows = 2 * pairs * length
    student = BlockStudent(MlpBlock(rows, width, hidden, dropout=dropout, seed=1),
                           PreferenceHead(rows, width, vocab, pairs, beta=0.1))
    ones, zeros = torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")
    start = torch.cat([ones, 0.05 * randn(hidden * width), torch.zeros(hidden, device="cuda"),
                       0.05 * randn(width * hidden), zeros, ones, 0.5 * ones,
                       ones, 0.05 * randn(vocab * width)])
    st = shard.ShardState(student.phi, 1, 0, 0, student.phi, zs.ZS_BF16, zs.ZS_BF16,
                          shard.AdamW(lr=lr, weight_decay=0.0), loss_scale=loss_scale,
                          dynamic=True, growth_interval=1000, device_commit=True,
                          state_layout="grouped")

    def fill(first, count, master, m, v):
        master.copy_(start[first:first + count])
        m.zero_()
        v.zero_()

    st.fill_state(fill)
    st.params.copy_(start)
    x, res = randn(rows, width).bfloat16(), randn(rows, width).bfloat16()
    ids = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    ids.view(2 * pairs, length)[:, :length // 4] = -1        # the prompts
    starts = torch.arange(0, rows + 1, length, device="cuda", dtype=torch.int32)
    weight = torch.full((pairs,), 1.0 / pairs, device="cuda")
    # the reference: the student before its first step, without dropout
    ref = student.logprobs(st.params, x, res, ids).view(2 * pairs, length).sum(1)
    losses = []
    for i in range(steps):
        student.step(st.params, x, res, offset=i, ids=ids, starts=starts, ref_logp=ref,
                     pair_weight=weight, dev_scaler=st.dev)
        st.step_device([student.grads])
        if i % 10 == 0 or i == steps - 1:
            losses.append(float(student.head.loss.sum()))
            report(f"step {i:4d}  loss {losses[-1]:.4f}")
    st.sync_scaler()
    report(f"{st.t} steps committed, {int(st.scaler.skipped)} skipped, scale {st.loss_scale:g}")
    return losses, student, st


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("steps", 40), ("pairs", 8), ("length", 32), ("width", 256)):
        p.add_argument(f"--{name}", type=int, default=default)
    train(**vars(p.parse_args()))
