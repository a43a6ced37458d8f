"""libzeroshard for AMD Instinct MI355X: the per-rank ZeRO-2 optimizer-shard step.

  zeroshard  -- ctypes binding of the C ABI (include/zeroshard.h); importing it
                loads libzeroshard.so and raises if it is not built.
  head       -- a low-precision student's output end over the operators of the
                same library, between the parameters and the gradients.
  block      -- its last block in front of the output end, likewise.
  synth      -- seeded synthetic inputs (host and device twins) and the
                workload definitions used by the tests and the benchmark.
  build      -- compiles the in-tree shared libraries.
"""
__all__ = ["zeroshard", "synth", "build"]
