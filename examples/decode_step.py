#!/usr/bin/env python3
"""One decode step of a Mixture-of-Experts block for a few tokens, from the library's
entry points, eager and replayed from a HIP graph:

  gate    linear   hidden -> expert logits (FP32)
  router  route    top-k experts, weights
  layer   moe_ffn  gate+up, SwiGLU, down, weighted sum, added to the residual stream
  head    linear   vocabulary logits (FP32), then the largest

Weights are random NVFP4 (quantised on the GPU).  The sizes default to the decode shard
of bench.py: 256 experts, hidden 6144, intermediate 256, top-8.

  python examples/decode_step.py [--tokens 1] [--experts 256] [--topk 8] ...
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from block_scaled_fp4_05_amd import moe_fp4  # noqa: E402


def random_weights(rows: int, k: int, generator, gain: float = 1.0):
    """A random [rows][k] matrix as NVFP4: codes, block scales, tensor scale."""
    w = torch.randn(rows, k, device="cuda", generator=generator) * (gain / k ** 0.5)
    return moe_fp4.quantize(w)


class Block:
    """The weights of one block: gate, experts and vocabulary head."""

    def __init__(self, experts, topk, hidden, inter, vocab, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.topk = topk
        self.gate = random_weights(experts, hidden, g, 2.0)
        up = [random_weights(2 * inter, hidden, g, 2.0) for _ in range(experts)]
        down = [random_weights(hidden, inter, g) for _ in range(experts)]
        self.w13 = [torch.stack([u[0] for u in up]), torch.stack([u[1] for u in up]),
                    torch.cat([u[2] for u in up])]
        self.w2 = [torch.stack([d[0] for d in down]), torch.stack([d[1] for d in down]),
                   torch.cat([d[2] for d in down])]
        self.head = random_weights(vocab, hidden, g)

    def step(self, x, residual):
        """x: the block's normalised input, residual: the stream it adds onto.  Returns
        (next tokens, stream after the block, routing)."""
        r = moe_fp4.route(moe_fp4.linear(x, *self.gate, out_dtype=torch.float32), self.topk)
        y = moe_fp4.moe_ffn(x, r.ids, r.weights, *self.w13, *self.w2, residual=residual)
        logits = moe_fp4.linear(y, *self.head, out_dtype=torch.float32)
        return logits.argmax(1), y, r


def microseconds(fn, calls=50):
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    fn()
    torch.cuda.synchronize()
    a.record()
    for _ in range(calls):
        fn()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / calls * 1e3


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawTextHelpFormatter)
    for name, value in (("tokens", 1), ("experts", 256), ("topk", 8), ("hidden", 6144), ("inter", 256),
                        ("vocab", 32768)):
        ap.add_argument(f"--{name}", type=int, default=value)
    args = ap.parse_args()
    block = Block(args.experts, args.topk, args.hidden, args.inter, args.vocab)
    x = torch.randn(args.tokens, args.hidden, device="cuda").bfloat16()
    residual = torch.randn_like(x)
    tokens, _, r = block.step(x, residual)
    print(f"tokens {tokens.tolist()}, experts {r.ids.tolist()}")
    print(f"eager {microseconds(lambda: block.step(x, residual)):.1f} us a step")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step(x, residual)
    print(f"graph {microseconds(graph.replay):.1f} us a step")


if __name__ == "__main__":
    main()
