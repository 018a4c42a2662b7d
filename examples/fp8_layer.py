#!/usr/bin/env python3
"""A Mixture-of-Experts layer with frozen FP8 experts, forward and backward, from the library's
entry points: what tuning a gate, or anything below the layer, runs.

  forward   route            gate logits -> top-k experts, weights, rows by expert
            quantize_fp8     tokens to FP8, 1 x 128 blocks
            grouped_gemm_fp8 gate and up projection (rows gathered through row_token)
            quantize_fp8     silu(gate) * up to FP8
            grouped_gemm_fp8 down projection
            combine          weighted sum in token order, added to the residual stream
  backward  combine_backward gradients of the rows and of the routing weights
            quantize_fp8, grouped_gemm_fp8   through the down projection (transposed weights)
            quantize_fp8 (swiglu, grad)      through SwiGLU
            grouped_gemm_fp8                 through gate and up
            dispatch_backward                gradients of the tokens
            route_backward                   gradients of the gate logits

  python examples/fp8_layer.py [--tokens 512] [--experts 256] [--topk 8] ...
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


class Layer:
    """Frozen experts in FP8, each matrix with its transposed copy for the way back."""

    def __init__(self, experts, topk, hidden, inter, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.topk = topk
        w13 = torch.randn(experts, 2 * inter, hidden, device="cuda", generator=g) * (2 / hidden ** 0.5)
        w2 = torch.randn(experts, hidden, inter, device="cuda", generator=g) / inter ** 0.5
        self.w13 = moe_fp4.quantize_fp8_weights(w13, transposed=True)
        self.w2 = moe_fp4.quantize_fp8_weights(w2, transposed=True)

    def forward(self, x, logits, residual):
        """x: bfloat16 tokens, logits: the gate's, residual: the float32 stream.  Returns the stream
        after the layer (float32) and what the backward pass reads."""
        r = moe_fp4.route(logits, self.topk)
        xq, xs = moe_fp4.quantize_fp8(x)
        gu = moe_fp4.grouped_gemm_fp8(xq, xs, *self.w13[:2], r.offsets, a_row_index=r.row_token)
        hq, hs = moe_fp4.quantize_fp8(gu, swiglu=True)
        rows = moe_fp4.grouped_gemm_fp8(hq, hs, *self.w2[:2], r.offsets)
        y = moe_fp4.combine(rows, r.token_rows, r.weights, residual=residual, out_dtype=torch.float32)
        return y, (logits, r, gu, rows)

    def backward(self, dy, saved):
        """dy: float32 gradient of the stream.  Returns the gradients of the tokens (bfloat16) and of
        the gate logits; the residual's is dy itself."""
        logits, r, gu, rows = saved
        drows, dweights = moe_fp4.combine_backward(dy, rows, r.token_rows, r.weights, row_token=r.row_token)
        dq, ds = moe_fp4.quantize_fp8(drows)
        dh = moe_fp4.grouped_gemm_fp8(dq, ds, *self.w2[2:], r.offsets)
        dq, ds = moe_fp4.quantize_fp8(gu, swiglu=True, grad=dh)
        dx_rows = moe_fp4.grouped_gemm_fp8(dq, ds, *self.w13[2:], r.offsets)
        dx = moe_fp4.dispatch_backward(dx_rows, r.token_rows)
        return dx, moe_fp4.route_backward(logits, r.ids, dweights)


def milliseconds(fn, calls=20):
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    fn()
    torch.cuda.synchronize()
    a.record()
    for _ in range(calls):
        fn()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / calls


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawTextHelpFormatter)
    for name, value in (("tokens", 512), ("experts", 64), ("topk", 8), ("hidden", 6144), ("inter", 256)):
        ap.add_argument(f"--{name}", type=int, default=value)
    args = ap.parse_args()
    layer = Layer(args.experts, args.topk, args.hidden, args.inter)
    x = torch.randn(args.tokens, args.hidden, device="cuda").bfloat16()
    logits = torch.randn(args.tokens, args.experts, device="cuda")
    residual, dy = torch.randn(2, args.tokens, args.hidden, device="cuda")
    y, saved = layer.forward(x, logits, residual)
    dx, dlogits = layer.backward(dy, saved)
    print(f"stream {tuple(y.shape)}, token gradients {tuple(dx.shape)}, gate gradients {tuple(dlogits.shape)}")
    print(f"forward {milliseconds(lambda: layer.forward(x, logits, residual)):.3f} ms, "
          f"backward {milliseconds(lambda: layer.backward(dy, saved)):.3f} ms")


if __name__ == "__main__":
    main()
