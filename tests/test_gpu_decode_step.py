"""The example decode step: gate, router, layer and head together, each against its
64-bit reference on the step's own inputs, and replayed from a graph."""
import os
import sys

import pytest
import torch

import few_token_ref as ref
from conftest import ROOT
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 6])
def test_decode_step(tokens):
    require_gpu()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    from decode_step import Block
    E, K, H, I, V = 24, 3, 272, 80, 200
    block = Block(E, K, H, I, V, seed=tokens)
    x = torch.randn(tokens, H, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    residual = torch.roll(x, 1, 1)
    token, y, r = block.step(x, residual)

    def dense(q, sf):
        return ref.values(q.cpu().numpy(), sf.cpu().numpy())

    gate, _ = ref.linear(x.cpu().double(), dense(*block.gate[:2]), float(block.gate[2]))
    w = torch.softmax(gate.gather(1, r.ids.cpu().long()), 1)
    # Logits within (H + 2) u of their absolute sums (below 8 here): e^ of that, and the sums.
    assert ((r.weights.cpu().double() - w).abs() <= w * (4 * (H + 2) * 8 + 64) * ref.U).all()
    assert torch.equal(gate.argmax(1), r.ids[:, 0].cpu().long())
    w13 = [dense(block.w13[0][e], block.w13[1][e]) for e in range(E)]
    w2 = [dense(block.w2[0][e], block.w2[1][e]) for e in range(E)]
    ref.check(y, *ref.ffn(x.cpu().double(), r.ids.cpu(), r.weights.cpu(), w13, block.w13[2].cpu().double(),
                          w2, block.w2[2].cpu().double(), residual.cpu().double()))
    head, _ = ref.linear(y.cpu().double(), dense(*block.head[:2]), float(block.head[2]))
    assert torch.equal(head.argmax(1), token.cpu())

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block.step(x, residual)
    for _ in range(3):
        x.copy_(torch.roll(x, 1, 1))
        graph.replay()
        torch.cuda.synchronize()
        want = block.step(x, residual)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
