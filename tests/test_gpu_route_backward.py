"""The gradient of the routing weights against its formulas in 64 bits, those against central
differences, and the cases at the edges of the scores."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

KINDS = [(s, r) for s in ("softmax", "sigmoid") for r in (True, False)]


def inputs(seed, T, E, K, dtype, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, E, generator=g) * spread).to(ref.DT[dtype])
    ids = torch.topk(x.float(), K, dim=1).indices
    return x, ids, torch.randn(T, K, generator=g)


@pytest.mark.parametrize("score,renorm", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 256, 8), (3, 7, 2), (5, 64, 6), (70, 100, 1), (9, 257, 10),
                                   (2, 1024, 32), (8200, 16, 3)])
def test_against_the_formulas(T, E, K, dtype, score, renorm):
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"route_backward {T} x {E} top-{K} {dtype} {score} renorm={renorm}")
    x, ids, d = inputs(T + E, T, E, K, dtype)
    wide = torch.zeros(T, E + 3, dtype=x.dtype).cuda()
    wide[:, :E] = x.cuda()
    out = torch.full((T, E + 2), 5.0, dtype=x.dtype, device="cuda")
    m.route_backward(wide[:, :E], ids.int().cuda(), d.cuda(), score, renorm, out=out[:, :E])
    ref.check(out[:, :E], *ref.route_backward(x.double(), ids, d.double(), score, renorm))
    assert (out[:, E:] == 5).all()


@pytest.mark.parametrize("score,renorm", KINDS)
def test_the_formulas_are_the_gradients(score, renorm):
    x, ids, d = inputs(1, 4, 9, 3, "fp32")
    x, d, h = x.double(), d.double(), 1e-5
    want = torch.zeros_like(x)
    for j in range(9):
        e = torch.zeros_like(x)
        e[:, j] = h
        up, down = (ref.route_weights(x + s * e, ids, score, renorm) for s in (1, -1))
        want[:, j] = ((up - down) * d).sum(1) / (2 * h)
    assert (ref.route_backward(x, ids, d, score, renorm)[0] - want).abs().max() < 1e-8


@pytest.mark.parametrize("score,renorm", KINDS)
def test_with_the_router_in_front(score, renorm):
    """Its own ids (with a selection bias and groups for the sigmoid), and the weights it gave."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    T, E, K = 40, 64, 4
    x, _, d = inputs(2, T, E, K, "fp32")
    more = dict(bias=torch.randn(E, device="cuda") * 0.1, num_groups=8, topk_groups=3) if score == "sigmoid" else {}
    r = m.route(x.cuda(), K, score, renormalize=renorm, **more)
    out = m.route_backward(x.cuda(), r.ids, d.cuda(), score, renorm)
    ids = r.ids.cpu().long()
    assert torch.allclose(ref.route_weights(x.double(), ids, score, renorm), r.weights.cpu().double(), rtol=1e-5)
    ref.check(out, *ref.route_backward(x.double(), ids, d.double(), score, renorm))


@pytest.mark.parametrize("score,renorm", KINDS)
def test_far_logits(score, renorm):
    """Scores down to e^-87 keep their proportions; -inf outside the choice is a score of 0."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    T, E, K = 6, 40, 5
    x, ids, d = inputs(3, T, E, K, "fp32", 1.0)
    x[0] += 80
    x[1] -= 80
    x[2] *= 20
    x[3, ids[3, 1:]] -= 60
    x[4] -= 300 if renorm else 60
    closed = torch.ones(T, E, dtype=torch.bool).scatter_(1, ids, False)
    x[5][closed[5]] = -np.inf
    out = m.route_backward(x.cuda(), ids.int().cuda(), d.cuda(), score, renorm)
    y, b = ref.route_backward(x.double(), ids, d.double(), score, renorm)
    b = torch.where(torch.isfinite(x), b, torch.zeros_like(b))
    ref.check(out, y, b)


def test_slots_without_an_expert_and_named_twice():
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    x, ids, d = inputs(4, 5, 12, 4, "fp32")
    on = x.cuda()
    for score, renorm in KINDS:
        base = m.route_backward(on, ids[:, :3].int().cuda().contiguous(), d[:, :3].cuda().contiguous(), score, renorm)
        for bad in (-1, 12, 2 ** 31 - 1):
            ids4 = ids.clone()
            ids4[:, 3] = bad
            assert torch.equal(base, m.route_backward(on, ids4.int().cuda(), d.cuda(), score, renorm))
        none = m.route_backward(on, torch.full((5, 4), -1, dtype=torch.int32, device="cuda"), d.cuda(), score, renorm)
        assert (none == 0).all()
        twice = ids.clone()
        twice[:, 2] = twice[:, 0]
        out = m.route_backward(on, twice.int().cuda(), d.cuda(), score, renorm)
        ref.check(out, *ref.route_backward(x.double(), twice, d.double(), score, renorm))


def test_what_the_formula_has_no_value_for():
    """All chosen logits -inf, a NaN or +inf among them: NaN in that token's row, others untouched."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    x, ids, d = inputs(5, 4, 10, 3, "fp32")
    x[1, ids[1]] = -np.inf
    x[2, ids[2, 1]] = np.nan
    out = m.route_backward(x.cuda(), ids.int().cuda(), d.cuda()).cpu()
    assert out[1, ids[1]].isnan().all() and out[2, ids[2]].isnan().all()
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[3]).all()
    assert m.route_backward(x[:0].cuda(), ids[:0].int().cuda(), d[:0].cuda()).shape == (0, 10)
