"""The gradients of combine and router at their largest sizes: rows past 2^31 bytes, the most tokens, the
most slots."""
import pytest
import torch

import fp8_ref as ref
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,K,n,dtype", [(50_001, 6, 8192, "bf16"), (2 ** 23, 2, 64, "fp32"), (3, 1024, 4096, "fp32")])
def test_combine_backward(T, K, n, dtype):
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"combine_backward {T} x {n} top-{K} {dtype}")
    M = T * K + 70  # the last rows of no token
    assert M * n * 2 > 2 ** 31 or T < 4
    g = torch.Generator("cuda").manual_seed(T)
    token_rows = torch.randperm(T * K, device="cuda", generator=g).to(torch.int32).view(T, K)
    row_token = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    row_token[token_rows.flatten().long()] = torch.arange(T, dtype=torch.int32, device="cuda").repeat_interleave(K)
    dout = torch.randn(T, n, device="cuda", generator=g).to(ref.DT[dtype])
    rows = torch.empty(M, n, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    weights = torch.rand(T, K, device="cuda", generator=g)
    drows, dw = m.combine_backward(dout, rows, token_rows, weights, row_token)
    assert (drows[-70:] == 0).all()
    for t in {0, T // 2, T - 1}:
        r = token_rows[t].long()
        assert torch.equal(drows[r], (weights[t][:, None] * dout[t].float()).bfloat16())
        p = rows[r].double() * dout[t].double()
        assert ((dw[t].double() - p.sum(1)).abs() <= (n + 1) * ref.U * p.abs().sum(1)).all()
    # Every row somewhere: the first column.
    owner = row_token[:T * K].long()
    slot = torch.empty(T * K, dtype=torch.long, device="cuda")
    slot[token_rows.flatten().long()] = torch.arange(T * K, device="cuda")
    want = (weights.flatten()[slot] * dout[owner, 0].float()).bfloat16()
    assert torch.equal(drows[:T * K, 0], want)


@pytest.mark.parametrize("score,renorm", [("softmax", False), ("sigmoid", True)])
def test_route_backward_of_the_most_tokens(score, renorm):
    from block_scaled_fp4_05_amd import moe_fp4 as m
    T, E, K = 2 ** 24, 130, 2
    say(f"route_backward {T} x {E} {score}")
    assert T * E * 2 > 2 ** 31
    x = torch.empty(T, E, dtype=torch.bfloat16, device="cuda").normal_()
    ids = torch.randint(0, E // 2, (T, K), dtype=torch.int32, device="cuda")
    ids[:, 1] += E // 2
    d = torch.randn(T, K, device="cuda")
    out = m.route_backward(x, ids, d, score, renorm)
    at = torch.tensor([0, 1, 2 ** 23 + 5, T - 16, T - 1], device="cuda")
    ref.check(out[at], *ref.route_backward(x[at].double().cpu(), ids[at].long().cpu(), d[at].double().cpu(), score, renorm))
