"""moe_fp4.route against sorting in 64 bits: choices and rows exactly, weights within their
FP32 bound.  softmax: the exponential's argument is off by u |x - max|, the exponential by
a few steps, the sum of n terms by n u; sigmoid: a few steps after binary64."""
import numpy as np
import pytest
import torch

import few_token_ref as ref
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _check(logits, topk, score="softmax", bias=None, renorm=True, groups=1, topk_groups=None, **kw):
    from block_scaled_fp4_05_amd import moe_fp4
    r = moe_fp4.route(kw.pop("given", logits.cuda()), topk, score=score,
                      bias=None if bias is None else bias.cuda(), renormalize=renorm, num_groups=groups,
                      topk_groups=topk_groups, **kw)
    ids, w, off, row, slot = ref.route(logits, topk, score, bias, renorm, groups, topk_groups or groups)
    for name, got, want in (("ids", r.ids, ids), ("offsets", r.offsets, off), ("row_token", r.row_token, row),
                            ("token_rows", r.token_rows, slot)):
        assert got.dtype == torch.int32
        assert np.array_equal(got.cpu().numpy(), want), name
    g, w = r.weights.cpu().double(), torch.from_numpy(np.asarray(w, np.float64))
    x = logits.double()
    span = (x.amax(1) - x.amin(1)).clamp(max=200.0)[:, None] if x.numel() else 0.0
    rel = (x.shape[1] + 16 + 2 * torch.as_tensor(span).nan_to_num(200.0)) * ref.U
    ok = (g - w).abs() <= rel * w.abs() + 2.0 ** -140
    assert (ok | (g.isnan() & w.isnan())).all(), float(((g - w).abs() / w.abs()).max())
    return r


def _logits(T, E, dtype="fp32", seed=0):
    rng = np.random.default_rng(seed + 100 * T + E)
    return torch.from_numpy(rng.standard_normal((T, E)) * 2).to(ref.DT[dtype])


@pytest.mark.parametrize("T", [0, 1, 2, 16, 31, 32, 33, 63, 64, 65, 100, 513, 3001])
@pytest.mark.parametrize("E,topk", [(1, 1), (2, 2), (8, 3), (60, 4), (64, 8), (65, 8), (256, 8), (257, 9),
                                    (384, 1), (1000, 32), (1024, 6)])
def test_route_softmax(T, E, topk):
    say(f"route softmax T{T} E{E} K{topk}")
    _check(_logits(T, E), topk, renorm=T % 2 == 0)


@pytest.mark.parametrize("T", [1, 32, 70, 600])
@pytest.mark.parametrize("E,topk,groups,topk_groups", [
    (64, 6, 8, 3), (256, 8, 8, 4), (160, 6, 8, 3), (60, 4, 6, 2), (48, 5, 3, 1), (384, 8, 4, 4),
    (63, 7, 9, 2), (64, 2, 64, 5), (40, 4, 20, 2), (1024, 16, 16, 2)])
@pytest.mark.parametrize("score,bias", [("softmax", False), ("sigmoid", False), ("sigmoid", True)])
def test_route_groups(T, E, topk, groups, topk_groups, score, bias):
    say(f"route T{T} E{E} K{topk} G{groups}/{topk_groups} {score} {bias}")
    b = torch.from_numpy(np.random.default_rng(E).standard_normal(E).astype(np.float32) * 0.1) if bias else None
    _check(_logits(T, E), topk, score, b, True, groups, topk_groups)
    _check(_logits(T, E, seed=9), topk, score, b, False)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_route_sixteen_bit_logits_with_ties(dtype):
    x = (_logits(200, 128) * 2).round().to(ref.DT[dtype])  # a few distinct values
    for score in ("softmax", "sigmoid"):
        _check(x, 7, score)
        _check(x, 4, score, None, False, 8, 2)


def test_route_equal_and_signed_zero_logits():
    _check(torch.zeros(40, 96), 5)
    x = torch.zeros(3, 70)
    x[:, 1::2] = -0.0  # equal to +0: index order
    r = _check(x, 6)
    assert r.ids[0].tolist() == [0, 1, 2, 3, 4, 5]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_values_that_are_not_finite(score):
    x = _logits(6, 20)
    x[0, 3:] = float("-inf")            # three experts left, four asked for
    x[1, 4] = float("nan")              # ranked last, below -inf
    x[1, :4] = float("-inf")
    x[2] = float("-inf")                # nothing left: index order
    x[3, 7] = float("inf")
    x[4] = float("nan")
    from block_scaled_fp4_05_amd import moe_fp4
    for T in (6, 60):
        big = x.repeat(T // 6, 1)
        r = moe_fp4.route(big.cuda(), 4, score=score)
        ids = ref.route(big, 4, score, None, True, 1, 1)[0]
        assert np.array_equal(r.ids.cpu().numpy(), ids)
        assert sorted(r.token_rows.flatten().tolist()) == list(range(4 * T))
        assert torch.isfinite(r.weights[5]).all()
    if score == "softmax":
        assert r.weights[0, 3] == 0 and abs(float(r.weights[0, :3].sum()) - 1) < 1e-6


# From 4096 tokens on, 16 lanes rank a token where they can hold its experts.
@pytest.mark.parametrize("T", [4096, 4099])
@pytest.mark.parametrize("E,topk", [(3, 2), (16, 1), (24, 5), (64, 8), (100, 6), (128, 16), (256, 8), (257, 8)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_route_sixteen_lanes_a_token(T, E, topk, dtype):
    """Softmax and sigmoid, with many equal logits (a few distinct values) and few."""
    say(f"route 16 lanes T{T} E{E} K{topk} {dtype}")
    x = _logits(T, E, dtype)
    _check(x, topk, renorm=False)
    _check((x * 2).round(), topk, renorm=T % 2 == 0)
    _check((x * 2).round(), topk, "sigmoid", None, T % 2 == 1)


@pytest.mark.parametrize("T", [4096, 4099])
@pytest.mark.parametrize("E,topk,groups,topk_groups", [
    (256, 8, 8, 4), (160, 6, 8, 3), (48, 5, 3, 1), (64, 4, 16, 5), (30, 3, 2, 1), (128, 8, 4, 2), (256, 8, 16, 4)])
@pytest.mark.parametrize("score,bias,dtype", [("softmax", False, "fp32"), ("softmax", False, "bf16"),
                                              ("sigmoid", False, "fp32"), ("sigmoid", True, "bf16"),
                                              ("sigmoid", True, "fp32")])
def test_route_groups_with_sixteen_lanes_a_token(T, E, topk, groups, topk_groups, score, bias, dtype):
    say(f"route 16 lanes T{T} E{E} K{topk} G{groups}/{topk_groups} {score} {bias} {dtype}")
    b = torch.from_numpy(np.random.default_rng(E).standard_normal(E).astype(np.float32) * 0.1) if bias else None
    x = _logits(T, E, dtype)
    if dtype == "bf16":
        x = (x * 2).round()
    _check(x, topk, score, b, T % 2 == 0, groups, topk_groups)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_route_values_that_are_not_finite_with_sixteen_lanes_a_token(score, dtype):
    x = _logits(4098, 20, dtype)
    x[0::6, 3:] = float("-inf")
    x[1::6, 4] = float("nan")
    x[1::6, :4] = float("-inf")
    x[2::6] = float("-inf")
    x[3::6, 7] = float("inf")
    x[4::6] = float("nan")
    from block_scaled_fp4_05_amd import moe_fp4
    r = moe_fp4.route(x.cuda(), 4, score=score)
    assert np.array_equal(r.ids.cpu().numpy(), ref.route(x, 4, score, None, True, 1, 1)[0])
    assert sorted(r.token_rows.flatten().tolist()) == list(range(4 * 4098))
    assert torch.isfinite(r.weights[5::6]).all()


def test_route_sigmoid_scores_closer_than_fp32():
    """Scores that differ by less than an FP32 step at 1 keep their order."""
    x = torch.full((2, 64), -3.0)
    x[0, 10], x[0, 50] = 17.0, 17.5      # 1 - 4.1e-8 and 1 - 2.5e-8
    x[1, 50], x[1, 10] = 17.0, 17.5
    r = _check(x, 2, "sigmoid")
    assert r.ids.tolist() == [[50, 10], [10, 50]]


@pytest.mark.parametrize("T", [1, 5, 70, 4100])
def test_route_sigmoid_weights_below_fp32(T):
    """Scores that FP32 holds in a few bits or not at all (below 2^-126) still have their
    proportions as weights."""
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.uniform(-300.0, -85.0, (T, 20)).astype(np.float32))
    x[0, :] = torch.linspace(-106.0, -99.0, 20)
    _check(x, 4, "sigmoid")
    _check(x, 4, "sigmoid", torch.linspace(0, 1, 20), True, 4, 2)
    _check(x, 4, "sigmoid", None, False)


def test_route_bias_may_close_experts():
    b = torch.zeros(32)
    b[5:] = float("-inf")
    r = _check(_logits(50, 32), 5, "sigmoid", b)
    assert (r.ids < 5).all()


@pytest.mark.parametrize("T,E,topk", [(20000, 24, 4), (70000, 16, 2), (140000, 9, 3)])
def test_route_long_batches(T, E, topk):
    """Blocks of 128 tokens and of 512, and more than 256 blocks."""
    say(f"route T{T}")
    _check(_logits(T, E), topk)


def test_route_pitch_outputs_and_workspace():
    from block_scaled_fp4_05_amd import moe_fp4
    T, E, K = 77, 48, 5
    x = _logits(T, E)
    wide = torch.full((T, E + 5), float("nan"), device="cuda")
    wide[:, :E] = x.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    out = moe_fp4.Routing(torch.full((T, K), -7, **i32), torch.full((T, K), -7.0, device="cuda"),
                          torch.full((E + 1,), -7, **i32), torch.full((T * K,), -7, **i32),
                          torch.full((T, K), -7, **i32))
    ws = torch.full((moe_fp4.route_workspace_size(T, E) + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    r = _check(x, K, given=wide[:, :E], out=out, workspace=ws)
    assert r.ids.data_ptr() == out.ids.data_ptr() and (ws[-64:] == 0xFF).all()


@pytest.mark.parametrize("T", [3, 200])
def test_route_repeats_its_bits_on_other_streams_and_in_graphs(T):
    from block_scaled_fp4_05_amd import moe_fp4
    x = _logits(T, 100).cuda()
    want = moe_fp4.route(x, 6)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = moe_fp4.route(x, 6, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = moe_fp4.route(x, 6)
    for i in range(3):
        x.copy_(torch.roll(x, 3, 1))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, moe_fp4.route(x, 6))), i


def test_route_feeds_the_grouped_gemm_and_the_combine():
    """row_token gathers and token_rows scatters: with rows r holding their token's vector,
    the combine returns every token's vector times the sum of its weights."""
    from block_scaled_fp4_05_amd import moe_fp4
    T, E, K, n = 90, 40, 4, 32
    r = moe_fp4.route(_logits(T, E).cuda(), K)
    vec = torch.randn(T, n, device="cuda").bfloat16()
    out = moe_fp4.combine(vec[r.row_token.long()], r.token_rows, r.weights, out_dtype=torch.float32)
    # K products and sums in FP32 of weights that sum to 1.
    assert ((out - vec.float()).abs() <= vec.float().abs() * (2 * K + 40) * ref.U * 2).all()
    counts = (r.offsets[1:] - r.offsets[:-1]).cpu()
    assert torch.equal(counts, torch.bincount(r.ids.flatten().cpu().long(), minlength=E).int())
