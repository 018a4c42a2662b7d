"""FP8 block quantisers: plain rows and weights bit for bit against IEEE arithmetic on the CPU,
SwiGLU and its gradient within their FP32 roundings of the 64-bit formulas."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


def _rows(seed, rows, k, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, k, generator=g) * torch.exp2(torch.randint(-12, 12, (rows, 1), generator=g).float())
    return x.to(ref.DT[dtype])


def _same(q, s, want_q, want_s):
    assert np.array_equal(s.cpu().numpy().view(np.uint32), want_s.view(np.uint32))
    got = q.cpu().view(torch.uint8).numpy()
    nan = (want_q & 0x7F) == 0x7F
    assert np.array_equal(got[~nan], want_q[~nan]) and ((got[nan] & 0x7F) == 0x7F).all()


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,k", [(1, 16), (1, 6144), (3, 128), (7, 144), (33, 272), (129, 1552)])
def test_rows_bit_for_bit(rows, k, dtype, pow2):
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"quantize_fp8 {rows} x {k} {dtype} pow2={pow2}")
    x = _rows(rows * 7 + k, rows, k, dtype)
    q, s = m.quantize_fp8(x.cuda(), power_of_two=pow2)
    assert q.dtype == torch.float8_e4m3fn and q.shape == (rows, k) and s.shape == (rows, ref.blocks(k))
    _same(q, s, *ref.quantize(x.float().numpy(), 1, pow2))


@pytest.mark.parametrize("pow2", [False, True])
def test_special_values(pow2):
    """Zeros and their signs, subnormal and huge blocks, NaN, infinities, boundaries of the codes."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    x = torch.zeros(40, 128)
    x[1] = -0.0
    g = torch.Generator().manual_seed(0)
    for i, e in enumerate((-149, -140, -130, -126, -120, -100, -92, -91, -90, -83, -82, -81, -60, 60, 100, 119, 126)):
        x[2 + i] = torch.randn(128, generator=g).clamp(-1.9, 1.9) * 2.0 ** e
    x[20, 5], x[20, 6], x[20, 7] = 3.0, float("nan"), -1.0
    x[21, 3], x[21, 4] = float("inf"), 2.0
    x[22] = float("nan")
    x[23, 0], x[23, 1] = float("-inf"), float("nan")
    x[24, 9] = 1e-45
    # Ties and neighbours of every code boundary under a scale of one.
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = (codes[1:] + codes[:-1]) / 2
    for i, v in enumerate((codes[:126], mid, torch.nextafter(mid, torch.tensor(0.0)), torch.nextafter(mid, torch.tensor(1e9)))):
        x[25 + i, :126] = v
        x[25 + i, 127] = 448.0
        x[30 + i] = -x[25 + i]
    q, s = m.quantize_fp8(x.cuda(), power_of_two=pow2)
    _same(q, s, *ref.quantize(x.numpy(), 1, pow2))
    # An infinity leaves nothing finite; a NaN leaves the others alone.
    v = ref.values(q, s, 1)
    assert not np.isfinite(v[21]).any() and np.isfinite(v[20]).sum() == 127


def test_pitches_given_outputs_and_no_rows():
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    wide = _rows(1, 9, 400, "bf16").cuda()
    x = wide[1::2, 16:288]
    q = torch.full((6, 272), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((6, 3), -1.0, device="cuda")
    m.quantize_fp8(x, q=q[:4].view(ref.FP8), sf=s[:4])
    _same(q[:4], s[:4], *ref.quantize(x.float().cpu().numpy()))
    assert (q[4:] == 0x55).all() and (s[4:] == -1).all()
    q, s = m.quantize_fp8(x[:0])
    assert q.shape == (0, 272) and s.shape == (0, 3)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,k", [(1, 16), (301, 16), (2, 256), (5, 144), (66, 1424), (9, 2064), (3, 8192), (2, 8208)])
def test_swiglu_and_its_gradient(rows, k, dtype, pow2):
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"quantize_fp8 swiglu {rows} x {k} {dtype} pow2={pow2}")
    g = torch.Generator().manual_seed(rows + k)
    wide = (torch.randn(rows, 2 * k + 16, generator=g) * 2.5).to(ref.DT[dtype])
    wide[0, :8] = torch.tensor([0.0, -0.0, 60.0, -60.0, 88.0, -88.0, 100.0, -100.0])
    x, d = wide[:, :2 * k], (torch.randn(rows, k, generator=g) * 0.01).to(ref.DT[dtype])
    on = wide.cuda()[:, :2 * k]
    x64, d64 = x.double().numpy(), d.double().numpy()
    q, s = m.quantize_fp8(on, swiglu=True, power_of_two=pow2)
    assert q.shape == (rows, k)
    ref.check_quantized(q, s, *ref.swiglu(x64), pow2, "swiglu")
    q, s = m.quantize_fp8(on, swiglu=True, grad=d.cuda(), power_of_two=pow2)
    assert q.shape == (rows, 2 * k) and s.shape == (rows, ref.blocks(2 * k))
    ref.check_quantized(q, s, *ref.swiglu_grad(x64, d64), pow2, "gradient")


def test_the_gradient_formula_is_that_of_swiglu():
    """Central differences of silu(g) u in binary64 against the formula the kernel is held to."""
    rng = np.random.default_rng(0)
    x, d, h = rng.normal(size=(3, 64)) * 2, rng.normal(size=(3, 32)), 1e-5
    want = np.zeros_like(x)
    for j in range(64):
        e = np.zeros_like(x)
        e[:, j] = h
        want[:, j] = ((ref.swiglu(x + e)[0] - ref.swiglu(x - e)[0]) * d).sum(1) / (2 * h)
    assert np.abs(ref.swiglu_grad(x, d)[0] - want).max() < 1e-8  # h^2 and 2^-53 / h


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("E,n,k", [(1, 16, 16), (2, 128, 128), (3, 144, 272), (1, 400, 1040)])
def test_weights_and_their_transpose_bit_for_bit(E, n, k, dtype, pow2):
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"quantize_fp8_weights {E} x {n} x {k} {dtype} pow2={pow2}")
    w = _rows(n + k, E * n, k, dtype).view(E, n, k)
    q, s, qt, st = m.quantize_fp8_weights(w.cuda(), transposed=True, power_of_two=pow2)
    wq, ws = ref.quantize(w.float().numpy(), 128, pow2)
    _same(q, s, wq, ws)
    _same(qt, st, np.ascontiguousarray(wq.transpose(0, 2, 1)), np.ascontiguousarray(ws.transpose(0, 2, 1)))
    only = m.quantize_fp8_weights(w[0].cuda(), power_of_two=pow2)
    assert len(only) == 2 and only[0].shape == (n, k)
    _same(*only, wq[0], ws[0])


def test_weights_with_an_odd_number_of_rows():
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    w = _rows(3, 131, 144, "bf16")
    _same(*m.quantize_fp8_weights(w.cuda()), *ref.quantize(w.float().numpy(), 128))
    with pytest.raises(m.MoeFp4Error, match="sizes"):
        m.quantize_fp8_weights(w.cuda(), transposed=True)


@pytest.mark.parametrize("k", [128, 1424, 8320])
def test_a_run_of_nan_gradients_leaves_its_blocks_scales_alone(k):
    """Eight NaN that one thread holds, in blocks with numbers, in both halves."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"quantize_fp8 swiglu gradient with NaN, k={k}")
    g = torch.Generator().manual_seed(k)
    x, d = torch.randn(3, 2 * k, generator=g), torch.randn(3, k, generator=g)
    d[1, 16:24] = float("nan")
    q, s = m.quantize_fp8(x.cuda(), swiglu=True, grad=d.cuda())
    hole = torch.zeros(3, 2 * k, dtype=torch.bool)
    hole[1, 16:24] = hole[1, k + 16:k + 24] = True
    assert torch.equal(q.cpu().float().isnan(), hole)
    # The scales are those of zeros in the NaN's place.
    q0, s0 = m.quantize_fp8(x.cuda(), swiglu=True, grad=torch.nan_to_num(d, nan=0.0).cuda())
    assert torch.equal(s, s0)
    assert torch.equal(q.cpu().view(torch.uint8)[~hole], q0.cpu().view(torch.uint8)[~hole])
