"""moe_fp4.linear against a plain 64-bit product: sizes, types, epilogues, row pitches,
values that must stay where they are, streams and graphs.  Bounds: few_token_ref."""
import numpy as np
import pytest
import torch

import few_token_ref as ref
from gpu_util import dev, require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _case(m, n, k, dtype, seed=0, gain=1.0):
    rng = np.random.default_rng(seed + 7919 * m + 31 * n + k)
    q, sf = ref.weights(rng, (n, k))
    x = torch.from_numpy(rng.standard_normal((m, k)) * gain).to(ref.DT[dtype])
    return rng, q, sf, x, float(np.float32(rng.uniform(0.2, 2.0) / np.sqrt(k)))


def _run(x, q, sf, scale, **kw):
    from block_scaled_fp4_05_amd import moe_fp4
    return moe_fp4.linear(x, dev(q), dev(sf), torch.tensor([scale], device="cuda"), **kw)


SIZES = [(1, 1, 64), (1, 16, 64), (2, 17, 80), (3, 15, 96), (4, 33, 112), (5, 31, 240), (7, 1001, 784),
         (8, 48, 256), (16, 40, 272), (16, 130, 1040), (17, 40, 288), (31, 64, 1008), (32, 20, 528),
         (33, 50, 320), (70, 24, 64), (1, 8200, 2064), (3, 8192, 512), (20, 8208, 144), (1, 96, 18448),
         (9, 16, 20000)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_linear_sizes(m, n, k, dtype):
    say(f"linear {m}x{n}x{k} {dtype}")
    rng, q, sf, x, scale = _case(m, n, k, dtype)
    w = ref.values(q, sf)
    out = _run(x.cuda(), q, sf, scale)
    assert out.dtype == ref.DT[dtype] and out.shape == (m, n)
    ref.check(out, *ref.linear(x.double(), w, scale), what="same type")
    res = torch.from_numpy(rng.standard_normal((m, n))).to(ref.DT[dtype])
    out = _run(x.cuda(), q, sf, scale, residual=res.cuda(), out_dtype=torch.float32)
    ref.check(out, *ref.linear(x.double(), w, scale, residual=res.double()), what="residual, FP32")


@pytest.mark.parametrize("m,n,k", [(1, 2, 64), (2, 30, 128), (7, 74, 784), (16, 256, 256), (19, 48, 2080),
                                   (1, 8400, 128), (4, 8192, 272), (40, 34, 96)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32"),
                                       ("fp16", "bf16"), ("bf16", "fp16")])
def test_linear_swiglu(m, n, k, dtype, out):
    say(f"linear swiglu {m}x{n}x{k} {dtype} {out}")
    _, q, sf, x, scale = _case(m, n, k, dtype)
    got = _run(x.cuda(), q, sf, 3 * scale, swiglu=True, out_dtype=ref.DT[out])
    assert got.shape == (m, n // 2) and got.dtype == ref.DT[out]
    ref.check(got, *ref.linear(x.double(), ref.values(q, sf), float(np.float32(3 * scale)), True))


@pytest.mark.parametrize("k", range(64, 592, 16))
def test_linear_many_rows_ending_anywhere_in_a_step(k):
    """Rows enough for two tiles a wavefront, whose codes are turned in LDS: every place
    in a step where a row can end."""
    for m, dtype in ((2, "bf16"), (4, "fp16"), (7, "bf16")):
        say(f"linear tail {m}x8200x{k} {dtype}")
        _, q, sf, x, scale = _case(m, 8200, k, dtype)
        got = _run(x.cuda(), q, sf, scale, out_dtype=torch.float32)
        ref.check(got, *ref.linear(x.double(), ref.values(q, sf), scale))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_linear_every_code_and_scale_is_exact(dtype):
    """One-hot activations read single weights: the result is the rounded weight itself,
    for every code under every finite block scale."""
    codes = np.arange(16, dtype=np.uint8)
    scales = np.array([s for s in range(256) if s & 0x7F != 0x7F], np.uint8)
    n, k = len(scales), 64
    q = np.tile(codes[0::2] | codes[1::2] << 4, (n, k // 16))
    sf = np.tile(scales[:, None], (1, k // 16))
    x = torch.eye(16, k, dtype=ref.DT[dtype])
    got = _run(x.cuda(), q, sf, 1.0, out_dtype=torch.float32).cpu().double()
    assert torch.equal(got, ref.values(q, sf)[:, :16].t())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_linear_swiglu_far_from_zero(dtype):
    """One-hot activations and a scale that is a power of two make gate and up exact, up to
    +-45: the epilogue's exponential (2 u), sum, quotient and product (u each) are then within
    6 u of silu(g) * u wherever g lies (below -87 FP32 runs out; not reached)."""
    n, k, m = 512, 64, 16
    _, q, sf, _, _ = _case(m, n, k, dtype)
    x = torch.eye(m, k, dtype=ref.DT[dtype])
    got = _run(x.cuda(), q, sf, 4.0, swiglu=True, out_dtype=torch.float32).cpu().double()
    y = ref.values(q, sf)[:, :m].t() * 4
    g, u = y[:, :n // 2], y[:, n // 2:]
    assert float(g.min()) < -30 and float(g.max()) > 30
    want = g * torch.sigmoid(g) * u
    assert ((got - want).abs() <= 6 * ref.U * (1 + 2 ** -6) * want.abs()).all(), \
        float(((got - want).abs() / want.abs().clamp(min=1e-300)).max() / ref.U)


def test_linear_pitches_and_untouched_columns():
    m, n, k = 6, 45, 176
    rng, q, sf, x, scale = _case(m, n, k, "bf16")
    wide = torch.full((m, k + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :k] = x.cuda()
    res = torch.full((m, n + 3), float("nan"), dtype=torch.bfloat16, device="cuda")
    r = torch.from_numpy(rng.standard_normal((m, n))).bfloat16()
    res[:, :n] = r.cuda()
    out = torch.full((m + 1, n + 5), 7.0, dtype=torch.float32, device="cuda")
    got = _run(wide[:, :k], q, sf, scale, residual=res[:, :n], out=out[:m, :n])
    assert got.data_ptr() == out.data_ptr()
    ref.check(out[:m, :n], *ref.linear(x.double(), ref.values(q, sf), scale, residual=r.double()))
    assert (out[:, n:] == 7).all() and (out[m] == 7).all()


def test_linear_adds_onto_the_residual_in_place():
    m, n, k = 5, 64, 128
    rng, q, sf, x, scale = _case(m, n, k, "fp16")
    r = torch.from_numpy(rng.standard_normal((m, n))).half()
    y = r.cuda()
    _run(x.cuda(), q, sf, scale, residual=y, out=y)
    ref.check(y, *ref.linear(x.double(), ref.values(q, sf), scale, residual=r.double()))


@pytest.mark.parametrize("k", [64, 80, 256, 272, 784, 2064])
def test_linear_nothing_leaks_across_rows_and_tokens(k):
    """A NaN block scale stays in its row, a NaN or infinity in its token, at the rows'
    ends too."""
    m, n = 5, 20
    _, q, sf, x, scale = _case(m, n, k, "bf16")
    sf[7, 0] = 0x7F    # the block right behind row 6's end
    sf[11, -1] = 0xFF  # the block right before row 12's start
    x[1, 0] = float("nan")
    x[3, k - 1] = float("inf")
    got = _run(x.cuda(), q, sf, scale).cpu()
    assert got[1].isnan().all() and got[:, 7].isnan().all() and got[:, 11].isnan().all()
    rows, cols = [0, 2, 4], [j for j in range(n) if j not in (7, 11)]
    y, d = ref.linear(x[rows].double(), ref.values(q, sf)[cols], scale)
    ref.check(got[rows][:, cols], y, d)
    last = ref.values(q, sf)[:, -1]
    for j in cols:  # infinity times the row's last weight
        assert got[3, j].isnan() if last[j] == 0 else got[3, j] == float("inf") * last[j].sign()


def test_linear_large_and_small_activations():
    """BF16 keeps its range: activations near 2^100 and 2^-100 multiply exactly."""
    for e in (100, -100):
        _, q, sf, x, scale = _case(3, 32, 128, "bf16", gain=2.0 ** e)
        ref.check(_run(x.cuda(), q, sf, scale, out_dtype=torch.float32),
                  *ref.linear(x.double(), ref.values(q, sf), scale), what=f"2^{e}")


def test_linear_zero_rows():
    _, q, sf, x, scale = _case(1, 32, 64, "bf16")
    assert _run(x[:0].cuda(), q, sf, scale).shape == (0, 32)


def test_linear_offsets_up_to_31_bits():
    """Weights of nearly 2^31 bytes: the first and last rows."""
    n, k = 131071, 32752
    say("linear 2 GiB of codes")
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    sf = torch.randint(0x28, 0x40, (n, k // 16), dtype=torch.uint8, device="cuda", generator=g)
    x = torch.randn(2, k, device="cuda", generator=g).bfloat16()
    from block_scaled_fp4_05_amd import moe_fp4
    got = moe_fp4.linear(x, q, sf, torch.tensor([0.01], device="cuda"), out_dtype=torch.float32)
    rows = [0, 1, 65535, 65536, n - 17, n - 2, n - 1]
    w = ref.values(q[rows].cpu().numpy(), sf[rows].cpu().numpy())
    ref.check(got[:, rows], *ref.linear(x.cpu().double(), w, float(np.float32(0.01))))


@pytest.mark.parametrize("m,n,k", [(2, 100, 1040), (16, 8200, 256)])
def test_linear_repeats_its_bits_on_other_streams_and_in_graphs(m, n, k):
    from block_scaled_fp4_05_amd import moe_fp4
    _, q, sf, x, scale = _case(m, n, k, "bf16")
    x, q, sf, s = x.cuda(), dev(q), dev(sf), torch.tensor([scale], device="cuda")
    want = moe_fp4.linear(x, q, sf, s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = moe_fp4.linear(x, q, sf, s, stream=side)
    side.synchronize()
    assert torch.equal(other, want)
    g, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(g):
        moe_fp4.linear(x, q, sf, s, out=out)
    for i in range(3):
        x.copy_(torch.roll(x, 1, 1))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, moe_fp4.linear(x, q, sf, s)), i
