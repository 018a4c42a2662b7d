"""The FP8 operators at the largest sizes that they take: every 32-bit buffer offset just below its
limit, every 64-bit one past 2^31, grids of more than one row; sampled rows and columns against 64 bits."""
import numpy as np
import pytest
import torch

import fp8_paths as paths
import fp8_ref as ref
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

LIMIT = 2 ** 31 - 4096  # n * k, and a_rows * k with a row index, are below


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()


def codes(seed, *shape):
    """Random E4M3 codes below 2 in magnitude."""
    g = torch.Generator("cuda").manual_seed(seed)
    q = torch.randint(0, 0x40, shape, dtype=torch.uint8, device="cuda", generator=g)
    return q.bitwise_or_(torch.randint(0, 2, shape, dtype=torch.uint8, device="cuda", generator=g) << 7).view(ref.FP8)


def scales(seed, *shape):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.rand(*shape, device="cuda", generator=g).add_(0.5)


def check(out, a, sa, w, sw, rows, source, expert, eight_bit, take=5):
    """Result rows `rows` (of rows `source` of a, `expert` of w), first, last and some other columns."""
    n, k = w.shape[1:]
    cols = sorted({0, n - 1, n // 2, max(0, n - 129), min(n - 1, 77)})[:take]
    wb = w.view(torch.uint8)
    for r, s, e in zip(rows, source, expert):
        av = torch.from_numpy(ref.values(a.view(torch.uint8)[s:s + 1], sa[s:s + 1], 1)).cuda()
        wv = torch.cat([wb[e, c:c + 1] for c in cols])
        ws = torch.stack([sw[e, c // 128] for c in cols])
        wv = torch.from_numpy(ref.values(wv, ws, 1)).cuda()
        p = av * wv
        # Inside a block 128 additions, each off by a step of at most the block's size, and a few
        # roundings; from block to block half a step of a sum of some consecutive ones.
        sums = torch.nn.functional.pad(p, (0, -k % 128)).view(len(cols), -1, 128).sum(2).cumsum(1)
        bound = 2 * (128 + 16) * ref.U * p.abs().sum(1) + 4 * (ref.blocks(k) + 8) * ref.U * sums.abs().amax(1)
        if eight_bit:
            bound = bound + 7 * 2.0 ** -13 * torch.nn.functional.pad(p.abs(), (0, -k % 8)).view(len(cols), -1, 8).amax(2).sum(1)
        ref.check(out[r, cols], p.sum(1).cpu(), bound.cpu(), f"row {r}")


@pytest.mark.parametrize("m,dtype,kernel", [
    (1, "bf16", "stream 4 1"), (100, "bf16", "tile 64 three stages"), (300, "fp16", "tile 128"),
    (1024, "bf16", "tile 256"), (300, "fp32", "tile 128 exact")])
def test_weights_of_just_below_two_to_the_31(m, dtype, kernel):
    from block_scaled_fp4_05_amd import moe_fp4
    n, k = 32768, 65520
    assert n * k < LIMIT < (n + 16) * k and paths.kernel(m, 1, n, k, dtype) == kernel
    say(f"linear_fp8 {m} x {n} x {k} {dtype}")
    a, sa, w, sw = codes(1, m, k), scales(2, m, ref.blocks(k)), codes(3, n, k), scales(4, ref.blocks(n), ref.blocks(k))
    if dtype == "fp16":
        sw *= 2.0 ** -8
    out = moe_fp4.linear_fp8(a, sa, w, sw, out_dtype=ref.DT[dtype])
    rows = sorted({0, m - 1})
    check(out, a, sa, w[None], sw[None], rows, rows, [0] * 2, dtype != "fp32")


@pytest.mark.parametrize("m,dtype,kernel", [(3, "fp32", "stream 1 1"), (2000, "bf16", "tile 64 three stages"),
                                            (2000, "fp32", "tile 64 exact")])
def test_longest_k(m, dtype, kernel):
    from block_scaled_fp4_05_amd import moe_fp4
    n, k = 511, 2 ** 22
    assert n * k < LIMIT < (n + 1) * k and paths.kernel(m, 1, n, k, dtype) == kernel
    say(f"linear_fp8 {m} x {n} x {k} {dtype}")
    a, sa, w, sw = codes(1, m, k), scales(2, m, k // 128), codes(3, n, k), scales(4, ref.blocks(n), k // 128)
    out = moe_fp4.linear_fp8(a, sa, w, sw, out_dtype=ref.DT[dtype])
    check(out, a, sa, w[None], sw[None], [0, m - 1], [0, m - 1], [0] * 2, dtype != "fp32")


@pytest.mark.parametrize("m,n,dtype,kernel", [(40, 600, "fp32", "stream 4 2"), (700, 4000, "bf16", "tile 64 three stages"),
                                              (2000, 7168, "bf16", "tile 256"), (1100, 8000, "fp32", "tile 128 exact")])
def test_gathered_rows_of_just_below_two_to_the_31(m, n, dtype, kernel):
    from block_scaled_fp4_05_amd import moe_fp4
    rows, k = 32767, 65520
    assert rows * k < LIMIT < (rows + 16) * k and paths.kernel(m, 1, n, k, dtype) == kernel
    say(f"grouped_gemm_fp8 {m} of {rows} x {k}, {n} columns {dtype}")
    a, sa = codes(1, rows, k), scales(2, rows, ref.blocks(k))
    w, sw = codes(3, 1, n, k), scales(4, 1, ref.blocks(n), ref.blocks(k))
    index = torch.randint(0, rows, (m,), dtype=torch.int32, device="cuda")
    index[0], index[m - 1], index[m - 2] = rows - 1, 2 ** 31 - 1, 0
    offsets = torch.tensor([0, m], dtype=torch.int32, device="cuda")
    out = moe_fp4.grouped_gemm_fp8(a, sa, w, sw, offsets, a_row_index=index, out_dtype=ref.DT[dtype])
    check(out, a, sa, w, sw, [0, m - 2, m - 1], [rows - 1, 0, rows - 1], [0] * 3, dtype != "fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_and_experts_past_two_to_the_31(dtype):
    """Rows without an index, of 4.6 GB, tiles; and 8192 experts of 8.6 GB in all with 2.1 GB of rows, the
    few-row kernel."""
    from block_scaled_fp4_05_amd import moe_fp4
    m, n, k = 70000, 16, 65520
    say(f"linear_fp8 {m} x {n} x {k} {dtype}")
    a, sa, w, sw = codes(1, m, k), scales(2, m, ref.blocks(k)), codes(3, n, k), scales(4, 1, ref.blocks(k))
    out = moe_fp4.linear_fp8(a, sa, w, sw, out_dtype=ref.DT[dtype])
    rows = [0, 40000, m - 1]
    check(out, a, sa, w[None], sw[None], rows, rows, [0] * 3, dtype != "fp32")
    del a, sa, w, sw
    E, m, k = 8192, 32767, 65552
    assert m < 4 * E and m * k > 2 ** 31
    say(f"grouped_gemm_fp8 {E} experts, {m} x {n} x {k} {dtype}")
    a, sa, w, sw = codes(1, m, k), scales(2, m, ref.blocks(k)), codes(3, E, n, k), scales(4, E, 1, ref.blocks(k))
    offsets = torch.arange(E + 1, dtype=torch.int32, device="cuda") * 4
    offsets[E] = m
    out = moe_fp4.grouped_gemm_fp8(a, sa, w, sw, offsets, out_dtype=ref.DT[dtype])
    rows = [0, 20001, m - 1]
    check(out, a, sa, w, sw, rows, rows, [r // 4 for r in rows], False)


@pytest.mark.parametrize("m,n,k,dtype,kernel", [
    (700, 300, 144, "fp32", "stream 4 4"), (700, 5000, 144, "fp32", "tile 64 exact"), (1500, 5000, 656, "bf16", "tile 64"),
    (1100, 2 ** 20, 16, "fp32", "tile 128 exact"), (1100, 2 ** 20, 512, "bf16", "short 128 span 4")])
def test_widest_output(m, n, k, dtype, kernel):
    """Pitch 2^20, results past 2^31 bytes; the last but one with more workgroups than one row of a grid."""
    from block_scaled_fp4_05_amd import moe_fp4
    assert paths.kernel(m, 1, n, k, dtype) == kernel
    say(f"linear_fp8 {m} x {n} x {k} {dtype}, pitch 2^20")
    a, sa, w, sw = codes(1, m, k), scales(2, m, ref.blocks(k)), codes(3, n, k), scales(4, ref.blocks(n), ref.blocks(k))
    wide = torch.full((m + 1, 2 ** 20), 7.0, dtype=ref.DT[dtype], device="cuda")
    assert wide[:m].numel() * wide.element_size() > 2 ** 31
    moe_fp4.linear_fp8(a, sa, w, sw, out=wide[:m, :n])
    check(wide, a, sa, w[None], sw[None], [0, m // 2, m - 1], [0, m // 2, m - 1], [0] * 3, dtype != "fp32")
    assert (wide[m] == 7).all() and (wide[:, n:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_most_rows(dtype):
    from block_scaled_fp4_05_amd import moe_fp4
    m, n, k = LIMIT // 4 - 1, 16, 16
    say(f"linear_fp8 {m} x {n} x {k} {dtype}")
    part, sa = codes(1, 1 << 20, k), scales(2, m, 1)
    a = torch.empty(m, k, dtype=torch.uint8, device="cuda")
    for i in range(0, m, 1 << 20):
        a[i:i + (1 << 20)] = part.view(torch.uint8)[:min(1 << 20, m - i)]
    a = a.view(ref.FP8)
    w, sw = codes(3, n, k), scales(4, 1, 1)
    out = moe_fp4.linear_fp8(a, sa, w, sw, out_dtype=ref.DT[dtype])
    rows = [0, 2 ** 28 + 12345, m - 129, m - 1]
    check(out, a, sa, w[None], sw[None], rows, rows, [0] * 4, dtype != "fp32")


def same(q, s, x, tall=1):
    want_q, want_s = ref.quantize(x.float().cpu().numpy(), tall)
    assert np.array_equal(q.cpu().view(torch.uint8).numpy(), want_q) and np.array_equal(s.cpu().numpy(), want_s)


def test_quantised_rows_past_two_to_the_31():
    from block_scaled_fp4_05_amd import moe_fp4
    rows, k = 300_000, 8192
    say(f"quantize_fp8 {rows} x {k}")
    x = torch.randn(1000, k, device="cuda").bfloat16().repeat(300, 1)
    x *= torch.rand(rows, 1, device="cuda").bfloat16()
    q, s = moe_fp4.quantize_fp8(x)
    for r in (0, 262_143, rows - 1):
        same(q[r:r + 1], s[r:r + 1], x[r:r + 1])


def test_longest_quantised_row():
    from block_scaled_fp4_05_amd import moe_fp4
    k = 2 ** 29 - 1152  # whole blocks below the limit of 2^29 - 1024
    say(f"quantize_fp8 1 x {k}, plain and SwiGLU's gradient")
    x = torch.empty(1, 2 * k, dtype=torch.bfloat16, device="cuda").normal_()
    q, s = moe_fp4.quantize_fp8(x[:, :k])
    for c in (0, k // 2 // 128 * 128, k - 256):
        same(q[:, c:c + 256], s[:, c // 128:c // 128 + 2], x[:, c:c + 256])
    d = torch.empty(1, k, dtype=torch.bfloat16, device="cuda").normal_()
    q, s = moe_fp4.quantize_fp8(x, swiglu=True, grad=d)
    for c in (0, k - 256):
        part = torch.cat((x[:, c:c + 256], x[:, k + c:k + c + 256]), 1).double().cpu().numpy()
        v, off = ref.swiglu_grad(part, d[:, c:c + 256].double().cpu().numpy())
        for half, at in enumerate((c, k + c)):
            cols = slice(256 * half, 256 * half + 256)
            ref.check_quantized(q[:, at:at + 256], s[:, at // 128:at // 128 + 2], v[:, cols], off[:, cols], False, f"{at}")


def test_largest_quantised_weights():
    from block_scaled_fp4_05_amd import moe_fp4
    E, n, k = 2, 32768, 65520
    assert n * k < LIMIT
    say(f"quantize_fp8_weights {E} x {n} x {k}")
    w = torch.empty(E, n, k, dtype=torch.bfloat16, device="cuda").normal_()
    q, s, qt, st = moe_fp4.quantize_fp8_weights(w, transposed=True)
    for e in range(E):
        for r, c in ((0, 0), (n - 128, k // 128 * 128)):
            part, where = w[e, r:r + 128, c:c + 128], (e, slice(r, r + 128), slice(c, c + 128))
            same(q[where], s[e, r // 128:r // 128 + 1, c // 128:c // 128 + 1], part, 128)
            assert torch.equal(qt[e, c:c + 128, r:r + 128].view(torch.uint8), q[where].view(torch.uint8).t())
            assert st[e, c // 128, r // 128] == s[e, r // 128, c // 128]
