"""Scales whose product is no FP32 number, or a subnormal one with few bits, where the result is a
number: in every kernel of the FP8 product."""
import numpy as np
import pytest
import torch

import fp8_paths as paths
import fp8_ref as ref
from gpu_util import require_gpu, say
from test_gpu_gemm_fp8 import check_sampled, i32, on_gpu, operands as ordinary

pytestmark = pytest.mark.gpu

# (exponents of activation scales, of weight scales, codes).  Products of scales of 2^122 to 2^132
# with values of 2^-9 to 2^-7 (their products' sums stay below 2^127); products of 2^-146 to
# 2^-136 with values of 224 to 448 (sums of about 2^20).
RANGES = {"large": ((60, 66), (62, 66), (1, 5)), "small": ((-76, -70), (-70, -66), (0x76, 0x7F))}


def operands(seed, rows, E, n, k, which):
    rng = np.random.default_rng(seed)
    ea, ew, codes = RANGES[which]

    def fp8(*shape):
        return rng.integers(*codes, shape, dtype=np.uint8) | (rng.integers(0, 2, shape, dtype=np.uint8) << 7)

    def scales(e, *shape):
        return np.exp2(rng.uniform(*e, shape)).astype(np.float32)

    return (fp8(rows, k), scales(ea, rows, ref.blocks(k)), fp8(E, n, k), scales(ew, E, ref.blocks(n), ref.blocks(k)))


@pytest.mark.parametrize("which", RANGES)
@pytest.mark.parametrize("name", paths.PATHS)
def test_products_of_scales_outside_fp32(name, which):
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    counts, n, k, dtype = paths.PATHS[name]
    dtype = "bf16" if dtype == "fp16" else dtype  # (FP16 has no such numbers; the kernels are the same)
    say(f"grouped_gemm_fp8 {name}, {which} scales")
    offsets = paths.offsets(name)
    a, sa, w, sw = operands(n + k, int(offsets[-1]), len(counts), n, k, which)
    out = m.grouped_gemm_fp8(*on_gpu(a, sa, w, sw), i32(offsets), out_dtype=ref.DT[dtype])
    check_sampled(out, a, sa, w, sw, offsets, dtype != "fp32", n)


@pytest.mark.parametrize("name", paths.PATHS)
def test_zeros_infinities_and_nan_as_scales(name):
    """Rows and weight blocks of zeros with the least scale (as the quantisers give them) among others,
    scales of zero on codes that are not: nothing is added.  An infinite or NaN scale, on zeros
    too, leaves nothing finite in its row, and touches no other."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    counts, n, k, dtype = paths.PATHS[name]
    say(f"grouped_gemm_fp8 {name}, zeros and infinite scales")
    offsets = paths.offsets(name)
    rows = int(offsets[-1])
    a, sa, w, sw = ordinary(n + k, rows, len(counts), n, k)
    if dtype == "fp16":
        sa, sw = sa * np.float32(2.0 ** -6), sw * np.float32(2.0 ** -6)
    a[1::3], sa[1::3] = 0, 2.0 ** -126
    w[:, :128, :128], sw[:, 0, 0] = 0, 2.0 ** -126
    sa[2::5, 0] = 0
    sw[:, -1, -1] = 0
    args = on_gpu(a, sa, w, sw)
    out = m.grouped_gemm_fp8(*args, i32(offsets), out_dtype=ref.DT[dtype])
    check_sampled(out, a, sa, w, sw, offsets, dtype != "fp32", n)
    bad = {0: np.inf, rows - 1: np.nan, rows // 2: -np.inf}
    for row, s in bad.items():
        args[1][row, -1] = float(s)
    args[0].view(torch.uint8)[rows // 2] = 0
    again = m.grouped_gemm_fp8(*args, i32(offsets), out_dtype=ref.DT[dtype])
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[list(bad)] = False
    assert torch.equal(again[keep], out[keep])
    assert not again[~keep].isfinite().any()
