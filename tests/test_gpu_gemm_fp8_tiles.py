"""Every kernel of the FP8 product (fp8_paths.py) with uneven and empty experts, gathered rows, clamped
indices, every width of stores, NaN, dense calls and replayed graphs."""
import numpy as np
import pytest
import torch

import fp8_paths as paths
import fp8_ref as ref
from gpu_util import require_gpu, say
from test_gpu_gemm_fp8 import check_sampled, i32, on_gpu, operands

pytestmark = pytest.mark.gpu

# layout -> (multiple of n, columns of the output behind n): stores of eight columns, four and one.
LAYOUTS = {"eight": (8, 8), "four": (4, 4), "one": (1, 3)}


def case(name, multiple=1):
    """Offsets, n, k and type of a path, n rounded down to a multiple; the kernel stays the path's."""
    counts, n, k, dtype = paths.PATHS[name]
    n = n // multiple * multiple - (4 if multiple == 4 and n // 4 % 2 == 0 else 0)
    assert paths.kernel(sum(counts), len(counts), n, k, dtype) == name
    return paths.offsets(name), n, k, dtype


def small(sa, sw, dtype):
    """Scales whose results are inside FP16's range."""
    return (sa * np.float32(2.0 ** -6), sw * np.float32(2.0 ** -6)) if dtype == "fp16" else (sa, sw)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("name", paths.PATHS)
def test_gathered_rows_and_stores(name, layout):
    """Rows in any order, some twice, some through an index outside (the nearest row is taken); columns
    past n and rows behind the last one are left."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    multiple, more = LAYOUTS[layout]
    offsets, n, k, dtype = case(name, multiple)
    say(f"grouped_gemm_fp8 {name}, stores of {layout}, n={n}")
    M, T, E = int(offsets[-1]), 211, len(offsets) - 1
    a, sa, w, sw = operands(n + k, T, E, n, k)
    sa, sw = small(sa, sw, dtype)
    index = np.random.default_rng(n).integers(0, T, M + 3)
    index[[0, M // 2, M - 1]] = -5, T + 9, 2 ** 31 - 1
    out = torch.full((M + 3, n + more), 7.0, dtype=ref.DT[dtype], device="cuda")
    args = on_gpu(a, sa, w, sw)
    m.grouped_gemm_fp8(*args, i32(offsets), a_row_index=i32(index), out=out[:, :n])
    at = np.clip(index, 0, T - 1)[:M]
    check_sampled(out[:M, :n], a[at], sa[at], w, sw, offsets, dtype != "fp32", n)
    assert (out[M:] == 7).all() and (out[:, n:] == 7).all()


@pytest.mark.parametrize("name", paths.PATHS)
def test_nan_stays_in_its_row_and_column(name):
    """NaN codes in a row's last piece and in a weight's first (which is read in place of pieces past
    k), in an expert's last rows and columns: no other result changes."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    offsets, n, k, dtype = case(name)
    say(f"grouped_gemm_fp8 {name}, NaN")
    M, E = int(offsets[-1]), len(offsets) - 1
    a, sa, w, sw = operands(n, M, E, n, k)
    args = on_gpu(a, *small(sa, sw, dtype)[:1], w, small(sa, sw, dtype)[1])
    clean = m.grouped_gemm_fp8(*args, i32(offsets), out_dtype=ref.DT[dtype])
    hit = torch.zeros(M, n, dtype=torch.bool, device="cuda")
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo and e % 2 == 0:
            args[0].view(torch.uint8)[hi - 1, k - 1] = 0x7F
            hit[hi - 1] = True
        if hi > lo and e % 3 != 1:
            for col in (7, n - 1):
                args[2].view(torch.uint8)[e, col, 0] = 0xFF
                hit[lo:hi, col] = True
    out = m.grouped_gemm_fp8(*args, i32(offsets), out_dtype=ref.DT[dtype])
    assert torch.equal(out.isnan(), hit | clean.isnan())
    assert torch.equal(out[~hit], clean[~hit])


@pytest.mark.parametrize("kernel,m,n,k,dtype", [
    ("tile 64", 300, 5001, 1040, "fp16"), ("tile 64 three stages", 300, 5001, 4240, "bf16"),
    ("tile 64 exact", 300, 5001, 656, "fp32"), ("tile 128", 2050, 7303, 1168, "bf16"),
    ("tile 128 exact", 2050, 4102, 272, "fp32"), ("tile 256", 1900, 7171, 1040, "fp16"),
    ("tile 256", 1981, 7300, 1296, "bf16"), ("short 128 span 4", 900, 32770, 240, "bf16"),
    ("short 64 span 2", 80, 65601, 400, "bf16")])
def test_dense(kernel, m, n, k, dtype):
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4
    assert paths.kernel(m, 1, n, k, dtype) == kernel
    say(f"linear_fp8 {kernel}: {m} x {n} x {k} {dtype}")
    a, sa, w, sw = operands(n, m, 1, n, k)
    sa, sw = small(sa, sw, dtype)
    aq, asf, wq, wsf = on_gpu(a, sa, w, sw)
    out = moe_fp4.linear_fp8(aq, asf, wq[0], wsf[0], out_dtype=ref.DT[dtype])
    check_sampled(out, a, sa, w, sw, [0, m], dtype != "fp32", n)
    # As one expert of a grouped call: the same bits.
    assert torch.equal(out, moe_fp4.grouped_gemm_fp8(aq, asf, wq, wsf, i32([0, m]), out_dtype=ref.DT[dtype]))


@pytest.mark.parametrize("name", ["tile 64 three stages", "tile 128", "tile 256", "tile 128 exact", "short 64 span 3"])
def test_replayed_graph_follows_its_inputs(name):
    """Offsets, rows and weights change between replays; eager work runs in between."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    offsets, n, k, dtype = case(name)
    say(f"grouped_gemm_fp8 {name}, captured")
    M, E = int(offsets[-1]), len(offsets) - 1
    ops, off = on_gpu(*operands(1, M, E, n, k)), i32(offsets)
    m.grouped_gemm_fp8(*ops, off, out_dtype=ref.DT[dtype])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = m.grouped_gemm_fp8(*ops, off, out_dtype=ref.DT[dtype])
    rng = np.random.default_rng(2)
    for i in range(3):
        for t, v in zip(ops, on_gpu(*operands(10 + i, M, E, n, k))):
            t.view(torch.uint8).copy_(v.view(torch.uint8))
        off.copy_(i32(np.concatenate(([0], np.sort(rng.integers(0, M, E - 1)), [M]))))
        graph.replay()
        torch.cuda.synchronize()
        want = m.grouped_gemm_fp8(*ops, off, out_dtype=ref.DT[dtype])
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
