"""The FP8 block-scaled product against its 64-bit sum, over expert sizes, tails, types and layouts."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


def operands(seed, rows, E, n, k):
    """Random codes (no NaN) and scales of both signs' products."""
    rng = np.random.default_rng(seed)

    def codes(*shape):
        q = rng.integers(0, 0x7F, shape, dtype=np.uint8) | (rng.integers(0, 2, shape, dtype=np.uint8) << 7)
        return np.where(rng.random(shape) < 0.5, q & 0xBF, q).astype(np.uint8)

    a, w = codes(rows, k), codes(E, n, k)
    sa = np.exp2(rng.uniform(-6, 3, (rows, ref.blocks(k)))).astype(np.float32)
    sw = np.exp2(rng.uniform(-9, 2, (E, ref.blocks(n), ref.blocks(k)))).astype(np.float32)
    return a, sa, w, sw


def on_gpu(a, sa, w, sw):
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    return t(a).view(ref.FP8), t(sa), t(w).view(ref.FP8), t(sw)


def expected(a, sa, w, sw, offsets, index=None, eight_bit=False):
    av = ref.values(a, sa, 1)
    if index is not None:
        av = av[index]
    y = torch.zeros(offsets[-1], w.shape[1], dtype=torch.float64)
    b = torch.zeros_like(y)
    for e in range(w.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        if lo < hi:
            y[lo:hi], b[lo:hi] = ref.product(av[lo:hi], ref.values(w[e], sw[e], 128), eight_bit)
    return y, b


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# Rows of each expert: few, none, tiles that end inside, an expert above every tile's height.
COUNTS = {
    "one row": [1],
    "one of many": [0] * 5 + [1] + [0] * 3,
    "decode": [1, 0, 2, 3, 0, 1, 4, 0],
    "sixteen": [16, 15, 17, 16],
    "thirty": [31, 33, 1, 32],
    "sixties": [63, 64, 65, 0, 66],
    "hundreds": [127, 128, 129, 0, 200],
    "mixed": [300, 0, 5, 64, 257, 1, 40],
    "large": [512, 255, 256],
}


@pytest.mark.parametrize("n,k", [(16, 16), (128, 128), (130, 144), (256, 384), (333, 1040)])
@pytest.mark.parametrize("counts", COUNTS)
def test_expert_sizes(counts, n, k):
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"grouped_gemm_fp8 {counts} n={n} k={k}")
    offsets = np.concatenate(([0], np.cumsum(COUNTS[counts])))
    a, sa, w, sw = operands(n + k, offsets[-1], len(COUNTS[counts]), n, k)
    out = m.grouped_gemm_fp8(*on_gpu(a, sa, w, sw), i32(offsets), out_dtype=torch.float32)
    ref.check(out, *expected(a, sa, w, sw, offsets), counts)
    out = m.grouped_gemm_fp8(*on_gpu(a, sa, w, sw), i32(offsets))
    ref.check(out, *expected(a, sa, w, sw, offsets, eight_bit=True), counts)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("counts,n,k", [("decode", 96, 272), ("thirty", 200, 512), ("mixed", 136, 400)])
def test_types_row_index_and_pitch(counts, n, k, dtype):
    """Gathered rows (some twice, some clamped), an output wider than the result, rows outside the
    offsets and columns past n left as they were."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    offsets = np.concatenate(([0], np.cumsum(COUNTS[counts])))
    M, T = int(offsets[-1]), 23
    a, sa, w, sw = operands(M + n, T, len(COUNTS[counts]), n, k)
    if dtype == "fp16":  # results inside FP16's range: products of up to 2^16 k
        sa, sw = sa * np.float32(2.0 ** -6), sw * np.float32(2.0 ** -6)
    index = np.random.default_rng(M).integers(0, T, M + 7)
    index[1], index[2] = -5, T + 9
    for ldo in (n + 5, n + 24):
        say(f"grouped_gemm_fp8 gathered {counts} n={n} k={k} {dtype} ldo={ldo}")
        out = torch.full((M + 7, ldo), 7.0, dtype=ref.DT[dtype], device="cuda")
        m.grouped_gemm_fp8(*on_gpu(a, sa, w, sw), i32(offsets), a_row_index=i32(index), out=out[:, :n])
        ref.check(out[:M, :n], *expected(a, sa, w, sw, offsets, np.clip(index, 0, T - 1)[:M], dtype != "fp32"), dtype)
        assert (out[M:] == 7).all() and (out[:, n:] == 7).all()


@pytest.mark.parametrize("mrows", [1, 3, 16, 17, 64, 65, 128, 200, 256, 600])
@pytest.mark.parametrize("n,k", [(24, 144), (640, 768)])
def test_dense(mrows, n, k):
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"linear_fp8 {mrows} x {n} x {k}")
    a, sa, w, sw = operands(mrows, mrows, 1, n, k)
    aq, asf, wq, wsf = on_gpu(a, sa, w, sw)
    out = m.linear_fp8(aq, asf, wq[0], wsf[0], out_dtype=torch.float32)
    ref.check(out, *expected(a, sa, w, sw, [0, mrows]), "dense")
    assert torch.equal(out, m.linear_fp8(aq, asf, wq[0], wsf[0], out_dtype=torch.float32))
    out = m.linear_fp8(aq, asf, wq[0], wsf[0])
    ref.check(out, *expected(a, sa, w, sw, [0, mrows], eight_bit=True), "dense bf16")
    assert torch.equal(out, m.linear_fp8(aq, asf, wq[0], wsf[0]))


def test_large_dense():
    """Several workgroups in every direction: partial tiles at both ends."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    a, sa, w, sw = operands(5, 1100, 1, 1300, 1168)
    aq, asf, wq, wsf = on_gpu(a, sa, w, sw)
    out = m.linear_fp8(aq, asf, wq[0], wsf[0], out_dtype=torch.float32)
    ref.check(out, *expected(a, sa, w, sw, [0, 1100]), "large dense")
    out = m.linear_fp8(aq, asf, wq[0], wsf[0])
    ref.check(out, *expected(a, sa, w, sw, [0, 1100], eight_bit=True), "large dense bf16")


def sampled(rows, n, seed):
    """Some result rows and columns, the first and last ones among them."""
    rng = np.random.default_rng(seed)
    pick = lambda size: np.unique(np.concatenate((rng.integers(0, size, 150), [0, 1, size - 2, size - 1])))  # noqa: E731
    return pick(rows), pick(n)


def check_sampled(out, a, sa, w, sw, offsets, eight_bit, seed):
    rows, cols = sampled(out.shape[0], out.shape[1], seed)
    y = torch.zeros(len(rows), len(cols), dtype=torch.float64)
    b = torch.zeros_like(y)
    for e in range(w.shape[0]):
        at = np.nonzero((rows >= offsets[e]) & (rows < offsets[e + 1]))[0]
        if len(at):
            wv = ref.values(w[e], sw[e], 128)[cols]
            y[at], b[at] = ref.product(ref.values(a[rows[at]], sa[rows[at]], 1), wv, eight_bit)
    ref.check(out.cpu()[rows][:, cols], y, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,n,k", [(3580, 4000, 400), (2050, 7304, 1168), (400, 16380, 272)])
def test_many_tiles_dense(rows, n, k, dtype):
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"linear_fp8 {rows} x {n} x {k} {dtype}")
    a, sa, w, sw = operands(rows, rows, 1, n, k)
    aq, asf, wq, wsf = on_gpu(a, sa, w, sw)
    out = m.linear_fp8(aq, asf, wq[0], wsf[0], out_dtype=ref.DT[dtype])
    check_sampled(out, a, sa, w, sw, [0, rows], dtype != "fp32", rows)
    assert torch.equal(out, m.linear_fp8(aq, asf, wq[0], wsf[0], out_dtype=ref.DT[dtype]))


@pytest.mark.parametrize("dtype", ["fp16", "fp32"])
@pytest.mark.parametrize("E,avg,n,k", [(40, 130, 900, 272), (6, 420, 2600, 144), (64, 12, 2048, 528), (96, 3, 520, 1040)])
def test_many_tiles_of_many_experts(E, avg, n, k, dtype):
    """Uneven experts, some empty, rows gathered through an index."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"grouped_gemm_fp8 {E} experts of {avg} rows, {n} x {k} {dtype}")
    rng = np.random.default_rng(E)
    counts = rng.multinomial(E * avg, rng.dirichlet(np.full(E, 3.0)))
    counts[E // 2] = 0
    offsets = np.concatenate(([0], np.cumsum(counts)))
    M, T = int(offsets[-1]), 333
    a, sa, w, sw = operands(E, T, E, n, k)
    sa, sw = sa * np.float32(2.0 ** -6), sw * np.float32(2.0 ** -6)
    index = rng.integers(0, T, M)
    out = m.grouped_gemm_fp8(*on_gpu(a, sa, w, sw), i32(offsets), a_row_index=i32(index), out_dtype=ref.DT[dtype])
    check_sampled(out, a[index], sa[index], w, sw, offsets, dtype != "fp32", E)


def test_many_experts():
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    rng = np.random.default_rng(1)
    for E, most in ((700, 3), (1500, 2), (257, 40)):
        counts = rng.integers(0, most + 1, E)
        offsets = np.concatenate(([0], np.cumsum(counts)))
        a, sa, w, sw = operands(E, offsets[-1], E, 32, 128)
        say(f"grouped_gemm_fp8 {E} experts")
        out = m.grouped_gemm_fp8(*on_gpu(a, sa, w, sw), i32(offsets), out_dtype=torch.float32)
        ref.check(out, *expected(a, sa, w, sw, offsets), f"{E} experts")


@pytest.mark.parametrize("rows", [5, 40, 300])
def test_nan_stays_in_its_row_and_column(rows):
    """A NaN code of a row or of a weight touches that row or column alone; NaN in the memory behind
    a row's last block touches nothing."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    n, k = 144, 272
    a, sa, w, sw = operands(rows, rows, 1, n, k)
    aq, asf, wq, wsf = on_gpu(a, sa, w, sw)
    clean = {t: m.linear_fp8(aq, asf, wq[0], wsf[0], out_dtype=t) for t in ref.DT.values()}
    bad_a, bad_w = aq.view(torch.uint8).clone(), wq[0].view(torch.uint8).clone()
    bad_a[rows - 2, k - 1], bad_w[7, 0] = 0x7F, 0xFF
    hit = torch.zeros(rows, n, dtype=torch.bool, device="cuda")
    hit[rows - 2], hit[:, 7] = True, True
    for t, want in clean.items():
        out = m.linear_fp8(bad_a.view(ref.FP8), asf, bad_w.view(ref.FP8), wsf[0], out_dtype=t)
        assert torch.equal(out.isnan(), hit | want.isnan())
        assert torch.equal(out[~out.isnan()], want[~out.isnan()])


def test_offsets_outside_the_rows_are_clamped():
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    a, sa, w, sw = operands(3, 20, 3, 48, 144)
    out = torch.full((20, 48), 3.0, device="cuda")
    m.grouped_gemm_fp8(*on_gpu(a, sa, w, sw), i32([-4, 6, 4, 90]), out=out)  # expert 1: none; 2: 4 .. 20
    y, b = expected(a, sa, w, sw, [0, 4, 4, 20])
    ref.check(out[6:], y[6:], b[6:])
    ref.check(out[:4], y[:4], b[:4])


def test_replayed_graph_follows_its_inputs():
    """Offsets, rows and weights change between replays; eager work runs in between."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    E, n, k, M = 6, 160, 400, 150
    rng = np.random.default_rng(2)
    ops = on_gpu(*operands(1, M, E, n, k))
    off = i32(np.concatenate(([0], np.sort(rng.integers(0, M, E - 1)), [M])))
    m.grouped_gemm_fp8(*ops, off)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = m.grouped_gemm_fp8(*ops, off)
    for i in range(3):
        new = on_gpu(*operands(10 + i, M, E, n, k))
        for t, v in zip(ops, new):
            t.view(torch.uint8).copy_(v.view(torch.uint8))
        off.copy_(i32(np.concatenate(([0], np.sort(rng.integers(0, M, E - 1)), [M]))))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, m.grouped_gemm_fp8(*ops, off))


@pytest.mark.parametrize("counts,n,k,gather", [
    ([70, 0, 128, 33, 64, 65, 150, 1, 17, 200, 90, 22], 1156, 4112, False),
    ([5, 16, 64, 0, 48, 31, 130, 12] * 2, 1160, 4096, True), ([60] * 12, 1032, 4240, True)])
def test_long_products_of_small_experts(counts, n, k, gather):
    """Tiles of 64 rows with three stages in LDS: counts of blocks of every remainder by three."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"grouped_gemm_fp8 {len(counts)} experts n={n} k={k} gather={gather}")
    offsets = np.concatenate(([0], np.cumsum(counts)))
    M = int(offsets[-1])
    rows = 77 if gather else M
    a, sa, w, sw = operands(n + k, rows, len(counts), n, k)
    index = np.random.default_rng(k).integers(0, rows, M) if gather else None
    out = m.grouped_gemm_fp8(*on_gpu(a, sa, w, sw), i32(offsets), a_row_index=i32(index) if gather else None)
    ref.check(out, *expected(a, sa, w, sw, offsets, index, eight_bit=True), counts)


@pytest.mark.parametrize("E,M,n,k", [(8192, 700, 160, 16), (64, 400, 400, 272), (6, 900, 1160, 4112)])
def test_offsets_that_go_back_and_forth_stay_inside(E, M, n, k):
    """Far more rows in all than there are: which of them are computed is open, rows behind the last
    one and columns past n stay."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"grouped_gemm_fp8 offsets back and forth, {E} experts")
    off = np.zeros(E + 1, dtype=np.int32)
    off[1::2] = M
    ops = on_gpu(*operands(E, M, E, n, k))
    out = torch.full((M + 300, n + 8), 7.0, device="cuda")
    m.grouped_gemm_fp8(*ops, i32(off), out=out[:M, :n])
    assert (out[M:] == 7).all() and (out[:, n:] == 7).all() and out.isfinite().all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("k", [16, 112, 128, 240, 384, 400, 512])
@pytest.mark.parametrize("E,avg,n,gather", [(40, 30, 3000, True), (24, 150, 4004, False), (1, 700, 16400, False)])
def test_short_products_with_many_tiles(E, avg, n, gather, k, dtype):
    """Workgroups that run along the weights' tiles: one to four blocks, the last one whole or not,
    uneven experts, spans that end inside the matrix; rows and columns outside are left."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"grouped_gemm_fp8 short {E} experts of {avg} rows, {n} x {k} gather={gather} {dtype}")
    rng = np.random.default_rng(E + k)
    counts = rng.multinomial(E * avg, rng.dirichlet(np.full(E, 3.0)))
    if E > 1:
        counts[1] = 0
    offsets = np.concatenate(([0], np.cumsum(counts)))
    M = int(offsets[-1])
    rows = 211 if gather else M
    a, sa, w, sw = operands(E + k, rows, E, n, k)
    sa, sw = sa * np.float32(2.0 ** -6), sw * np.float32(2.0 ** -6)
    index = rng.integers(0, rows, M) if gather else None
    out = torch.full((M + 3, n + 8), 7.0, dtype=ref.DT[dtype], device="cuda")
    m.grouped_gemm_fp8(*on_gpu(a, sa, w, sw), i32(offsets), a_row_index=i32(index) if gather else None,
                       out=out[:M, :n])
    at = (lambda x: x[index]) if gather else (lambda x: x)
    check_sampled(out[:M, :n], at(a), at(sa), w, sw, offsets, True, E + k)
    assert (out[M:] == 7).all() and (out[:, n:] == 7).all()
