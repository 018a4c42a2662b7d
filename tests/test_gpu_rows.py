"""Rows into expert order and the gradients of the way there and back: copies and products bit for
bit, sums within their FP32 roundings, and the chain against autograd in 64 bits."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

TYPES = {**ref.DT, "fp8": ref.FP8}


def maps(seed, T, K, drop=0.0, extra=0):
    """token_rows and row_token of a random routing, rows renumbered where slots are dropped;
    `extra` rows that belong to no slot."""
    rng = np.random.default_rng(seed)
    rows = rng.permutation(T * K).reshape(T, K)
    keep = rng.random((T, K)) >= drop
    order = np.sort(rows[keep])
    new = np.full(T * K, -1)
    new[order] = np.arange(len(order))
    token_rows = np.where(keep, new[rows], rng.choice([-1, -7, 10 ** 9], (T, K)))
    row_token = np.full(len(order) + extra, -1)
    for t in range(T):
        row_token[token_rows[t][keep[t]]] = t
    t32 = lambda a: torch.tensor(a, dtype=torch.int32)  # noqa: E731
    return t32(token_rows), t32(row_token)


def bits(t):
    return t.contiguous().view(torch.uint8).cpu()


def data(seed, rows, n, dtype, pitch=None, shift=0):
    """[rows][n] on the GPU inside a wider buffer, `shift` elements from its start."""
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(rows, (pitch or n) + shift, generator=g).to(TYPES[dtype])
    return wide.cuda()[:, shift:shift + n]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,n,pitch,shift", [
    (1, 1, 1, None, 0), (1, 8, 6144, None, 0), (3, 2, 7, None, 0), (5, 4, 64, 80, 0), (9, 3, 33, 48, 16),
    (4, 3, 100, 104, 8), (6, 2, 257, None, 0), (17, 5, 2050, 2064, 3), (70, 6, 1100, 1104, 2)])
def test_dispatch_copies_rows(T, K, n, pitch, shift, dtype):
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"dispatch {T} x {n} top-{K} {dtype} pitch={pitch} shift={shift}")
    _, row_token = maps(T + n, T, K, extra=2)
    row_token[-1] = T  # behind the last token
    x = data(n, T, n, dtype, pitch, shift)
    out = torch.zeros(len(row_token), n + 3, dtype=TYPES[dtype], device="cuda")
    out.view(torch.uint8).fill_(0x41)
    m.dispatch(x, row_token.cuda(), out=out[:, :n])
    got, want = out.cpu(), x.cpu()
    for r, t in enumerate(row_token.tolist()):
        if 0 <= t < T:
            assert torch.equal(bits(got[r, :n]), bits(want[t])), r
        else:
            assert not bits(got[r, :n]).any(), r
    assert (bits(got[:, n:]) == 0x41).all()
    assert torch.equal(bits(m.dispatch(x, row_token.cuda())), bits(got[:, :n]))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,K,n,pitch,shift,drop", [
    (1, 1, 1, None, 0, 0), (1, 8, 6144, None, 0, 0.3), (5, 4, 64, 80, 0, 0.9), (9, 3, 33, 48, 16, 0),
    (4, 10, 100, 104, 4, 0.2), (17, 5, 2050, 2064, 3, 0.1), (33, 6, 1100, 1104, 2, 0)])
def test_dispatch_backward_sums_rows(T, K, n, pitch, shift, drop, dtype):
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"dispatch_backward {T} x {n} top-{K} {dtype} pitch={pitch} shift={shift} drop={drop}")
    token_rows, row_token = maps(T + n, T, K, drop)
    M = len(row_token)
    dy = data(n + 1, M, n, dtype, pitch, shift)
    out = torch.full((T, n + 5), 7.0, dtype=ref.DT[dtype], device="cuda")
    m.dispatch_backward(dy, token_rows.cuda(), out=out[:, :n])
    y = dy.cpu().double()
    want, size = torch.zeros(T, n, dtype=torch.float64), torch.zeros(T, n, dtype=torch.float64)
    for t in range(T):
        for r in token_rows[t].tolist():
            if 0 <= r < M:
                want[t] += y[r]
                size[t] += y[r].abs()
    ref.check(out[:, :n], want, K * ref.U * size)
    assert (out[:, n:] == 7).all()


def test_a_dropped_slot_takes_nothing_from_other_rows():
    """NaN and infinities in rows that a token does not name; a token without rows is 0."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    dy = torch.full((4, 40), float("nan"), device="cuda")
    dy[2] = 1.5
    token_rows = torch.tensor([[2, -1], [-1, 4], [2, 2]], dtype=torch.int32, device="cuda")
    out = m.dispatch_backward(dy, token_rows)
    assert (out[0] == 1.5).all() and (out[1] == 0).all() and (out[2] == 3).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,K,n,pad,drop,extra", [
    (1, 1, 16, 0, 0, 0), (1, 8, 6144, 0, 0, 0), (3, 2, 48, 8, 0, 1), (7, 10, 1024, 0, 0.3, 70), (5, 32, 1040, 16, 0, 0),
    (20, 6, 8208, 0, 0.2, 3), (2, 3, 13008, 0, 0, 0)])
def test_combine_backward(T, K, n, pad, drop, extra, dtype):
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"combine_backward {T} x {n} top-{K} {dtype} pad={pad} drop={drop} extra={extra}")
    token_rows, row_token = maps(T + n, T, K, drop, extra)
    M = len(row_token)
    dout, rows = data(1, T, n, dtype, n + pad), data(2, M, n, "bf16", n + pad)
    w = torch.randn(T, K, generator=torch.Generator().manual_seed(3)).cuda()
    drows = torch.full((M, n + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((T, K), 9.0, device="cuda")
    m.combine_backward(dout, rows, token_rows.cuda(), w, row_token.cuda(), drows[:, :n], dw)
    g, r64, wf = dout.cpu().float(), rows.cpu().double(), w.cpu()
    want = torch.zeros(M, n, dtype=torch.bfloat16)
    dw64, size = torch.zeros(T, K, dtype=torch.float64), torch.zeros(T, K, dtype=torch.float64)
    for t in range(T):
        for s, r in enumerate(token_rows[t].tolist()):
            if 0 <= r < M:
                want[r] = (wf[t, s] * g[t]).to(torch.bfloat16)
                dw64[t, s] = r64[r] @ g[t].double()
                size[t, s] = r64[r].abs() @ g[t].double().abs()
    assert torch.equal(bits(drows[:, :n]), bits(want))
    assert (drows[:, n:] == 9).all()
    ref.check(dw, dw64, (n + 2) * ref.U * size)
    # Without the rows' tokens: a new result is whole all the same, a given one keeps what no slot names.
    new, dw2 = m.combine_backward(dout, rows, token_rows.cuda(), w)
    assert torch.equal(bits(new), bits(want)) and torch.equal(dw, dw2)
    kept = torch.full((M, n), 9.0, dtype=torch.bfloat16, device="cuda")
    m.combine_backward(dout, rows, token_rows.cuda(), w, drows=kept)
    named = torch.zeros(M, dtype=torch.bool)
    named[[r for r in token_rows.flatten().tolist() if 0 <= r < M]] = True
    assert torch.equal(kept.cpu()[named], want[named]) and (kept.cpu()[~named] == 9).all()


def test_empty_calls():
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.randn(3, 32, device="cuda")
    assert m.dispatch(x, i(0)).shape == (0, 32)
    assert (m.dispatch(x[:0], i(4)) == 0).all()
    assert m.dispatch_backward(x, i(0, 2)).shape == (0, 32)
    assert (m.dispatch_backward(x[:0], i(2, 2)) == 0).all()
    b = x.bfloat16()
    dr, dw = m.combine_backward(x[:0], b, i(0, 2), x.new_zeros(0, 2), row_token=i(3))
    assert dr.shape == (3, 32) and (dr == 0).all() and dw.shape == (0, 2)
    dr, dw = m.combine_backward(x, b[:0], i(3, 2), x.new_ones(3, 2), row_token=i(0))
    assert dr.shape == (0, 32) and (dw == 0).all()


@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_there_and_back_against_autograd(drop):
    """dispatch and combine as one function of the tokens and the weights: the kernels' gradients
    against autograd in 64 bits, and that against central differences."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    T, K, n = 6, 3, 64
    token_rows, row_token = maps(4, T, K, drop)
    M = len(row_token)
    g = torch.Generator().manual_seed(0)
    x = torch.randn(T, n, generator=g).bfloat16()
    w = torch.rand(T, K, generator=g)
    dout = torch.randn(T, n, generator=g)
    here = (token_rows >= 0) & (token_rows < M)
    at = token_rows.clamp(0, M - 1).long()

    def f(x, w):
        rows = x[row_token.long()]
        return ((rows[at] * (w * here)[:, :, None]).sum(1) * dout.double()).sum()

    x64, w64 = x.double().requires_grad_(), w.double().requires_grad_()
    gx, gw = torch.autograd.grad(f(x64, w64), (x64, w64))
    with torch.no_grad():
        for at_x, at_w in (((2, 5), (1, 0)), ((5, 63), (5, 2))):
            for t, where, grad, h in ((x64, at_x, gx, 1e-3), (w64, at_w, gw, 1e-3)):
                old = float(t[where])
                t[where] = old + h
                up = float(f(x64, w64))
                t[where] = old - h
                down = float(f(x64, w64))
                t[where] = old
                # f is linear in each: only rounding of f's sum is left.
                assert abs((up - down) / (2 * h) - float(grad[where])) < 1e-9
    rows = m.dispatch(x.cuda(), row_token.cuda())
    drows, dw = m.combine_backward(dout.cuda(), rows, token_rows.cuda(), w.cuda(), row_token.cuda())
    dx = m.dispatch_backward(drows, token_rows.cuda())
    ref.check(dw, gw, (n + 2) * ref.U * (x.double().abs() @ dout.double().abs().t()).max().expand(T, K))
    # drows is rounded to BF16 (2^-9) before it is summed.
    size = ((w * here).double().sum(1)[:, None] * dout.double().abs())
    ref.check(dx, gx, size * (2.0 ** -8 * 1.01 + (K + 1) * ref.U))


@pytest.mark.parametrize("T,K,n,gap", [
    (4099, 4, 1024, 0), (9001, 5, 1096, 56), (2053, 8, 200, 56), (4099, 3, 1024, 0), (3001, 4, 1021, 0)])
def test_dispatch_of_many_tokens_copies_slice_by_slice(T, K, n, gap):
    """Narrower slices than a row, rows that no slice divides, rows that start inside a line."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"dispatch slices {T} x {n} top-{K} gap={gap}")
    g = torch.Generator().manual_seed(T)
    row_token = torch.randint(-1, T + 1, (K * T,), generator=g, dtype=torch.int32).cuda()
    x = torch.randn(T, n, generator=g).bfloat16().cuda()
    out = torch.full((K * T, n + gap), 3.0, dtype=torch.bfloat16, device="cuda")
    m.dispatch(x, row_token, out=out[:, :n])
    there = (row_token >= 0) & (row_token < T)
    want = torch.where(there[:, None], x[row_token.long().clamp(0, T - 1)], torch.zeros((), dtype=x.dtype, device="cuda"))
    assert torch.equal(out[:, :n].contiguous().view(torch.int16), want.view(torch.int16))
    assert (out[:, n:] == 3).all()


def test_rows_past_32_bit_offsets():
    """4.4 GB of rows, more workgroups than one launch has: every row, and the gradient of rows
    on both sides of the border."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    T, M, n = 1000, 4_300_000, 512
    say(f"dispatch {M} x {n}")
    g = torch.Generator().manual_seed(5)
    row_token = torch.randint(0, T, (M,), generator=g, dtype=torch.int32).cuda()
    x = torch.randn(T, n, generator=g).bfloat16().cuda()
    out = m.dispatch(x, row_token)
    for i in range(0, M, 1 << 20):
        part = slice(i, min(M, i + (1 << 20)))
        assert torch.equal(out[part].view(torch.int16), x[row_token[part].long()].view(torch.int16)), i
    token_rows = torch.tensor([[M - 1, 0], [2_200_000, M], [-1, M - 2]], dtype=torch.int32)
    got = m.dispatch_backward(out, token_rows.cuda()).cpu().float()
    pick = lambda r: out[r].cpu().float()  # noqa: E731
    want = torch.stack([(pick(M - 1) + pick(0)).bfloat16().float(), pick(2_200_000), pick(M - 2)])
    assert torch.equal(got, want)


@pytest.mark.parametrize("T,K,n", [(1030, 3, 48), (258, 9, 1040), (300, 2, 13008), (8200, 4, 2048)])
def test_combine_backward_of_many_tokens(T, K, n):
    """Beyond the few tokens whose rows several groups share; the last with rows read past the cache."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"combine_backward {T} x {n} top-{K}")
    g = torch.Generator().manual_seed(T)
    M = T * K - 5
    token_rows = torch.randperm(T * K, generator=g).to(torch.int32).view(T, K)  # five slots without a row
    rows = torch.randn(M, n, generator=g).bfloat16()
    dout = torch.randn(T, n, generator=g).bfloat16()
    weights = torch.rand(T, K, generator=g)
    drows, dw = m.combine_backward(dout.cuda(), rows.cuda(), token_rows.cuda(), weights.cuda())
    r, here = token_rows.long().clamp(max=M - 1), (token_rows < M)
    prod = rows[r.view(-1)].double() * dout.double().repeat_interleave(K, 0)
    want = torch.where(here, prod.sum(1).view(T, K), 0.0)
    # A sum of n products, each rounded once: at most n roundings of a partial sum each.
    assert ((dw.cpu().double() - want).abs() <= (n + 1) * ref.U * prod.abs().sum(1).view(T, K)).all()
    pair = here.view(-1)
    got = drows.cpu()[r.view(-1)[pair]]
    exact = (weights.view(-1, 1) * dout.float().repeat_interleave(K, 0))[pair].bfloat16()
    assert torch.equal(got, exact)
