"""The FP8 layer's operators together: every step of the example's forward and backward pass against its
64-bit reference on the step's own inputs, the whole pass against autograd in 64 bits, replayed
from a graph, and the memory of new results on a launch stream of their own."""
import os
import sys

import numpy as np
import pytest
import torch

import fp8_ref as ref
from conftest import ROOT
from gpu_util import require_gpu, say
from test_gpu_streams import _stream_of

pytestmark = pytest.mark.gpu

I32, F32 = torch.int32, torch.float32


def layer_and_inputs(T, E, K, H, I, seed=0):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    from fp8_layer import Layer
    g = torch.Generator("cuda").manual_seed(seed)
    make = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return Layer(E, K, H, I, seed), make(T, H).bfloat16(), make(T, E), make(T, H), make(T, H) * 0.1


def dense(q, s):
    return ref.values(q, s, 128)


def grouped(q, s, w, offsets, index=None):
    """(value, bound) of the grouped product for a 16-bit result."""
    a = ref.values(q, s, 1)
    if index is not None:
        a = a[index.cpu().numpy()]
    off = offsets.tolist()
    y = torch.zeros(a.shape[0], w.shape[1], dtype=torch.float64)
    b = torch.zeros_like(y)
    for e in range(w.shape[0]):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            y[lo:hi], b[lo:hi] = ref.product(a[lo:hi], w[e], True)
    return y, b


@pytest.mark.parametrize("T,E,K,H,I", [(1, 8, 2, 128, 64), (37, 12, 3, 272, 144)])
def test_forward_and_backward_step_by_step(T, E, K, H, I):
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"fp8 layer T={T} E={E} K={K} H={H} I={I}")
    layer, x, logits, residual, dy = layer_and_inputs(T, E, K, H, I)
    w13, w2 = dense(*layer.w13[:2]), dense(*layer.w2[:2])
    assert np.array_equal(dense(*layer.w13[2:]), w13.transpose(0, 2, 1))
    y, saved = layer.forward(x, logits, residual)
    _, r, gu, rows = saved
    xq, xs = m.quantize_fp8(x)
    ref.check(gu, *grouped(xq, xs, w13, r.offsets, r.row_token), "gate and up")
    hq, hs = m.quantize_fp8(gu, swiglu=True)
    ref.check_quantized(hq, hs, *ref.swiglu(gu.double().cpu().numpy()), False, "activation")
    ref.check(rows, *grouped(hq, hs, w2, r.offsets), "down")
    picked = rows.double().cpu()[r.token_rows.cpu().long()] * r.weights.double().cpu()[:, :, None]
    ref.check(y, picked.sum(1) + residual.double().cpu(),
              (K + 2) * ref.U * (picked.abs().sum(1) + residual.double().cpu().abs()), "combine")

    dx, dlogits = layer.backward(dy, saved)
    drows, dw = m.combine_backward(dy, rows, r.token_rows, r.weights, row_token=r.row_token)
    flat = r.token_rows.cpu().long().flatten()
    want = (r.weights.cpu()[:, :, None] * dy.cpu()[:, None, :]).reshape(-1, H).bfloat16()
    assert torch.equal(drows.cpu()[flat], want)
    dq, ds = m.quantize_fp8(drows)
    dh = m.grouped_gemm_fp8(dq, ds, *layer.w2[2:], r.offsets)
    ref.check(dh, *grouped(dq, ds, w2.transpose(0, 2, 1), r.offsets), "down's gradient")
    gq, gs = m.quantize_fp8(gu, swiglu=True, grad=dh)
    ref.check_quantized(gq, gs, *ref.swiglu_grad(gu.double().cpu().numpy(), dh.double().cpu().numpy()), False,
                        "activation's gradient")
    dxr = m.grouped_gemm_fp8(gq, gs, *layer.w13[2:], r.offsets)
    ref.check(dxr, *grouped(gq, gs, w13.transpose(0, 2, 1), r.offsets), "gate and up's gradient")
    parts = dxr.double().cpu()[r.token_rows.cpu().long()]
    ref.check(dx, parts.sum(1), K * ref.U * parts.abs().sum(1), "tokens' gradient")
    ref.check(dlogits, *ref.route_backward(logits.double().cpu(), r.ids.cpu().long(), dw.double().cpu(), "softmax", True),
              "gate's gradient")


def test_the_whole_pass_against_autograd():
    """The layer in 64 bits on the same FP8 weights: what separates them are the roundings of tokens,
    activations and gradients to FP8 (at most 2^-4 each, 2.6% in the mean) and BF16; norms within
    15%, the directions within what four such roundings in a row leave."""
    require_gpu()
    T, E, K, H, I = 48, 8, 2, 256, 128
    layer, x, logits, residual, dy = layer_and_inputs(T, E, K, H, I, seed=3)
    y, saved = layer.forward(x, logits, residual)
    dx, dlogits = layer.backward(dy, saved)
    ids = saved[1].ids.cpu().long()
    w13, w2 = (torch.from_numpy(dense(*w[:2])) for w in (layer.w13, layer.w2))
    x64, l64 = x.cpu().double().requires_grad_(), logits.cpu().double().requires_grad_()
    w = torch.softmax(l64.gather(1, ids), 1)
    gu = torch.einsum("tkno,to->tkn", w13[ids], x64)
    h = torch.nn.functional.silu(gu[:, :, :I]) * gu[:, :, I:]
    out = (torch.einsum("tkno,tko->tkn", w2[ids], h) * w[:, :, None]).sum(1) + residual.cpu().double()
    gx, gl = torch.autograd.grad((out * dy.cpu().double()).sum(), (x64, l64))
    for got, want, name in ((y, out.detach(), "y"), (dx, gx, "dx"), (dlogits, gl, "dlogits")):
        g = got.double().cpu()
        assert float((g - want).norm() / want.norm()) < 0.15, name


def test_captured_and_replayed():
    """Forward and backward in one graph, with new inputs before every replay and eager runs in between."""
    require_gpu()
    layer, x, logits, residual, dy = layer_and_inputs(65, 16, 4, 256, 128, seed=5)

    def both():
        y, saved = layer.forward(x, logits, residual)
        return (y, *layer.backward(dy, saved))

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for _ in range(4):
        for t in (x, logits, residual, dy):
            t.copy_(torch.roll(t, 1, 0))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, both()):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    """The same calls on two streams, interleaved: nothing is shared between them."""
    require_gpu()
    sets = [layer_and_inputs(40, 8, 2, 256, 128, seed=s) for s in (1, 2)]

    def run(layer, x, logits, residual, dy):
        y, saved = layer.forward(x, logits, residual)
        return (y, *layer.backward(dy, saved))

    want = [run(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(run(*s))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def _calls():
    f8 = lambda *s: torch.randint(0, 64, s, dtype=torch.uint8, device="cuda").view(ref.FP8)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=I32, device="cuda")  # noqa: E731
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    return {
        "quantize_fp8": dict(x=r(4, 64)),
        "quantize_fp8_weights": dict(w=r(2, 32, 64), transposed=True),
        "grouped_gemm_fp8": dict(a_q=f8(4, 64), a_sf=r(4, 1), w_q=f8(2, 32, 64), w_sf=r(2, 1, 1), offsets=i(3)),
        "linear_fp8": dict(a_q=f8(4, 64), a_sf=r(4, 1), w_q=f8(32, 64), w_sf=r(1, 1)),
        "dispatch": dict(x=r(4, 64), row_token=i(6)),
        "dispatch_backward": dict(dy=r(6, 64), token_rows=i(3, 2)),
        "combine_backward": dict(dout=r(3, 64), rows=r(6, 64).bfloat16(), token_rows=i(3, 2), token_weights=r(3, 2),
                                 row_token=i(6)),
        "route_backward": dict(logits=r(5, 16), ids=i(5, 2), dweights=r(5, 2)),
    }


@pytest.mark.parametrize("name", ["quantize_fp8", "quantize_fp8_weights", "grouped_gemm_fp8", "linear_fp8", "dispatch",
                                  "dispatch_backward", "combine_backward", "route_backward"])
def test_new_results_belong_to_the_launch_stream(name):
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    args = _calls()[name]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, None):
        got = getattr(m, name)(**args, stream=stream)
        side.synchronize()
        for t in got if isinstance(got, tuple) else (got,):
            assert _stream_of(t.data_ptr()) == (stream or torch.cuda.current_stream()).cuda_stream


@pytest.mark.parametrize("name", ["quantize_fp8", "grouped_gemm_fp8", "linear_fp8", "dispatch", "dispatch_backward",
                                  "combine_backward", "route_backward"])
def test_the_short_host_path_and_the_plain_one_agree(name, monkeypatch):
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    args = _calls()[name]
    if name == "grouped_gemm_fp8":
        args["offsets"] = torch.tensor([0, 1, 4], dtype=I32, device="cuda")
    if name == "combine_backward":
        args["token_rows"] = torch.arange(6, dtype=I32, device="cuda").view(3, 2)
        args["row_token"] = torch.tensor([0, 0, 1, 1, 2, 2], dtype=I32, device="cuda")
    assert m.lib() and m._calls is not None
    taken = []
    inner = "gemm_fp8" if "fp8" in name and name != "quantize_fp8" else name

    class Spy:
        def __getattr__(self, attr):
            fn = getattr(real, attr)
            if attr != inner:
                return fn

            def call(*a):
                out = fn(*a)
                taken.append(out is not None)
                return out
            return call

    real = m._calls
    monkeypatch.setattr(m, "_calls", Spy())
    short = getattr(m, name)(**args)
    plain = getattr(m, name)(**args, stream=torch.cuda.current_stream())
    assert taken == [True]
    for a, b in zip(*(v if isinstance(v, tuple) else (v,) for v in (short, plain))):
        assert a.dtype == b.dtype and torch.equal(a.view(torch.uint8), b.view(torch.uint8))
