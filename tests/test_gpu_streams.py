"""A call with a stream of its own allocates its results and its workspace on that stream,
not from the current stream's pool, whose free blocks may still be in use by work queued there.
Checked by address: nothing here depends on timing."""
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

U8, F32, I32, BF16 = torch.uint8, torch.float32, torch.int32, torch.bfloat16


def _rand(*shape):
    return torch.randint(0x28, 0x40, shape, dtype=U8, device="cuda")


def _gemm(n=64, k=256, E=2, rows=4):
    return dict(a_q=_rand(rows, k // 2), a_sf=_rand(rows, k // 16), a_scale=torch.ones(1, device="cuda"),
                w_q=_rand(E, n, k // 2), w_sf=_rand(E, n, k // 16), w_scale=torch.ones(E, device="cuda"),
                offsets=torch.tensor([0, 1, rows], dtype=I32, device="cuda"))


def _layer(T=3, E=5, K=2, H=128, I=64):
    return dict(x=torch.randn(T, H, device="cuda").bfloat16(), ids=torch.randint(0, E, (T, K), dtype=I32, device="cuda"),
                weights=torch.rand(T, K, device="cuda"), w13_q=_rand(E, 2 * I, H // 2), w13_sf=_rand(E, 2 * I, H // 16),
                w13_scale=torch.full((E,), 0.05, device="cuda"), w2_q=_rand(E, H, I // 2),
                w2_sf=_rand(E, H, I // 16), w2_scale=torch.full((E,), 0.05, device="cuda"))


# name: (arguments, the C entry point and which of its arguments is the workspace)
CALLS = {
    "quantize": (lambda: dict(x=torch.randn(4, 64, device="cuda")), None),
    "pack_weights": (lambda: dict(w_q=_gemm()["w_q"]), None),
    "unpack_weights": (lambda: dict(w_packed=_gemm()["w_q"]), None),
    "grouped_gemm": (_gemm, None),
    "grouped_gemm_swiglu": (lambda: dict(_gemm(), h_scale=torch.ones(1, device="cuda")), None),
    "combine": (lambda: dict(rows=torch.randn(6, 64, device="cuda").bfloat16(),
                             token_rows=torch.randint(0, 6, (3, 2), dtype=I32, device="cuda"),
                             token_weights=torch.rand(3, 2, device="cuda")), None),
    "linear": (lambda: dict(x=torch.randn(3, 128, device="cuda").bfloat16(), w_q=_rand(48, 64), w_sf=_rand(48, 8),
                            w_scale=torch.ones(1, device="cuda")), None),
    "moe_ffn": (_layer, ("moe_fp4_ffn", -3)),
    "route": (lambda: dict(logits=torch.randn(100, 16, device="cuda"), topk=3), ("moe_fp4_route", -3)),
}


def _stream_of(address):
    """The stream whose pool holds this address."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= address < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment holds the address")


@pytest.mark.parametrize("name", CALLS)
def test_new_tensors_belong_to_the_launch_stream(name, monkeypatch):
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    make, ws = CALLS[name]
    args = make()
    lib, seen = m.lib(), []

    class Spy:
        def __getattr__(self, attr):
            fn = getattr(lib, attr)
            if ws is None or attr != ws[0]:
                return fn

            def call(*a):
                seen.append(a[ws[1]])
                return fn(*a)
            return call

    monkeypatch.setattr(m, "_lib", Spy())
    side = torch.cuda.Stream()
    # Blocks of every small size, free in the current stream's pool but as good as in use:
    # what the call would be given if it asked there.
    free = [torch.empty(256 << i, dtype=U8, device="cuda") for i in range(8) for _ in range(4)]
    spans = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in free]
    side.wait_stream(torch.cuda.current_stream())
    del free
    got = getattr(m, name)(**args, stream=side)
    side.synchronize()
    outs = [t.data_ptr() for t in (got if isinstance(got, tuple) else (got,))]
    assert len(seen) == (ws is not None)
    for p in outs + seen:
        assert not any(a <= p < b for a, b in spans)
        assert _stream_of(p) == side.cuda_stream
    # On the current stream the results stay in its pool.
    got = getattr(m, name)(**args)
    for t in got if isinstance(got, tuple) else (got,):
        assert _stream_of(t.data_ptr()) == torch.cuda.current_stream().cuda_stream
