"""The binding's short host path: it is what plain calls take, gives the same bits as the
Python path (a call with an explicit stream), keeps given outputs, and leaves every
refusal to the Python path, which names what is wrong."""
import gc

import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

U8, F32, I32, BF16 = torch.uint8, torch.float32, torch.int32, torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _m():
    from block_scaled_fp4_05_amd import moe_fp4
    return moe_fp4


def _rand(*shape):
    return torch.randint(0x28, 0x40, shape, dtype=U8, device="cuda")


def _linear():
    return dict(x=torch.randn(3, 128, device="cuda").bfloat16(), w_q=_rand(48, 64), w_sf=_rand(48, 8),
                w_scale=torch.full((1,), 0.1, device="cuda"))


def _ffn():
    T, E, K, H, I = 3, 5, 2, 128, 64
    return dict(x=torch.randn(T, H, device="cuda").half(), ids=torch.randint(0, E, (T, K), dtype=I32, device="cuda"),
                weights=torch.rand(T, K, device="cuda"), w13_q=_rand(E, 2 * I, H // 2), w13_sf=_rand(E, 2 * I, H // 16),
                w13_scale=torch.full((E,), 0.05, device="cuda"), w2_q=_rand(E, H, I // 2),
                w2_sf=_rand(E, H, I // 16), w2_scale=torch.full((E,), 0.05, device="cuda"))


def _taken(name, args, monkeypatch):
    """The call's result, and that the short path gave it."""
    m = _m()
    assert m._calls is not None
    seen = []
    real = getattr(m._calls, name)

    class Spy:
        def __getattr__(self, attr):
            def call(*a):
                seen.append(real(*a) if attr == name else getattr(real, attr)(*a))
                return seen[-1]
            return call

    with monkeypatch.context() as mp:
        mp.setattr(m, "_calls", Spy())
        out = getattr(m, {"ffn": "moe_ffn"}.get(name, name))(**args)
    assert len(seen) == 1
    return out, seen[0]


def test_plain_calls_take_the_short_path(monkeypatch):
    m, here = _m(), torch.cuda.current_stream()
    res = torch.randn(3, 48, device="cuda").bfloat16()
    for extra in ({}, dict(residual=res), dict(out_dtype=F32), dict(swiglu=True), dict(out=torch.empty_like(res))):
        a = dict(_linear(), **extra)
        got, seen = _taken("linear", a, monkeypatch)
        assert got is seen
        b = dict(a, out=torch.empty_like(res)) if "out" in a else a
        assert torch.equal(got, m.linear(**b, stream=here))
        assert "out" not in a or got is a["out"]
    for extra in ({}, dict(residual=torch.randn(3, 128, device="cuda").half()), dict(out_dtype=F32)):
        a = dict(_ffn(), **extra)
        got, seen = _taken("ffn", a, monkeypatch)
        assert got is seen and torch.equal(got, m.moe_ffn(**a, stream=here))
    for T in (3, 100):
        for extra in ({}, dict(score="sigmoid", bias=torch.rand(16, device="cuda"), num_groups=4, topk_groups=2,
                               renormalize=False)):
            a = dict(logits=torch.randn(T, 16, device="cuda"), topk=3, **extra)
            got, seen = _taken("route", a, monkeypatch)
            assert isinstance(got, m.Routing) and seen is not None
            for p, q in zip(got, m.route(**a, stream=here)):
                assert p.dtype == q.dtype and torch.equal(p, q)


@pytest.mark.parametrize("change,message", [
    (dict(x=torch.zeros(3, 128)), "must be a CUDA tensor|x: expected"), (dict(w_q=torch.zeros(48, 64, dtype=U8)), "CUDA"),
    (dict(w_sf="no"), "w_sf"), (dict(w_scale=None), "w_scale"), (dict(residual=torch.zeros(3, 47, dtype=BF16)), "residual"),
    (dict(out_dtype=torch.float64), "out_dtype"), (dict(out=torch.zeros(3, 48, dtype=torch.float64)), "out"),
])
def test_linear_refusals_on_the_gpu(change, message):
    with pytest.raises(ValueError, match=message):
        _m().linear(**dict(_linear(), **change))


def test_refusals_of_the_library_on_the_gpu():
    m = _m()
    a = _linear()
    with pytest.raises(m.MoeFp4Error):  # K of 16
        m.linear(a["x"][:, :16].contiguous(), a["w_q"][:, :8].contiguous(), a["w_sf"][:, :1].contiguous(), a["w_scale"])
    with pytest.raises(ValueError, match="unit column stride"):
        m.linear(**dict(a, x=torch.zeros(128, 3, dtype=BF16, device="cuda").t()))
    with pytest.raises(m.MoeFp4Error):  # the output is the input
        m.linear(a["x"], _rand(128, 64), _rand(128, 8), a["w_scale"], out=a["x"])
    f = _ffn()
    with pytest.raises(ValueError, match="ids: dtype"):
        m.moe_ffn(**dict(f, ids=f["ids"].long()))
    with pytest.raises(ValueError, match="w2_sf: shape"):
        m.moe_ffn(**dict(f, w2_sf=f["w2_sf"][:, :, :1].contiguous()))
    with pytest.raises(m.MoeFp4Error):
        m.route(torch.zeros(3, 8, device="cuda"), 9)
    with pytest.raises(ValueError, match="bias: dtype"):
        m.route(torch.zeros(3, 8, device="cuda"), 2, score="sigmoid", bias=torch.zeros(8, device="cuda").half())


def test_more_tokens_than_the_layer_takes_are_refused_as_such():
    m, f = _m(), _ffn()
    many = dict(f, x=torch.zeros(65, 128, device="cuda").half(), weights=torch.zeros(65, 2, device="cuda"),
                ids=torch.zeros(65, 2, dtype=I32, device="cuda"))
    with pytest.raises(m.MoeFp4Error) as e:
        m.moe_ffn(**many)
    assert e.value.status == m.ERR_UNSUPPORTED


def test_short_path_keeps_no_references():
    m = _m()
    a, f, x = _linear(), _ffn(), torch.randn(100, 16, device="cuda")

    def calls():
        out = torch.empty(3, 48, dtype=BF16, device="cuda")
        m.linear(**a), m.linear(**a, out=out), m.moe_ffn(**f), m.route(x, 3)

    calls()
    gc.collect()
    before = torch.cuda.memory_allocated()
    for _ in range(50):
        calls()
    gc.collect()
    assert torch.cuda.memory_allocated() == before


def test_route_results_do_not_share_elements():
    """The five results of one call lie in one allocation: apart, aligned, and good for
    views, in-place operations and the library's other calls."""
    m = _m()
    r = m.route(torch.randn(37, 21, device="cuda"), 5)
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * 4) for t in r)
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
    assert all(t.data_ptr() % 256 == 0 and t.is_contiguous() for t in r)
    keep = [t.clone() for t in r]
    for i, t in enumerate(r):
        t.fill_(3)
        assert all(torch.equal(u, v) for u, v in zip(r[i + 1:], keep[i + 1:]))
    assert r.weights.view(-1)[2:].sum() == 3 * (37 * 5 - 2) and r.ids.t().contiguous().shape == (5, 37)
    del keep, t
    ids = r.ids
    del r
    torch.empty(1000, device="cuda").zero_()
    assert (ids == 3).all()
