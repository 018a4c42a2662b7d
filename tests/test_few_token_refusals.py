"""What the few-token entry points and the router refuse, on the CPU: the C ABI's status for
every kind of bad argument (fake pointers: nothing is launched) and the binding's errors."""
import pytest
import torch

from block_scaled_fp4_05_amd import moe_fp4 as m

OK, NULL, SHAPE, ALIGN, UNSUPPORTED, _, ARG = range(7)
U8, F32, I32, BF16 = torch.uint8, torch.float32, torch.int32, torch.bfloat16


def _at(i):
    return (i + 1) << 36  # far apart: no two buffers overlap


LINEAR = dict(x=_at(0), x_dtype=0, m=3, ld_x=64, w_q=_at(1), w_sf=_at(2), w_scale=_at(3), n=10, k=64,
              swiglu=0, residual=None, ld_res=0, out=_at(4), out_dtype=0, ldo=10, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), NULL), (dict(w_q=None), NULL), (dict(w_sf=None), NULL), (dict(w_scale=None), NULL),
    (dict(out=None), NULL), (dict(m=-1), SHAPE), (dict(n=0), SHAPE), (dict(k=0), SHAPE),
    (dict(ld_x=56), SHAPE), (dict(ldo=9), SHAPE), (dict(residual=_at(5), ld_res=9), SHAPE),
    (dict(swiglu=1, n=9), SHAPE), (dict(swiglu=1, residual=_at(5), ld_res=10), SHAPE),
    (dict(swiglu=2), ARG), (dict(x_dtype=1), ARG), (dict(x_dtype=3), ARG), (dict(out_dtype=3), ARG),
    (dict(x=_at(0) + 8), ALIGN), (dict(ld_x=68), ALIGN), (dict(w_q=_at(1) + 8), ALIGN),
    (dict(w_sf=_at(2) + 2), ALIGN), (dict(w_scale=_at(3) + 2), ALIGN), (dict(out=_at(4) + 1), ALIGN),
    (dict(out=_at(4) + 2, out_dtype=1), ALIGN), (dict(residual=_at(5) + 1, ld_res=10), ALIGN),
    (dict(k=72, ld_x=72), UNSUPPORTED), (dict(k=48), UNSUPPORTED),
    (dict(n=2 ** 26, ldo=2 ** 26), UNSUPPORTED), (dict(m=16 * 65535 + 1), UNSUPPORTED),
    (dict(ld_x=2 ** 29), UNSUPPORTED), (dict(out=_at(0)), ARG), (dict(out=_at(1) + 16), ARG),
    (dict(out=_at(2) + 4), ARG), (dict(residual=_at(4) + 2, ld_res=10), ARG),
    (dict(residual=_at(4), ld_res=12), ARG), (dict(residual=_at(4), ld_res=10, out_dtype=1), ARG),
    (dict(m=0, x=None, out=None), OK),
])
def test_linear_refuses(change, status):
    assert m.linear_raw(*dict(LINEAR, **change).values()) == status


FFN = dict(x=_at(0), x_dtype=0, tokens=3, ld_x=64, ids=_at(1), weights=_at(2), topk=2, w13_q=_at(3),
           w13_sf=_at(4), w13_scale=_at(5), w2_q=_at(6), w2_sf=_at(7), w2_scale=_at(8), num_experts=4,
           hidden=64, inter=80, residual=None, ld_res=0, out=_at(9), out_dtype=0, ldo=64,
           workspace=_at(10), workspace_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("change,status", [
    *[({nm: None}, NULL) for nm in ("x", "ids", "weights", "w13_q", "w13_sf", "w13_scale", "w2_q", "w2_sf",
                                    "w2_scale", "out", "workspace")],
    (dict(tokens=-1), SHAPE), (dict(topk=0), SHAPE), (dict(num_experts=0), SHAPE), (dict(hidden=0), SHAPE),
    (dict(inter=0), SHAPE), (dict(ld_x=56), SHAPE), (dict(ldo=63), SHAPE),
    (dict(residual=_at(11), ld_res=63), SHAPE), (dict(workspace_bytes=64), SHAPE),
    (dict(x_dtype=1), ARG), (dict(out_dtype=5), ARG),
    *[({nm: FFN[nm] + 8}, ALIGN) for nm in ("x", "w13_q", "w2_q", "workspace")],
    *[({nm: FFN[nm] + 2}, ALIGN) for nm in ("ids", "weights", "w13_sf", "w13_scale", "w2_sf", "w2_scale")],
    (dict(ld_x=65), ALIGN), (dict(out=_at(9) + 1), ALIGN),
    (dict(tokens=65), UNSUPPORTED), (dict(topk=700), UNSUPPORTED), (dict(num_experts=8193), UNSUPPORTED),
    (dict(hidden=72, ld_x=72, ldo=72), UNSUPPORTED), (dict(inter=48), UNSUPPORTED),
    (dict(hidden=2 ** 16, ld_x=2 ** 16, ldo=2 ** 16, inter=2 ** 15), UNSUPPORTED),
    *[(dict(out=FFN[nm]), ARG) for nm in ("x", "ids", "weights", "w13_q", "w2_sf", "workspace")],
    *[(dict(workspace=FFN[nm]), ARG) for nm in ("x", "ids", "w13_q", "w2_q", "w2_scale")],
    (dict(residual=_at(9) + 2, ld_res=64), ARG), (dict(residual=_at(10), ld_res=64), ARG),
    # The residual may be the output, but not while an input is that buffer too.
    *[(dict(residual=_at(9), ld_res=64, out=_at(9), **{nm: _at(9)}), ARG)
      for nm in ("x", "ids", "weights", "w13_q", "w13_sf", "w13_scale", "w2_q", "w2_sf", "w2_scale")],
    (dict(residual=_at(0), ld_res=64, out=_at(0), workspace=_at(0)), ARG),
    (dict(tokens=0, x=None, ids=None, weights=None, out=None, workspace=None, workspace_bytes=0), OK),
])
def test_ffn_refuses(change, status):
    assert m.ffn_raw(*dict(FFN, **change).values()) == status


@pytest.mark.parametrize("change", [dict(tokens=65), dict(topk=700), dict(tokens=64, topk=33),
                                    dict(inter=2 ** 20, topk=600)])
def test_ffn_names_a_size_it_does_not_run_before_the_workspace_that_has_none(change):
    """ffn_workspace_size is 0 for these: a caller that allocates it passes NULL."""
    a = dict(FFN, **change)
    assert m.ffn_workspace_size(a["tokens"], a["topk"], a["num_experts"], a["inter"]) == 0
    assert m.ffn_raw(*dict(a, workspace=None, workspace_bytes=0).values()) == UNSUPPORTED


def test_ffn_workspace_size():
    # The count, a 16-byte record per expert in use, and 4 bytes for each intermediate value.
    assert m.ffn_workspace_size(3, 2, 4, 80) == 16 + 16 * 4 + 6 * 80 * 4
    assert m.ffn_workspace_size(1, 8, 256, 256) == 16 + 16 * 8 + 8 * 256 * 4
    for bad in [(0, 1, 1, 64), (65, 1, 1, 64), (64, 33, 8, 64), (1, 0, 1, 64), (1, 1, 0, 64), (64, 32, 8, 2 ** 20)]:
        assert m.ffn_workspace_size(*bad) == 0


ROUTE = dict(logits=_at(0), dtype=1, tokens=100, num_experts=64, ld=64, score=1, bias=None, renormalize=1,
             topk=4, num_groups=8, topk_groups=2, ids=_at(1), weights=_at(2), offsets=_at(3),
             row_token=_at(4), token_rows=_at(5), workspace=_at(6), workspace_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("change,status", [
    *[({nm: None}, NULL) for nm in ("logits", "ids", "weights", "offsets", "row_token", "token_rows", "workspace")],
    (dict(tokens=-1), SHAPE), (dict(num_experts=0), SHAPE), (dict(ld=63), SHAPE), (dict(topk=0), SHAPE),
    (dict(topk=17), SHAPE), (dict(num_groups=0), SHAPE), (dict(num_groups=7), SHAPE),
    (dict(topk_groups=0), SHAPE), (dict(topk_groups=9), SHAPE), (dict(workspace_bytes=3199), SHAPE),
    (dict(dtype=3), ARG), (dict(score=2), ARG), (dict(renormalize=2), ARG), (dict(score=0, bias=_at(7)), ARG),
    *[({nm: ROUTE[nm] + 2}, ALIGN) for nm in ("logits", "ids", "weights", "offsets", "row_token", "token_rows")],
    (dict(workspace=_at(6) + 8), ALIGN), (dict(bias=_at(7) + 2), ALIGN),
    (dict(num_experts=1032, ld=1032), UNSUPPORTED), (dict(topk=33, topk_groups=8), UNSUPPORTED),
    (dict(num_experts=1024, ld=1024, num_groups=128), UNSUPPORTED),
    (dict(num_experts=680, ld=680, num_groups=40), UNSUPPORTED),  # 17 experts for a group's one lane
    (dict(ld=2 ** 27), UNSUPPORTED), (dict(tokens=2 ** 30), UNSUPPORTED),
    (dict(ids=_at(0)), ARG), (dict(token_rows=_at(1)), ARG), (dict(offsets=_at(2)), ARG),
    (dict(workspace=_at(4)), ARG), (dict(bias=_at(7), weights=_at(7)), ARG),
])
def test_route_refuses(change, status):
    assert m.route_raw(*dict(ROUTE, **change).values()) == status


def test_route_workspace_size():
    assert m.route_workspace_size(64, 256) == 0
    assert m.route_workspace_size(512, 256) == 128 * 256 * 2
    assert m.route_workspace_size(16384, 60) == 256 * 64 * 2


def _linear(**change):
    a = dict(x=torch.zeros(3, 64, dtype=BF16), w_q=torch.zeros(10, 32, dtype=U8),
             w_sf=torch.zeros(10, 4, dtype=U8), w_scale=torch.ones(1))
    return m.linear(**dict(a, **change))


@pytest.mark.parametrize("change,message", [
    (dict(x=torch.zeros(3, 64)), "x: expected a 2-D bfloat16"),
    (dict(x=torch.zeros(64, dtype=BF16)), "x: expected a 2-D bfloat16"),
    (dict(x=torch.zeros(64, 3, dtype=BF16).t()), "x: rows must have unit column stride"),
    (dict(x=torch.zeros(3, 80, dtype=BF16)), "w_q: shape"),
    (dict(w_q=torch.zeros(10, 32, dtype=torch.int8)), "w_q: dtype"),
    (dict(w_q=torch.zeros(10, 64, dtype=U8)[:, ::2]), "w_q: must be contiguous"),
    (dict(w_sf=torch.zeros(9, 4, dtype=U8)), "w_sf: shape"),
    (dict(w_scale=torch.ones(1, dtype=torch.float64)), "w_scale: dtype"),
    (dict(w_scale=torch.ones(2)), "w_scale: shape"),
    (dict(residual=torch.zeros(3, 9, dtype=BF16)), "residual: shape"),
    (dict(residual=torch.zeros(3, 10)), "residual: dtype"),
    (dict(swiglu=True, residual=torch.zeros(3, 10, dtype=BF16)), "swiglu: needs an even"),
    (dict(out=torch.zeros(3, 9, dtype=BF16)), "out: shape"),
    (dict(out=torch.zeros(10, 3, dtype=BF16).t()), "out: rows must have unit column stride"),
    (dict(out=torch.zeros(3, 10, dtype=torch.float64)), "out: expected a"),
    (dict(out=torch.zeros(3, 10), out_dtype=BF16), "out: expected a torch.bfloat16"),
    (dict(out_dtype=torch.float64), "out_dtype"),
    ({}, "must be a CUDA tensor"),
])
def test_linear_binding_checks_its_tensors(change, message):
    with pytest.raises(ValueError, match=message):
        _linear(**change)


def _ffn(**change):
    E, H, I, T, K = 4, 64, 80, 3, 2
    a = dict(x=torch.zeros(T, H, dtype=BF16), ids=torch.zeros(T, K, dtype=I32), weights=torch.zeros(T, K),
             w13_q=torch.zeros(E, 2 * I, H // 2, dtype=U8), w13_sf=torch.zeros(E, 2 * I, H // 16, dtype=U8),
             w13_scale=torch.ones(E), w2_q=torch.zeros(E, H, I // 2, dtype=U8),
             w2_sf=torch.zeros(E, H, I // 16, dtype=U8), w2_scale=torch.ones(E))
    return m.moe_ffn(**dict(a, **change))


@pytest.mark.parametrize("change,message", [
    (dict(x=torch.zeros(3, 64)), "x: expected"),
    (dict(ids=torch.zeros(3, 2, dtype=torch.int64)), "ids: dtype"),
    (dict(ids=torch.zeros(2, 2, dtype=I32)), "ids: shape"),
    (dict(weights=torch.zeros(3, 1)), "weights: shape"),
    (dict(weights=torch.zeros(2, 3).t()), "weights: must be contiguous"),
    (dict(w13_q=torch.zeros(4, 161, 32, dtype=U8)), "even number of rows"),
    (dict(w13_q=torch.zeros(4, 160, 40, dtype=U8)), "w13_q: shape"),
    (dict(w13_sf=torch.zeros(4, 160, 5, dtype=U8)), "w13_sf: shape"),
    (dict(w13_scale=torch.ones(1)), "w13_scale: shape"),
    (dict(w2_q=torch.zeros(4, 64, 32, dtype=U8)), "w2_q: shape"),
    (dict(w2_sf=torch.zeros(4, 64, 4, dtype=U8)), "w2_sf: shape"),
    (dict(w2_scale=torch.ones(4, dtype=torch.float16)), "w2_scale: dtype"),
    (dict(residual=torch.zeros(3, 64)), "residual: dtype"),
    (dict(workspace=torch.zeros(8, dtype=U8)), "workspace: shape"),
    ({}, "must be a CUDA tensor"),
])
def test_ffn_binding_checks_its_tensors(change, message):
    with pytest.raises(ValueError, match=message):
        _ffn(**change)


@pytest.mark.parametrize("args,kw,message", [
    ((torch.zeros(3, 8, dtype=torch.float64), 2), {}, "logits: expected"),
    ((torch.zeros(8), 2), {}, "logits: expected"),
    ((torch.zeros(8, 3).t(), 2), {}, "logits: rows"),
    ((torch.zeros(3, 8), 2), dict(score="top"), "score"),
    ((torch.zeros(3, 8), 0), {}, "topk"),
    ((torch.zeros(3, 8), 2), dict(bias=torch.zeros(7)), "bias: shape"),
    ((torch.zeros(100, 8), 2), dict(workspace=torch.zeros(1, dtype=U8)), "workspace: shape"),
    ((torch.zeros(3, 8), 2), dict(out=m.Routing(*[torch.zeros(3, 2, dtype=I32)] * 5)), "weights: dtype"),
    ((torch.zeros(3, 8), 2), {}, "must be a CUDA tensor"),
])
def test_route_binding_checks_its_tensors(args, kw, message):
    with pytest.raises(ValueError, match=message):
        m.route(*args, **kw)
