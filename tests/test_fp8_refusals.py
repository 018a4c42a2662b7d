"""What the FP8 entry points and the gradients refuse, on the CPU: the C ABI's status for every kind of
bad argument (fake pointers: nothing is launched) and the binding's errors."""
import pytest
import torch

from block_scaled_fp4_05_amd import moe_fp4 as m

OK, NULL, SHAPE, ALIGN, UNSUPPORTED, _, ARG = range(7)
F32, I32, BF16, FP8 = torch.float32, torch.int32, torch.bfloat16, torch.float8_e4m3fn


def _at(i):
    return (i + 1) << 40  # far apart: no two buffers overlap


QUANT = dict(x=_at(0), in_dtype=0, rows=5, k=144, ld_x=288, swiglu=1, grad=_at(1), ld_grad=144, pow2=0,
             q=_at(2), sf=_at(3), stream=None)


@pytest.mark.parametrize("change,status", [
    *[({nm: None}, NULL) for nm in ("x", "q", "sf")],
    (dict(rows=-1), SHAPE), (dict(k=0), SHAPE), (dict(k=136), SHAPE), (dict(ld_x=280), SHAPE),
    (dict(ld_grad=136), SHAPE), (dict(swiglu=0, grad=None, ld_x=136), SHAPE), (dict(ld_x=2 ** 61), SHAPE),
    *[({nm: QUANT[nm] + 8}, ALIGN) for nm in ("x", "grad", "q")], (dict(sf=_at(3) + 2), ALIGN),
    (dict(ld_x=292), ALIGN), (dict(ld_grad=148), ALIGN), (dict(in_dtype=1, ld_x=290), ALIGN),
    (dict(in_dtype=3), ARG), (dict(swiglu=2), ARG), (dict(swiglu=0), ARG), (dict(pow2=2), ARG),
    *[({out: QUANT[nm]}, ARG) for out in ("q", "sf") for nm in ("x", "grad")], (dict(sf=_at(2) + 16), ARG),
    (dict(k=2 ** 29), UNSUPPORTED), (dict(rows=2 ** 30), UNSUPPORTED),
    (dict(rows=0, x=None, grad=None, q=None, sf=None), OK),
])
def test_quantize_refuses(change, status):
    assert m.quantize_fp8_raw(*dict(QUANT, **change).values()) == status


WEIGHTS = dict(w=_at(0), in_dtype=0, experts=3, n=144, k=272, pow2=0, q=_at(1), sf=_at(2), qt=_at(3), sft=_at(4),
               stream=None)


@pytest.mark.parametrize("change,status", [
    *[({nm: None}, NULL) for nm in ("w", "q", "sf", "qt", "sft")],
    (dict(experts=0), SHAPE), (dict(n=0), SHAPE), (dict(k=0), SHAPE), (dict(k=264), SHAPE), (dict(n=136), SHAPE),
    *[({nm: WEIGHTS[nm] + 8}, ALIGN) for nm in ("w", "q", "qt")],
    *[({nm: WEIGHTS[nm] + 2}, ALIGN) for nm in ("sf", "sft")],
    (dict(in_dtype=3), ARG), (dict(pow2=-1), ARG),
    *[({nm: _at(0) + 16}, ARG) for nm in ("q", "sf", "qt", "sft")], (dict(qt=_at(1)), ARG), (dict(sft=_at(2)), ARG),
    (dict(experts=8193), UNSUPPORTED), (dict(n=2 ** 16, k=2 ** 15), UNSUPPORTED), (dict(n=128 * 65536, k=16), UNSUPPORTED),
])
def test_quantize_weights_refuses(change, status):
    assert m.quantize_fp8_weights_raw(*dict(WEIGHTS, **change).values()) == status


GEMM = dict(a_q=_at(0), a_sf=_at(1), a_rows=9, a_row_index=_at(2), w_q=_at(3), w_sf=_at(4), offsets=_at(5), experts=4,
            m_total=20, n=50, k=144, out=_at(6), out_dtype=0, ldo=50, stream=None)


@pytest.mark.parametrize("change,status", [
    *[({nm: None}, NULL) for nm in ("a_q", "a_sf", "w_q", "w_sf", "offsets", "out")],
    (dict(experts=0), SHAPE), (dict(m_total=-1), SHAPE), (dict(n=0), SHAPE), (dict(k=0), SHAPE), (dict(ldo=49), SHAPE),
    (dict(a_rows=0), SHAPE), (dict(a_row_index=None), SHAPE), (dict(ldo=2 ** 20 + 1), UNSUPPORTED),
    (dict(a_q=_at(0) + 8), ALIGN), (dict(w_q=_at(3) + 8), ALIGN),
    *[({nm: GEMM[nm] + 2}, ALIGN) for nm in ("a_sf", "a_row_index", "w_sf", "offsets")],
    (dict(out=_at(6) + 1), ALIGN), (dict(out=_at(6) + 2, out_dtype=1), ALIGN),
    (dict(out_dtype=3), ARG), *[(dict(out=GEMM[nm]), ARG) for nm in ("a_q", "a_sf", "a_row_index", "w_q", "w_sf", "offsets")],
    (dict(k=136), UNSUPPORTED), (dict(k=2 ** 23), UNSUPPORTED), (dict(experts=8193), UNSUPPORTED),
    (dict(n=2 ** 25, ldo=2 ** 25), UNSUPPORTED), (dict(a_rows=2 ** 24), UNSUPPORTED), (dict(m_total=2 ** 29), UNSUPPORTED),
    (dict(n=2 ** 20, k=16, ldo=2 ** 20, m_total=2 ** 20), UNSUPPORTED),
    (dict(m_total=0, a_q=None, a_sf=None, out=None, a_rows=0), OK),
    (dict(experts=1, offsets=None, m_total=0), OK),
])
def test_gemm_refuses(change, status):
    assert m.gemm_fp8_raw(*dict(GEMM, **change).values()) == status


DISPATCH = dict(x=_at(0), dtype=0, tokens=4, n=30, ld_x=32, row_token=_at(1), m_total=9, out=_at(2), ldo=30, stream=None)


@pytest.mark.parametrize("change,status", [
    *[({nm: None}, NULL) for nm in ("x", "row_token", "out")],
    (dict(tokens=-1), SHAPE), (dict(m_total=-1), SHAPE), (dict(n=0), SHAPE), (dict(ld_x=29), SHAPE), (dict(ldo=29), SHAPE),
    (dict(ldo=2 ** 61), SHAPE), (dict(x=_at(0) + 1), ALIGN), (dict(out=_at(2) + 1), ALIGN), (dict(row_token=_at(1) + 2), ALIGN),
    (dict(x=_at(0) + 2, dtype=1), ALIGN), (dict(dtype=4), ARG), (dict(out=_at(0)), ARG), (dict(out=_at(1) + 4), ARG),
    (dict(m_total=2 ** 31), UNSUPPORTED), (dict(tokens=2 ** 31), UNSUPPORTED),
    (dict(m_total=0, x=None, row_token=None, out=None), OK),
])
def test_dispatch_refuses(change, status):
    assert m.dispatch_raw(*dict(DISPATCH, **change).values()) == status


BACK = dict(dy=_at(0), dtype=2, m_total=9, n=30, ld_dy=32, token_rows=_at(1), topk=2, tokens=4, dx=_at(2), ld_dx=30,
            stream=None)


@pytest.mark.parametrize("change,status", [
    *[({nm: None}, NULL) for nm in ("dy", "token_rows", "dx")],
    (dict(tokens=-1), SHAPE), (dict(m_total=-1), SHAPE), (dict(n=0), SHAPE), (dict(topk=0), SHAPE), (dict(ld_dy=29), SHAPE),
    (dict(ld_dx=29), SHAPE), (dict(dy=_at(0) + 1), ALIGN), (dict(dx=_at(2) + 1), ALIGN), (dict(token_rows=_at(1) + 2), ALIGN),
    (dict(dtype=3), ARG), (dict(dx=_at(0)), ARG), (dict(dx=_at(1)), ARG), (dict(topk=1025), UNSUPPORTED),
    (dict(m_total=2 ** 31), UNSUPPORTED), (dict(tokens=0, dy=None, token_rows=None, dx=None), OK),
])
def test_dispatch_backward_refuses(change, status):
    assert m.dispatch_backward_raw(*dict(BACK, **change).values()) == status


COMBINE = dict(dout=_at(0), dtype=0, num_tokens=4, n=32, ld_dout=32, rows=_at(1), ld_rows=40, m_total=9, token_rows=_at(2),
               weights=_at(3), topk=2, row_token=_at(4), drows=_at(5), ld_drows=32, dweights=_at(6), stream=None)


@pytest.mark.parametrize("change,status", [
    *[({nm: None}, NULL) for nm in ("dout", "rows", "token_rows", "weights", "drows", "dweights")],
    (dict(num_tokens=-1), SHAPE), (dict(m_total=-1), SHAPE), (dict(n=0), SHAPE), (dict(topk=0), SHAPE),
    (dict(ld_dout=24), SHAPE), (dict(ld_rows=24), SHAPE), (dict(ld_drows=24), SHAPE),
    *[({nm: COMBINE[nm] + 8}, ALIGN) for nm in ("dout", "rows", "drows")],
    *[({nm: COMBINE[nm] + 2}, ALIGN) for nm in ("token_rows", "weights", "row_token", "dweights")],
    (dict(ld_dout=36), ALIGN), (dict(ld_dout=34, dtype=1), ALIGN), (dict(ld_rows=36), ALIGN), (dict(ld_drows=36), ALIGN),
    (dict(dtype=2), ARG), *[(dict(drows=COMBINE[nm]), ARG) for nm in ("dout", "rows", "token_rows", "weights", "row_token")],
    *[(dict(dweights=COMBINE[nm]), ARG) for nm in ("dout", "rows", "token_rows", "weights", "drows")],
    (dict(n=24), UNSUPPORTED), (dict(topk=1025), UNSUPPORTED), (dict(num_tokens=2 ** 23 + 1), UNSUPPORTED),
    (dict(m_total=2 ** 28), UNSUPPORTED),
    (dict(num_tokens=0, row_token=None, dout=None, rows=None, drows=None, token_rows=None, weights=None, dweights=None), OK),
])
def test_combine_backward_refuses(change, status):
    assert m.combine_backward_raw(*dict(COMBINE, **change).values()) == status


ROUTE = dict(logits=_at(0), dtype=0, tokens=4, experts=30, ld=30, ids=_at(1), dweights=_at(2), topk=2, score=1,
             renormalize=1, dlogits=_at(3), ld_out=30, stream=None)


@pytest.mark.parametrize("change,status", [
    *[({nm: None}, NULL) for nm in ("logits", "ids", "dweights", "dlogits")],
    (dict(tokens=-1), SHAPE), (dict(experts=0), SHAPE), (dict(topk=0), SHAPE), (dict(ld=29), SHAPE), (dict(ld_out=29), SHAPE),
    (dict(logits=_at(0) + 1), ALIGN), (dict(dlogits=_at(3) + 2, dtype=1), ALIGN), (dict(ids=_at(1) + 2), ALIGN),
    (dict(dweights=_at(2) + 1), ALIGN), (dict(dtype=3), ARG), (dict(score=2), ARG), (dict(renormalize=3), ARG),
    *[(dict(dlogits=ROUTE[nm]), ARG) for nm in ("logits", "ids", "dweights")],
    (dict(experts=1025, ld=1025, ld_out=1025), UNSUPPORTED), (dict(topk=33), UNSUPPORTED), (dict(tokens=2 ** 24 + 1), UNSUPPORTED),
    (dict(tokens=0, logits=None, ids=None, dweights=None, dlogits=None), OK),
])
def test_route_backward_refuses(change, status):
    assert m.route_backward_raw(*dict(ROUTE, **change).values()) == status


def _z(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=torch.uint8).view(FP8) if dtype is FP8 else torch.zeros(*shape, dtype=dtype)


def _gemm(E=2, n=32, k=144, rows=6):
    return dict(a_q=_z(rows, k, dtype=FP8), a_sf=_z(rows, 2, dtype=F32), w_q=_z(E, n, k, dtype=FP8),
                w_sf=_z(E, 1, 2, dtype=F32), offsets=_z(E + 1, dtype=I32))


@pytest.mark.parametrize("call,message", [
    (lambda: m.quantize_fp8(_z(4, 32, dtype=I32)), "x: expected a 2-D"),
    (lambda: m.quantize_fp8(_z(4, 33), swiglu=True), "even number of columns"),
    (lambda: m.quantize_fp8(_z(4, 32), grad=_z(4, 32)), "grad: only with swiglu"),
    (lambda: m.quantize_fp8(_z(4, 32), swiglu=True, grad=_z(4, 16, dtype=F32)), "grad: dtype"),
    (lambda: m.quantize_fp8(_z(4, 32), swiglu=True, grad=_z(4, 32)), "grad: shape"),
    (lambda: m.quantize_fp8(_z(32, 4).t()), "x: rows must have unit column stride"),
    (lambda: m.quantize_fp8(_z(4, 32), q=_z(4, 32, dtype=torch.uint8)), "q: dtype"),
    (lambda: m.quantize_fp8(_z(4, 144), sf=_z(4, 1, dtype=F32)), "sf: shape"),
    (lambda: m.quantize_fp8(_z(4, 32)), "x: must be a CUDA tensor"),
    (lambda: m.quantize_fp8_weights(_z(32)), "w: expected a 2-D or 3-D"),
    (lambda: m.quantize_fp8_weights(_z(2, 32, 16).transpose(1, 2)), "w: must be contiguous"),
    (lambda: m.quantize_fp8_weights(_z(32, 16)), "w: must be a CUDA tensor"),
    (lambda: m.grouped_gemm_fp8(**dict(_gemm(), w_q=_z(2, 32, 128, dtype=FP8))), "w_q: shape"),
    (lambda: m.grouped_gemm_fp8(**dict(_gemm(), w_q=_z(2, 32, 144, dtype=torch.uint8))), "w_q: expected a 3-D"),
    (lambda: m.grouped_gemm_fp8(**dict(_gemm(), w_sf=_z(2, 2, 2, dtype=F32))), "w_sf: shape"),
    (lambda: m.grouped_gemm_fp8(**dict(_gemm(), a_sf=_z(6, 1, dtype=F32))), "a_sf: shape"),
    (lambda: m.grouped_gemm_fp8(**dict(_gemm(), offsets=_z(2, dtype=I32))), "offsets: shape"),
    (lambda: m.grouped_gemm_fp8(**_gemm(), a_row_index=_z(3, dtype=torch.int64)), "a_row_index: dtype"),
    (lambda: m.grouped_gemm_fp8(**_gemm(), out_dtype=I32), "out_dtype"),
    (lambda: m.grouped_gemm_fp8(**_gemm(), out=_z(5, 32)), "out: shape"),
    (lambda: m.grouped_gemm_fp8(**_gemm()), "must be a CUDA tensor"),
    (lambda: m.linear_fp8(_z(4, 16, dtype=FP8), _z(4, 1, dtype=F32), _z(1, 8, 16, dtype=FP8), _z(1, 1, 1, dtype=F32)), "w_q: expected a 2-D"),
    (lambda: m.dispatch(_z(4, 16, dtype=I32), _z(3, dtype=I32)), "x: expected a 2-D"),
    (lambda: m.dispatch(_z(4, 16), _z(3, dtype=torch.int64)), "row_token: dtype"),
    (lambda: m.dispatch(_z(4, 16), _z(3, dtype=I32), out=_z(2, 16)), "out: shape"),
    (lambda: m.dispatch(_z(4, 16), _z(3, dtype=I32)), "must be a CUDA tensor"),
    (lambda: m.dispatch_backward(_z(4, 16, dtype=FP8), _z(3, 2, dtype=I32)), "dy: expected a 2-D"),
    (lambda: m.dispatch_backward(_z(4, 16), _z(3, dtype=I32)), "token_rows: shape"),
    (lambda: m.dispatch_backward(_z(4, 16), _z(3, 2, dtype=I32), out=_z(3, 16, dtype=F32)), "out: dtype"),
    (lambda: m.combine_backward(_z(3, 16, dtype=torch.float16), _z(4, 16), _z(3, 2, dtype=I32), _z(3, 2, dtype=F32)), "dout: expected"),
    (lambda: m.combine_backward(_z(3, 16), _z(4, 32), _z(3, 2, dtype=I32), _z(3, 2, dtype=F32)), "rows: shape"),
    (lambda: m.combine_backward(_z(3, 16), _z(4, 16), _z(2, 2, dtype=I32), _z(3, 2, dtype=F32)), "token_rows: shape"),
    (lambda: m.combine_backward(_z(3, 16), _z(4, 16), _z(3, 2, dtype=I32), _z(3, 2)), "token_weights: dtype"),
    (lambda: m.combine_backward(_z(3, 16), _z(4, 16), _z(3, 2, dtype=I32), _z(3, 2, dtype=F32), _z(3, dtype=I32)), "row_token: shape"),
    (lambda: m.route_backward(_z(3, 8), _z(3, 2, dtype=torch.int64), _z(3, 2, dtype=F32)), "ids: dtype"),
    (lambda: m.route_backward(_z(3, 8), _z(3, 2, dtype=I32), _z(3, 3, dtype=F32)), "dweights: shape"),
    (lambda: m.route_backward(_z(3, 8), _z(3, 2, dtype=I32), _z(3, 2, dtype=F32), "tanh"), "score"),
    (lambda: m.route_backward(_z(3, 8), _z(3, 2, dtype=I32), _z(3, 2, dtype=F32), out=_z(3, 8, dtype=F32)), "out: dtype"),
    (lambda: m.route_backward(_z(3, 8), _z(3, 2, dtype=I32), _z(3, 2, dtype=F32)), "must be a CUDA tensor"),
])
def test_binding_checks_its_tensors(call, message):
    with pytest.raises(ValueError, match=message):
        call()


def test_expanded_rows_are_refused():
    """A pitch of 0 (rows that are one row): for the library a pitch below its row."""
    x = torch.zeros(1, 32, dtype=BF16).expand(4, 32)
    assert m._pitch(x, "x", BF16, (4, 32)) == 0
    assert m.quantize_fp8_raw(_at(0), 0, 4, 32, 0, 0, None, 0, 0, _at(1), _at(2), None) == SHAPE


def test_quantize_refuses_more_blocks_than_a_launch_has_threads_for():
    """2^29 - 2^17 blocks of 128 and fewer pass the checks (rows of one block at addresses that
    overlap are refused behind that check)."""
    one = dict(QUANT, k=16, ld_x=16, swiglu=0, grad=None, ld_grad=0)
    most = 2 ** 29 - 2 ** 17
    assert m.quantize_fp8_raw(*dict(one, rows=most + 1).values()) == UNSUPPORTED
    assert m.quantize_fp8_raw(*dict(one, rows=most, q=one["x"]).values()) == ARG
