"""The sizes where the FP8 entry points begin to refuse, as the header gives them (on the CPU: the calls
that are within them are refused for buffers that overlap)."""
from block_scaled_fp4_05_amd import moe_fp4 as m
from test_fp8_refusals import ARG, COMBINE, GEMM, QUANT, UNSUPPORTED, _at


def test_longest_row_and_most_rows():
    one = dict(QUANT, swiglu=0, grad=None, ld_grad=0, rows=1, q=QUANT["x"])
    at = 2 ** 29 - 1024
    assert m.quantize_fp8_raw(*dict(one, k=at, ld_x=at).values()) == UNSUPPORTED
    assert m.quantize_fp8_raw(*dict(one, k=at - 16, ld_x=at - 16).values()) == ARG
    gemm = dict(GEMM, a_row_index=None, n=16, k=16, ldo=16, experts=1, out=_at(0))
    assert m.gemm_fp8_raw(*dict(gemm, m_total=at, a_rows=at).values()) == UNSUPPORTED
    assert m.gemm_fp8_raw(*dict(gemm, m_total=at - 1, a_rows=at - 1).values()) == ARG
    back = dict(COMBINE, drows=COMBINE["rows"])
    most = 2 ** 27 - 257
    assert m.combine_backward_raw(*dict(back, m_total=most + 1).values()) == UNSUPPORTED
    assert m.combine_backward_raw(*dict(back, m_total=most).values()) == ARG
