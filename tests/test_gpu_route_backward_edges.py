"""The router's gradient where its formulas have no value or an edge: NaN and infinities among the
chosen logits and beside them, for every score."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
from gpu_util import require_gpu, say
from test_gpu_route_backward import KINDS, inputs

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("score,renorm", KINDS)
@pytest.mark.parametrize("E,K", [(12, 3), (300, 20)])  # 16 and 64 lanes a token
def test_logits_without_a_value(E, K, score, renorm):
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"route_backward edges {E} top-{K} {score} renorm={renorm}")
    x, ids, d = inputs(E, 10, E, K, "fp32")
    beside = [int(next(e for e in range(E) if e not in ids[t])) for t in range(10)]
    x[1, ids[1, 1]] = NAN
    x[2, ids[2, 0]] = INF
    x[3, ids[3]] = -INF
    x[4, ids[4, 1:]] = -INF
    x[5, beside[5]] = NAN
    x[6, beside[6]] = INF
    x[7] = -INF
    x[8, beside[8]] = -INF
    out = m.route_backward(x.cuda(), ids.int().cuda(), d.cuda(), score, renorm).cpu()

    nan = torch.zeros(10, E, dtype=torch.bool)
    if score == "softmax" and not renorm:
        nan[[1, 2, 5, 6, 7]] = True  # every logit is in every score
    else:
        for t in (1, 2, 3, 7) if score == "softmax" else (1, 3, 7) if renorm else ():
            nan[t, ids[t]] = True
        if score == "sigmoid" and not renorm:
            nan[1, ids[1, 1]] = True
    assert torch.equal(out.isnan(), nan)

    # The others by the formulas in 64 bits; an infinity by a number as far as matters there.
    near = torch.nan_to_num(x.double(), nan=0.0, posinf=800.0, neginf=-800.0)
    y, b = ref.route_backward(near, ids, d.double(), score, renorm)
    if score == "sigmoid":  # (the bound of a far logit's score counts its steps, 0 is 0)
        b = torch.where(x.isfinite(), b, torch.zeros_like(b))
    there = ~nan
    for t in (1, 5, 6, 7):
        there[t, x[t].isnan()] = False
    ref.check(out[there], y[there], b[there])
