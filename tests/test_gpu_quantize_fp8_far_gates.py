"""SwiGLU modes of the FP8 quantiser where the sigmoid is no normal FP32 number (gates below -87.3),
and infinite gates."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

LEAST = 2.0 ** -126


@pytest.mark.parametrize("k", [16, 144, 8208])
def test_a_sigmoid_below_the_least_normal_number_counts_as_zero(k):
    """Gates from -87 to -104, -1e30 among them, with factors that make the difference visible: the
    value, or 0 where the sigmoid is below 2^-126."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"quantize_fp8 swiglu, gates of -87 to -104, k={k}")
    g = torch.Generator().manual_seed(k)
    gate = -87 - 17 * torch.rand(5, k, generator=g) ** 4
    gate[:, 3::7] = -1e30
    up, d = torch.randn(2, 5, k, generator=g) * 2.0 ** 20
    x = torch.cat((gate, up), 1)
    x64, d64 = x.double().numpy(), d.double().numpy()
    with np.errstate(over="ignore"):
        sigmoid = 1 / (1 + np.exp(-x64[:, :k]))
        zero = sigmoid < LEAST
        # e^87 is off by some 88 steps: at the border it is the one or the other.
        border = np.abs(sigmoid / LEAST - 1) < 100 * ref.U
        for grad in (None, d):
            v, off = ref.swiglu(x64) if grad is None else ref.swiglu_grad(x64, d64)
            hole, either = (z if grad is None else np.concatenate((z, z), 1) for z in (zero, border))
            q, s = m.quantize_fp8(x.cuda(), swiglu=True, grad=None if grad is None else grad.cuda())
            off = off + np.abs(v) * np.where(either, 1.0, 100 * ref.U)
            ref.check_quantized(q, s, np.where(hole, 0.0, v), off, False, f"grad={grad is not None}")


@pytest.mark.parametrize("gate", [np.inf, -np.inf])
def test_an_infinite_gate(gate):
    """An infinity leaves nothing finite in its block; minus infinity times a sigmoid of 0 is a NaN,
    which leaves the others of its block alone."""
    require_gpu()
    from block_scaled_fp4_05_amd import moe_fp4 as m
    say(f"quantize_fp8 swiglu, a gate of {gate}")
    x = torch.randn(3, 512, generator=torch.Generator().manual_seed(1))
    x[1, 130] = gate
    q, s = m.quantize_fp8(x.cuda(), swiglu=True)
    q0, s0 = m.quantize_fp8(torch.nan_to_num(x, posinf=0.0, neginf=0.0).cuda(), swiglu=True)
    values = ref.values(q, s, 1)
    there = torch.ones(3, 256, dtype=torch.bool)
    if gate > 0:
        assert s[1, 1] == np.inf
        there[1, 128:] = False
        s[1, 1] = s0[1, 1]
    else:
        there[1, 130] = False
    assert not np.isfinite(values[~there.numpy()]).any()
    assert torch.equal(q.cpu().view(torch.uint8)[there], q0.cpu().view(torch.uint8)[there])
    assert torch.equal(s, s0)
