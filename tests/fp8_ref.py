"""Plain 64-bit references of the FP8 block-scaled operators and of the rows' and router's
gradients, and the error their kernels may have.  u = 2^-24 is half an FP32 step."""
import numpy as np
import torch

from few_token_ref import DT, U, check, rounding  # noqa: F401  (used by the tests too)

FP8 = torch.float8_e4m3fn
TOP = 448.0
LEAST = np.float32(TOP * 2.0 ** -126)


def blocks(n):
    return -(-n // 128)


def scale32(amax, pow2):
    """The scale of blocks whose largest magnitudes are amax (float32 array): IEEE division."""
    with np.errstate(all="ignore"):
        s = (np.maximum(amax.astype(np.float32), LEAST) / np.float32(TOP)).astype(np.float32)
    if pow2:
        m, e = np.frexp(s)
        s = np.where(np.isfinite(s), np.ldexp(np.float32(1), e - (m == 0.5)), s).astype(np.float32)
    return s


def spread(s, tall, rows, k):
    """Block scales as one per element."""
    return np.repeat(np.repeat(s, tall, -2)[..., :rows, :], 128, -1)[..., :k]


def amax(v, tall):
    """Largest magnitude of each block of tall x 128 (NaN passed over)."""
    rows, k = v.shape[-2:]
    pad = [(0, 0)] * (v.ndim - 2) + [(0, blocks(rows) * 128 - rows if tall > 1 else 0), (0, blocks(k) * 128 - k)]
    a = np.pad(np.abs(np.nan_to_num(v, nan=0.0, posinf=np.inf, neginf=np.inf)), pad)
    a = a.reshape(*v.shape[:-2], a.shape[-2] // tall, tall, a.shape[-1] // 128, 128)
    return a.max((-3, -1))


def quantize(x, tall=1, pow2=False):
    """Codes (uint8) and scales of float32 values, step by step."""
    s = scale32(amax(x, tall), pow2)
    with np.errstate(all="ignore"):
        y = (x / spread(s, tall, *x.shape[-2:])).astype(np.float32)
    y = torch.from_numpy(np.clip(y, -TOP, TOP))  # (clip keeps NaN)
    return y.to(FP8).view(torch.uint8).numpy(), s


def values(q, s, tall):
    """Binary64 values of FP8 codes (tensor or array) with block scales, from the format's definition."""
    q = np.asarray(q.view(torch.uint8).cpu() if isinstance(q, torch.Tensor) else q)
    s = np.asarray(s.cpu() if isinstance(s, torch.Tensor) else s).astype(np.float64)
    e, f = (q >> 3) & 15, (q & 7).astype(np.float64)
    v = np.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e.astype(np.float64) - 7))
    v = np.where((q & 0x7F) == 0x7F, np.nan, v) * np.where(q & 0x80, -1.0, 1.0)
    with np.errstate(invalid="ignore"):  # 0 times an infinite scale
        return v * spread(s, tall, *q.shape[-2:])


def product(a, w, eight_bit=False):
    """(a w^T, bound): FP32 sums in any order of k exact products, each block's sum scaled (two
    roundings) and added; an addition of the matrix cores may be off by a whole step, 2u.
    eight_bit: the FP8 cores, which cut each of eight consecutive products 13 bits below the
    leading bit of the largest; seven of them can lose by it."""
    y, mag = a @ w.T, np.abs(a) @ np.abs(w).T
    m, k = a.shape
    bound = 2 * (k + 3 * blocks(k) + 8) * U * mag
    if eight_bit:
        lost = np.zeros_like(y)
        for j in range(0, k, 8):
            aj, wj = np.abs(a[:, j:j + 8]), np.abs(w[:, j:j + 8])
            top = aj[:, :1] * wj[None, :, 0]
            for i in range(1, aj.shape[1]):
                np.maximum(top, aj[:, i:i + 1] * wj[None, :, i], out=top)
            lost += top
        bound = bound + 7 * 2.0 ** -13 * lost
    return torch.from_numpy(y), torch.from_numpy(bound)


def silu(g):
    return g / (1 + np.exp(-g))


def swiglu(x):
    """(silu(g) u, bound) of binary64 [g | u]: e^-g is off by a few steps, silu by four more
    roundings, the product by one."""
    k = x.shape[1] // 2
    v = silu(x[:, :k]) * x[:, k:]
    return v, np.abs(v) * (np.minimum(np.abs(x[:, :k]), 1) + 10) * U


def swiglu_grad(x, d):
    """([dg | du], bound): the derivative's factor s (1 + g (1 - s)) has terms of up to 1 + |g|
    that partly cancel."""
    k = x.shape[1] // 2
    g, u = x[:, :k], x[:, k:]
    s = 1 / (1 + np.exp(-g))
    dg, du = d * u * s * (1 + g * (1 - s)), d * silu(g)
    off = np.concatenate((np.abs(d * u) * s * (1 + np.abs(g)) * 24, np.abs(du) * 12), 1) * U
    return np.concatenate((dg, du), 1), off


def check_quantized(q, s, v, off, pow2, what=""):
    """Codes and scales of values known to within `off`: the scale of a largest magnitude within its
    bound, every element within half an E4M3 step of its value."""
    q, s = q.cpu(), s.cpu().numpy()
    a = amax(v, 1)
    da = amax(off, 1) * 1.01 + 1e-300
    lo = scale32(np.maximum(a - da, 0) * (1 - 2 * U), pow2)
    hi = scale32((a + da) * (1 + 2 * U), pow2)
    assert ((s >= lo * np.float32(1 - 2 * U)) & (s <= hi * np.float32(1 + 4 * U))).all(), what
    got = values(q, s, 1)
    sw = spread(s.astype(np.float64), 1, *v.shape)
    y = np.abs(v) / sw
    room = sw * np.maximum(y * 2.0 ** -4, 2.0 ** -10) * (1 + 2.0 ** -20) + 1.1 * off
    bad = ~(np.abs(got - v) <= room)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:3], v[bad][:3])


def route_weights(x, ids, score, renorm):
    """The router's weights of binary64 logits with the choice of experts given."""
    chosen = x.gather(1, ids)
    if score == "softmax":
        return torch.softmax(chosen, 1) if renorm else torch.softmax(x, 1).gather(1, ids)
    p = torch.sigmoid(chosen)
    return p / p.sum(1, keepdim=True) if renorm else p


def route_backward(x, ids, d, score, renorm):
    """(gradient, bound) by the formulas, in binary64.  An FP32 score e^(x - m) is off by a few
    steps and |x - m| u, a sum of n terms by n u."""
    T, E = x.shape
    n = ids.shape[1]
    chosen = x.gather(1, ids)
    if score == "softmax" and not renorm:
        p = torch.softmax(x, 1)
        full = torch.zeros_like(x).scatter_add_(1, ids, d)
        size = torch.zeros_like(x).scatter_add_(1, ids, d.abs())
        mean, mag = (p * full).sum(1, keepdim=True), (p * size).sum(1, keepdim=True)
        # (e^-inf is 0 on both sides, with nothing to be off by.)
        r = torch.where(p > 0, x.amax(1, keepdim=True) - x + 2 * E + 16, 0.0) * U
        rm = (p * size * r).sum(1, keepdim=True) + 2 * E * U * mag
        return p * (full - mean), p * (r * (size + mag) + rm + 4 * U * (size + mag) + n * U * size)
    if score == "softmax":
        w, left = torch.softmax(chosen, 1), torch.ones_like(chosen)
        r = (chosen.amax(1, keepdim=True) - chosen + 2 * n + 16) * U
    else:
        p, left = torch.sigmoid(chosen), torch.sigmoid(-chosen)
        low = chosen.clamp(max=0)
        # |x| steps from the exponents' arguments, of e^min(x,0) and of the complement.
        r = (chosen.abs() + low.amax(1, keepdim=True) - low + 2 * n + 24) * U
        if renorm:
            w = torch.exp(low - low.amax(1, keepdim=True)) / (1 + torch.exp(-chosen.abs()))
            w = w / w.sum(1, keepdim=True)
    if score == "sigmoid" and not renorm:
        v, off = p * left * d, (p * left * d).abs() * r
    else:
        mean, mag = (w * d).sum(1, keepdim=True), (w * d.abs()).sum(1, keepdim=True)
        v = w * left * (d - mean)
        off = w * left * (r * (d.abs() + mag) + (w * d.abs() * r).sum(1, keepdim=True) + (2 * n + 4) * U * (d.abs() + mag))
    zero = torch.zeros_like(x)
    # Terms below the smallest normal number lose bits: a few of their steps.
    return zero.scatter_add(1, ids, v), zero.scatter_add(1, ids, off) * (1 + n * U) + 2.0 ** -140
