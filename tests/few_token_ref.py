"""Plain 64-bit references of the few-token operators, and the error their kernels may
have.  u = 2^-24 is half an FP32 step, eps / 2 half a step of the output's type.

A dot product of K exact products summed in FP32 in any order is off by at most
(K + 1) u sum|x w|; every further FP32 operation adds one u."""
import numpy as np
import torch

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(ref, dtype):
    """Largest error of rounding ref (plus its own error, second order) to dtype."""
    t = torch.finfo(dtype)
    return ref.abs() * half_step(dtype) * (1 + 2 ** -6) + t.tiny * t.eps / 2


def weights(rng, shape, lo=0x28, hi=0x40):
    """Random codes and E4M3 block scales (all of [lo, hi), some negative, some zero)."""
    *lead, k = shape
    q = rng.integers(0, 256, (*lead, k // 2), dtype=np.uint8)
    sf = rng.integers(lo, hi, (*lead, k // 16), dtype=np.uint8)
    sf |= (rng.random(sf.shape) < 0.1).astype(np.uint8) << 7
    sf[rng.random(sf.shape) < 0.05] = 0
    return q, sf


def values(q, sf):
    """NVFP4 rows as binary64 (tensor scale apart), from the formats' definitions."""
    mag = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6])
    e, f = (sf >> 3) & 15, (sf & 7).astype(np.float64)
    s = np.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e.astype(np.float64) - 7))
    s = np.where((sf & 0x7F) == 0x7F, np.nan, s) * np.where(sf & 0x80, -1.0, 1.0)
    v = np.empty((*q.shape[:-1], q.shape[-1] * 2))
    v[..., 0::2], v[..., 1::2] = mag[q & 15], mag[q >> 4]
    return torch.from_numpy(v * np.repeat(s, 16, -1))


def dot(x, w, scale):
    """(value, bound) of fl(scale * sum x w) in FP32: x [m][k], w [n][k] binary64."""
    y, mag = x @ w.t() * scale, x.abs() @ w.abs().t() * abs(scale)
    return y, (x.shape[1] + 2) * U * mag


def swiglu(g, dg, u, du):
    """silu(g) * u and its bound, given the bounds of g and u.  |silu'| <= 1.1; the FP32
    exponential of -g is off by a few steps and by |g| steps from its argument."""
    s = g * torch.sigmoid(g)
    ds = 1.1 * dg + s.abs() * (g.abs() + 8) * 2 * U
    return s * u, ds * u.abs() + s.abs() * du + ds * du + (s * u).abs() * 2 * U


def linear(x, w, scale, swiglu_=False, residual=None):
    y, d = dot(x, w, scale)
    if swiglu_:
        h = y.shape[1] // 2
        return swiglu(y[:, :h], d[:, :h], y[:, h:], d[:, h:])
    if residual is not None:
        y = y + residual
        d = d + y.abs() * U
    return y, d


def ffn(x, ids, wts, w13, s13, w2, s2, residual=None):
    """w13 / w2: lists of binary64 matrices per expert."""
    T, H = x.shape
    out, bound = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    mag = torch.zeros(T, H, dtype=torch.float64)
    terms = 0
    for e in range(len(w13)):
        rows = [t for t in range(T) if (ids[t] == e).any()]
        if not rows:
            continue
        c = torch.tensor([float(wts[t][ids[t] == e].double().sum()) for t in rows],
                         dtype=torch.float64)[:, None] * s2[e]
        y, d = dot(x[rows], w13[e], s13[e])
        h = y.shape[1] // 2
        v, dv = swiglu(y[:, :h], d[:, :h], y[:, h:], d[:, h:])
        # Times c (its sum of weights, product and use: ids.shape[1] + 2 roundings), then two
        # BF16 parts: 2^-9 of a rest of at most 2^-9.
        cs = c.abs() + ids.shape[1] * U * c.abs()
        dh = dv * cs + (v * c).abs() * ((ids.shape[1] + 3) * U + 2.0 ** -18)
        out[rows] += (v * c) @ w2[e].t()
        bound[rows] += dh @ w2[e].abs().t()
        mag[rows] += ((v * c).abs() + dh) @ w2[e].abs().t()
        terms += h
    if residual is not None:
        out, mag = out + residual, mag + residual.abs()
    return out, bound + (2 * terms + len(w13) + 4) * U * mag


def check(got, ref, bound, what=""):
    """Every element within its bound plus the rounding to its type."""
    g = got.detach().cpu().double()
    room = bound + rounding(ref.abs() + bound, got.dtype)
    bad = ~((g - ref).abs() <= room)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {i}: "
                             f"{float(g[i])!r} for {float(ref[i])!r}, room {float(room[i])!r}")


def route(logits, topk, score, bias, renorm, groups, topk_groups):
    """ids, weights (binary64), offsets, row_token, token_rows, by sorting."""
    x = logits.double().numpy()
    T, E = x.shape
    with np.errstate(all="ignore"):
        if score == "softmax":
            key = x.copy()
            p = np.exp(x - x.max(1, keepdims=True)) if E else x
            p = p / p.sum(1, keepdims=True)
        else:
            p = 1 / (1 + np.exp(-x))
            key = p if bias is None else p + bias.double().numpy()
        # Order of the ranking: NaN below -inf, equal values by index.
        rank = np.where(np.isnan(key), -2, np.where(key == -np.inf, -1, 0))
        val = np.where(rank < 0, 0.0, key)
        order = np.stack([np.lexsort((np.arange(E), -val[t], -rank[t])) for t in range(T)]) \
            if T else np.zeros((0, E), np.int64)
        size = E // groups
        ids = np.zeros((T, topk), np.int64)
        for t in range(T):
            open_ = np.ones(E, bool)
            if topk_groups < groups:
                sc = np.where(np.isnan(key[t]), -1.5e308, np.maximum(key[t], -1e308))
                best = np.sort(sc.reshape(groups, size), 1)[:, ::-1]
                gv = best[:, 0] if score == "softmax" else best[:, :2].sum(1)
                first = np.lexsort((np.arange(groups), -gv))
                open_ = np.zeros(E, bool)
                for g in first[:topk_groups]:
                    open_[g * size:(g + 1) * size] = True
            ids[t] = [e for e in order[t] if open_[e]][:topk]
        w = np.take_along_axis(p, ids, 1)
        if renorm and score == "softmax":
            xs = np.take_along_axis(x, ids, 1)
            w = np.exp(xs - xs.max(1, keepdims=True)) if T else w
        if renorm:
            w = w / w.sum(1, keepdims=True)
    flat = ids.reshape(-1)
    order = np.argsort(flat, kind="stable")
    slots = np.empty_like(order)
    slots[order] = np.arange(T * topk)
    offsets = np.searchsorted(flat[order], np.arange(E + 1))
    return ids, w, offsets, order // topk, slots.reshape(T, topk)
