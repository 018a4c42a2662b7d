"""moe_fp4.moe_ffn against a plain 64-bit layer: sizes, routings, values that must stay
where they are, workspaces, streams and graphs.  Bounds: few_token_ref."""
import numpy as np
import pytest
import torch

import few_token_ref as ref
from gpu_util import dev, require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _layer(T, E, K, H, I, dtype, seed=0, ids=None, gain=1.0):
    rng = np.random.default_rng(seed + 1000 * T + E + 7 * H + I)
    if ids is None:
        ids = np.stack([rng.permutation(E)[:K] if K <= E else rng.integers(0, E, K) for _ in range(T)])
    q1, f1 = ref.weights(rng, (E, 2 * I, H))
    q2, f2 = ref.weights(rng, (E, H, I))
    f = lambda s: torch.from_numpy((rng.uniform(0.3, 1.5, E) * s).astype(np.float32))  # noqa: E731
    return dict(x=torch.from_numpy(rng.standard_normal((T, H)) * gain).to(ref.DT[dtype]),
                ids=torch.from_numpy(np.asarray(ids, np.int32)).reshape(T, -1),
                weights=torch.from_numpy(rng.uniform(0, 1, (T, np.asarray(ids).reshape(T, -1).shape[1]))
                                         .astype(np.float32)),
                w13_q=q1, w13_sf=f1, w13_scale=f(1.5 / np.sqrt(H)), w2_q=q2, w2_sf=f2,
                w2_scale=f(1 / np.sqrt(I)),
                residual=torch.from_numpy(rng.standard_normal((T, H))).to(ref.DT[dtype]))


def _gpu_args(L):
    return {k: (dev(v) if isinstance(v, np.ndarray) else v.cuda()) for k, v in L.items()}


def _run(L, **kw):
    from block_scaled_fp4_05_amd import moe_fp4
    a = _gpu_args(L)
    if not kw.pop("residual", True):
        a["residual"] = None
    return moe_fp4.moe_ffn(**a, **kw)


def _want(L, residual=True):
    E = L["w13_q"].shape[0]
    w13 = [ref.values(L["w13_q"][e], L["w13_sf"][e]) for e in range(E)]
    w2 = [ref.values(L["w2_q"][e], L["w2_sf"][e]) for e in range(E)]
    return ref.ffn(L["x"].double(), L["ids"], L["weights"], w13, L["w13_scale"].double(), w2,
                   L["w2_scale"].double(), L["residual"].double() if residual else None)


SIZES = [(1, 1, 1, 64, 64), (1, 8, 2, 64, 80), (1, 40, 8, 528, 256), (2, 3, 2, 272, 64), (3, 5, 5, 96, 112),
         (4, 70, 6, 80, 272), (8, 16, 3, 784, 96), (9, 33, 4, 64, 528), (16, 4, 2, 256, 144),
         (17, 6, 3, 112, 256), (33, 130, 8, 64, 64), (40, 2, 2, 320, 80), (64, 3, 2, 64, 304),
         (64, 1, 1, 256, 64), (2, 300, 32, 64, 64), (5, 80, 16, 2064, 64)]


@pytest.mark.parametrize("T,E,K,H,I", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_ffn_sizes(T, E, K, H, I, dtype):
    say(f"ffn T{T} E{E} K{K} H{H} I{I} {dtype}")
    L = _layer(T, E, K, H, I, dtype)
    out = _run(L)
    assert out.dtype == ref.DT[dtype] and out.shape == (T, H)
    ref.check(out, *_want(L), what="same type")
    ref.check(_run(L, residual=False, out_dtype=torch.float32), *_want(L, False), what="FP32, no residual")


@pytest.mark.parametrize("ids", [
    [[-1, -1], [0, -1], [-1, 2]],                    # a token without a slot
    [[5, 9], [2 ** 31 - 1, 1], [-(2 ** 31), 4]],     # ids of other ranks
    [[3, 3], [3, 3], [0, 3]],                        # an expert named twice
    [[-1, -1], [-1, -1], [-1, -1]],                  # nothing routed
    [[4, 4], [4, 4], [4, 4]],                        # one expert only
])
@pytest.mark.parametrize("residual", [True, False])
def test_ffn_routings(ids, residual):
    L = _layer(3, 5, 2, 96, 80, "bf16", ids=ids)
    out = _run(L, residual=residual)
    y, d = _want(L, residual)
    ref.check(out, y, d)
    for t, row in enumerate(ids):
        if not any(0 <= e < 5 for e in row):
            assert torch.equal(out[t].cpu(), L["residual"][t] if residual else torch.zeros(96).bfloat16())


def _skewed(T, E, busy, others):
    """Every token to expert `busy`, but the first few to `others`."""
    return [[others[t]] if t < len(others) else [busy] for t in range(T)]


@pytest.mark.parametrize("T,E,K,H,I,ids", [
    # One expert takes all: its weights pass by 16 times (two tiles a wavefront, room for four
    # tokens, codes turned in LDS), and 13 groups of five rows are summed with four in flight.
    (64, 256, 1, 64, 512, _skewed(64, 256, 200, [])),
    # The same beside lighter experts, so that a wavefront's units begin and end inside one.
    (64, 256, 1, 80, 528, _skewed(64, 256, 200, [3, 255, 3, 7, 9, 255])),
    (41, 60, 1, 272, 800, _skewed(41, 60, 0, [59, 1, 2])),
    # Room for 16 tokens with two tiles a wavefront, even and uneven.
    (64, 8, 2, 64, 512, None),
    (40, 8, 3, 80, 528, [[1, 1 + t % 7, 0] for t in range(40)]),
    # More than eight steps a wavefront: two tiles, one tile.
    (4, 8, 2, 8720, 512, None),
    (2, 8, 4, 8464, 512, None),
    (3, 3, 1, 16656, 64, None),
])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_ffn_uneven_loads_and_long_rows(T, E, K, H, I, ids, dtype):
    say(f"ffn uneven T{T} E{E} K{K} H{H} I{I} {dtype}")
    L = _layer(T, E, K, H, I, dtype, ids=ids)
    ref.check(_run(L), *_want(L))
    ref.check(_run(L, residual=False, out_dtype=torch.float32), *_want(L, False))


def test_ffn_many_experts():
    """8192 experts, ids at both ends of the range."""
    E, H, I = 8192, 64, 64
    ids = [[0, 8191, 4095], [8191, 31, 32], [63, 64, 2048]]
    L = _layer(3, E, 3, H, I, "bf16", ids=ids)
    used = sorted({e for r in ids for e in r})
    w13 = [ref.values(L["w13_q"][e], L["w13_sf"][e]) for e in used]
    w2 = [ref.values(L["w2_q"][e], L["w2_sf"][e]) for e in used]
    local = torch.tensor([[used.index(e) for e in r] for r in ids])
    ref.check(_run(L), *ref.ffn(L["x"].double(), local, L["weights"], w13, L["w13_scale"].double()[used],
                                w2, L["w2_scale"].double()[used], L["residual"].double()))


def test_ffn_nothing_leaks_between_experts_and_tokens():
    """Experts that no token names may hold NaN scales; a named expert's NaN stays with
    its tokens, a token's NaN with the token."""
    T, E, H, I = 6, 7, 112, 96
    ids = [[0, 1], [1, 2], [2, 3], [0, 3], [5, 1], [0, 2]]
    L = _layer(T, E, 2, H, I, "bf16", ids=ids)
    for e in (4, 6):
        L["w13_sf"][e], L["w2_sf"][e] = 0x7F, 0xFF
        L["w13_scale"][e] = float("nan")
    L["w13_sf"][5, 3, 0] = 0x7F
    L["x"][2, 5] = float("nan")
    out = _run(L).cpu()
    assert out[2].isnan().all() and out[4].isnan().all()
    rows = [0, 1, 3, 5]
    sub = dict(L, x=L["x"][rows], ids=L["ids"][rows], weights=L["weights"][rows], residual=L["residual"][rows])
    ref.check(out[rows], *_want(sub))


def test_ffn_down_weights_that_are_not_finite_stay_with_their_tokens():
    L = _layer(4, 3, 1, 64, 64, "fp16", ids=[[0], [1], [2], [1]])
    L["w2_sf"][1, 5, 1] = 0x7F
    out = _run(L).cpu()
    assert out[[1, 3], 5].isnan().all()
    y, d = _want(L)
    ref.check(out[[0, 2]], y[[0, 2]], d[[0, 2]])
    cols = [j for j in range(64) if j != 5]
    ref.check(out[[1, 3]][:, cols], y[[1, 3]][:, cols], d[[1, 3]][:, cols])


def test_ffn_intermediate_beyond_fp16():
    """silu(g) * u reaches 1e6 while the FP16 layer's output stays finite."""
    L = _layer(2, 2, 1, 128, 64, "fp16", gain=300.0)
    L["w2_scale"] *= 2.0 ** -14
    y, d = _want(L)
    assert torch.isfinite(_run(L)).all()
    ref.check(_run(L), y, d)


@pytest.mark.parametrize("T", [1, 4, 9])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_ffn_intermediate_keeps_fp32(T, dtype):
    """One-hot activations make gate and up exact, a unit down projection sums one value a
    column: what is left of the error is the epilogue's few FP32 operations (swiglu's, and
    topk + 3 for the weight), with no rounding of the intermediate to fewer bits."""
    E, K, H, I = 3, 1, 256, 256
    L = _layer(T, E, K, H, I, dtype, ids=[[t % E] for t in range(T)])
    L["x"] = torch.eye(T, H, dtype=ref.DT[dtype])
    L["w2_q"] = np.zeros((E, H, I // 2), np.uint8)
    for j in range(H):
        L["w2_q"][:, j, j // 2] = 0x20 if j % 2 else 0x02  # code of 1
    L["w2_sf"] = np.full((E, H, I // 16), 0x38, np.uint8)  # block scale 1
    got = _run(L, residual=False, out_dtype=torch.float32).cpu().double()
    for t in range(T):
        e = t % E
        y = ref.values(L["w13_q"][e], L["w13_sf"][e])[:, t] * L["w13_scale"][e].double()
        v, dv = ref.swiglu(y[:I], y[:I].abs() * ref.U, y[I:], y[I:].abs() * ref.U)
        c = L["weights"][t, 0].double() * L["w2_scale"][e].double()
        want, bound = v * c, dv * c + (v * c).abs() * (K + 3) * ref.U
        assert ((got[t] - want).abs() <= bound).all(), float(((got[t] - want).abs() / bound.clamp(min=1e-300)).max())


def test_ffn_infinite_intermediate_has_its_sign():
    """An infinity in the intermediate is an infinity in the output, not a NaN: all weights
    positive, one activation infinite."""
    L = _layer(6, 2, 1, 64, 64, "bf16", ids=[[0], [1], [0], [0], [0], [0]])
    for q, f in (("w13_q", "w13_sf"), ("w2_q", "w2_sf")):
        L[q] = (L[q] & 0x66) | 0x11  # codes 0.5, 1.5, 3 and 6
        L[f] = (L[f] & 0x7F) | 0x20
    L["x"][3, 7] = float("inf")
    out = _run(L).cpu()
    assert (out[3] == float("inf")).all()
    rows = [0, 1, 2, 4, 5]
    y, d = _want(L)
    ref.check(out[rows], y[rows], d[rows])


def test_ffn_pitches_and_workspace():
    from block_scaled_fp4_05_amd import moe_fp4
    T, E, K, H, I = 5, 6, 3, 80, 64
    L = _layer(T, E, K, H, I, "bf16")
    a = _gpu_args(L)
    wide = torch.full((T, H + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :H] = a["x"]
    res = torch.full((T, H + 1), float("nan"), dtype=torch.bfloat16, device="cuda")
    res[:, :H] = a["residual"]
    out = torch.full((T + 1, H + 3), 7.0, device="cuda")
    ws = torch.full((moe_fp4.ffn_workspace_size(T, K, E, I) + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    a.update(x=wide[:, :H], residual=res[:, :H], out=out[:T, :H], workspace=ws)
    for _ in range(2):
        moe_fp4.moe_ffn(**a)
        ref.check(out[:T, :H], *_want(L))
    assert (out[:, H:] == 7).all() and (out[T] == 7).all() and (ws[-64:] == 0xFF).all()
    y = a["residual"].contiguous()
    a.update(residual=y, out=y, workspace=None)
    moe_fp4.moe_ffn(**a)
    ref.check(y, *_want(L))


def test_ffn_zero_tokens():
    L = _layer(1, 2, 1, 64, 64, "bf16")
    L = dict(L, **{k: L[k][:0] for k in ("x", "ids", "weights", "residual")})
    assert _run(L).shape == (0, 64)


@pytest.mark.parametrize("T", [1, 20])
def test_ffn_repeats_its_bits_on_other_streams_and_in_graphs(T):
    from block_scaled_fp4_05_amd import moe_fp4
    a = _gpu_args(_layer(T, 12, 4, 272, 80, "bf16"))
    want = moe_fp4.moe_ffn(**a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = moe_fp4.moe_ffn(**a, stream=side)
    side.synchronize()
    assert torch.equal(other, want)
    g, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(g):
        moe_fp4.moe_ffn(**a, out=out)
    for i in range(3):  # other activations, and another routing
        a["x"].copy_(torch.roll(a["x"], 1, 1))
        a["ids"].copy_((a["ids"] + 5) % 12)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, moe_fp4.moe_ffn(**a)), i
