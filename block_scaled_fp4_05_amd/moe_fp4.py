"""Python binding of libmoe_fp4.so (the C ABI in include/moe_fp4.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels.  PyTorch supplies device memory and the current stream.  If the
compiled library is missing the calls raise; there is no CPU fallback.

Streams: a call runs on `stream` (default: the current stream), and the results and
workspaces that it allocates itself belong to that stream.  As with any torch tensor, the
caller makes the launch stream wait for inputs that other streams write, makes another stream
wait for it before using the results there, and calls record_stream on a result that is dropped
while another stream still uses it.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.util
import os
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# MOE_FP4_LIB may name another build of the same sources (the host-sanitizer
# build of the CPU tests); by default the in-tree library.
LIB_PATH = os.environ.get("MOE_FP4_LIB") or os.path.join(_PKG, "libmoe_fp4.so")

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED, ERR_HIP, ERR_ARG = range(7)
OUT_BF16, OUT_FP32, OUT_FP16 = 0, 1, 2
IN_BF16, IN_FP32, IN_FP16 = 0, 1, 2
SCALE_STATIC, SCALE_DYNAMIC = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1

# Every symbol include/moe_fp4.h declares.
EXPORTED = ("moe_fp4_quantize", "moe_grouped_gemm_fp4", "moe_grouped_gemm_fp4_packed",
            "moe_grouped_gemm_fp4_finalize", "moe_grouped_gemm_fp4_swiglu", "moe_fp4_combine",
            "moe_fp4_linear", "moe_fp4_ffn", "moe_fp4_ffn_workspace_size", "moe_fp4_route",
            "moe_fp4_route_workspace_size",
            "moe_fp4_pack_weights", "moe_fp4_unpack_weights", "moe_grouped_gemm_fp4_plan",
            "moe_grouped_gemm_fp4_workspace_size", "moe_fp4_stage_bytes",
            "moe_fp4_status_string", "moe_fp4_abi_version")


class MoeFp4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


class Plan(ctypes.Structure):
    _fields_ = [("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32),
                ("k_step", ctypes.c_int32), ("waves_per_group", ctypes.c_int32),
                ("lds_bytes", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load the compiled library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with block_scaled_fp4_05_amd.build")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, i = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
    L.moe_fp4_quantize.argtypes = [vp, i, i64, i64, i64, vp, vp, vp, i, vp]
    L.moe_fp4_quantize.restype = i
    L.moe_grouped_gemm_fp4.argtypes = [vp, vp, vp, i64, vp, vp, vp, vp, vp, i32, i64, i64, i64,
                                       vp, i64, vp]
    L.moe_grouped_gemm_fp4.restype = i
    L.moe_grouped_gemm_fp4_packed.argtypes = L.moe_grouped_gemm_fp4.argtypes
    L.moe_grouped_gemm_fp4_packed.restype = i
    L.moe_grouped_gemm_fp4_finalize.argtypes = [vp, vp, vp, i64, vp, vp, vp, vp, i, vp, i32, i64,
                                                 i64, i64, vp, vp, vp, i64, i64, vp]
    L.moe_grouped_gemm_fp4_finalize.restype = i
    L.moe_grouped_gemm_fp4_swiglu.argtypes = [vp, vp, vp, i64, vp, vp, vp, vp, i, vp, i32, i64,
                                               i64, i64, vp, vp, vp, vp]
    L.moe_grouped_gemm_fp4_swiglu.restype = i
    L.moe_fp4_combine.argtypes = [vp, i64, i64, vp, vp, i32, i64, i64, vp, i64, vp, i, i64, vp]
    L.moe_fp4_combine.restype = i
    L.moe_fp4_linear.argtypes = [vp, i, i64, i64, vp, vp, vp, i64, i64, i, vp, i64, vp, i, i64, vp]
    L.moe_fp4_linear.restype = i
    L.moe_fp4_ffn_workspace_size.argtypes = [i64, i32, i32, i64]
    L.moe_fp4_ffn_workspace_size.restype = ctypes.c_size_t
    L.moe_fp4_ffn.argtypes = [vp, i, i64, i64, vp, vp, i32, vp, vp, vp, vp, vp, vp, i32, i64, i64,
                              vp, i64, vp, i, i64, vp, ctypes.c_size_t, vp]
    L.moe_fp4_ffn.restype = i
    L.moe_fp4_route_workspace_size.argtypes = [i64, i32]
    L.moe_fp4_route_workspace_size.restype = ctypes.c_size_t
    L.moe_fp4_route.argtypes = [vp, i, i64, i32, i64, i, vp, i, i32, i32, i32, vp, vp, vp, vp, vp,
                                vp, ctypes.c_size_t, vp]
    L.moe_fp4_route.restype = i
    for f in (L.moe_fp4_pack_weights, L.moe_fp4_unpack_weights):
        f.argtypes = [vp, vp, i32, i64, i64, vp]
        f.restype = i
    L.moe_grouped_gemm_fp4_plan.argtypes = [i32, i64, i64, i64, ctypes.POINTER(Plan)]
    L.moe_grouped_gemm_fp4_plan.restype = i
    L.moe_grouped_gemm_fp4_workspace_size.argtypes = [i32, i64, i64, i64]
    L.moe_grouped_gemm_fp4_workspace_size.restype = ctypes.c_size_t
    L.moe_fp4_stage_bytes.argtypes = [i64, i64, i64]
    L.moe_fp4_stage_bytes.restype = i64
    L.moe_fp4_status_string.argtypes = [i]
    L.moe_fp4_status_string.restype = ctypes.c_char_p
    L.moe_fp4_abi_version.argtypes = []
    L.moe_fp4_abi_version.restype = i
    _load_calls(L)
    _lib = L
    return L


# The few-token calls' short host path (csrc/calls.cpp), or None where it was not built for
# this torch: the Python code below does the same, only slower.
_calls = None


def _load_calls(L) -> None:
    global _calls
    path = os.path.join(_PKG, "_calls.so")
    try:
        spec = importlib.util.spec_from_file_location("_calls", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except (ImportError, OSError):
        return
    module.bind(*(ctypes.cast(f, ctypes.c_void_p).value
                  for f in (L.moe_fp4_linear, L.moe_fp4_ffn, L.moe_fp4_ffn_workspace_size,
                            L.moe_fp4_route, L.moe_fp4_route_workspace_size)))
    _calls = module


def status_string(status: int) -> str:
    return lib().moe_fp4_status_string(int(status)).decode()


def abi_version() -> int:
    return lib().moe_fp4_abi_version()


def stage_bytes(bm: int, bn: int, bk: int) -> int:
    return lib().moe_fp4_stage_bytes(bm, bn, bk)


def workspace_size(num_experts: int, m_total: int, n: int, k: int) -> int:
    """Device workspace bytes of the grouped GEMM for these sizes (always 0)."""
    return lib().moe_grouped_gemm_fp4_workspace_size(num_experts, m_total, n, k)


def plan(num_experts: int, m_total: int, n: int, k: int) -> dict:
    p = Plan()
    st = lib().moe_grouped_gemm_fp4_plan(num_experts, m_total, n, k, ctypes.byref(p))
    if st != OK:
        raise MoeFp4Error(st, "moe_grouped_gemm_fp4_plan")
    return {f: getattr(p, f) for f, _ in Plan._fields_}


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, dev):
    """The launch stream (default: the current stream of the current device), which
    must belong to the tensors' device `dev`: the kernels run on the stream's device."""
    if stream is None:
        stream = torch.cuda.current_stream()
    if stream.device_index != dev:
        raise ValueError(f"stream on cuda:{stream.device_index}, tensors on cuda:{dev}")
    return ctypes.c_void_p(stream.cuda_stream)


_AS_IT_IS = contextlib.nullcontext()


def _on(stream):
    """Where a call makes its new tensors (results and workspaces): on its launch stream.
    From the current stream's pool they could be memory that work still queued there uses,
    which the launch stream does not wait for."""
    return _AS_IT_IS if stream is None else torch.cuda.stream(stream)


class _AtLeast(int):
    """A shape entry that admits any extent of at least this value."""

    def __repr__(self):
        return f">={int(self)}"


def _need(t, name, dtype, shape=None, contiguous=True, rows=False):
    """Check a tensor argument before its pointer is handed to the library: its dtype,
    its shape (None entries are free, _AtLeast(x) entries admit x or more), and its
    layout: contiguous, or with rows=True only unit stride along the last axis (rows
    at any leading dimension).  Raises ValueError.  (Plain loops: it runs on every
    call of a decode step.)"""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if shape is not None:
        ts = t.shape
        ok = len(ts) == len(shape)
        if ok:
            for i in range(len(shape)):
                w = shape[i]
                if w is not None and ((ts[i] < w) if type(w) is _AtLeast else (ts[i] != w)):
                    ok = False
                    break
        if not ok:
            raise ValueError(f"{name}: shape {tuple(ts)}, expected {tuple(shape)}")
    if rows:
        if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
            raise ValueError(f"{name}: rows must have unit column stride")
    elif contiguous and not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _same_cuda(names, *tensors):
    """All given tensors (None skipped) are CUDA tensors on one device, which is
    returned; `names` lists them, space-separated, for the error message."""
    dev = -1
    for t in tensors:
        if t is None:
            continue
        d = t.get_device()
        if d < 0 or (dev >= 0 and d != dev):
            devs = {nm: str(x.device) for nm, x in zip(names.split(), tensors) if x is not None}
            if d < 0:
                bad = [nm for nm, v in devs.items() if not v.startswith("cuda")]
                raise ValueError(f"{bad[0]}: must be a CUDA tensor (got {devs[bad[0]]})")
            raise ValueError(f"tensors on several devices: {devs}")
        dev = d
    return dev


def quantize_raw(x_ptr, in_dtype, rows, k, ld_x, q_ptr, sf_ptr, scale_ptr, scale_mode, stream_ptr):
    """Direct call with raw pointers; returns the status code."""
    return lib().moe_fp4_quantize(x_ptr, in_dtype, rows, k, ld_x, q_ptr, sf_ptr, scale_ptr,
                                  scale_mode, stream_ptr)


def gemm_raw(*args):
    """Direct call with raw pointers (C argument order); returns the status code."""
    return lib().moe_grouped_gemm_fp4(*args)


def gemm_packed_raw(*args):
    """moe_grouped_gemm_fp4_packed with raw pointers; returns the status code."""
    return lib().moe_grouped_gemm_fp4_packed(*args)


def pack_weights(w_q: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Row-major weight codes [E][n][k/2] (uint8, CUDA) -> the packed layout the
    packed GEMM reads (same shape and size; a byte permutation).  A new `out` belongs to the
    launch stream."""
    _need(w_q, "w_q", torch.uint8, (None, None, None))
    E, n, kb = w_q.shape
    if out is None:
        with _on(stream):
            out = torch.empty_like(w_q)
    _need(out, "out", torch.uint8, (E, n, kb))
    dev = _same_cuda("w_q out", w_q, out)
    st = lib().moe_fp4_pack_weights(_ptr(w_q), _ptr(out), E, n, 2 * kb, _stream(stream, dev))
    if st != OK:
        raise MoeFp4Error(st, "moe_fp4_pack_weights")
    return out


def unpack_weights(w_packed: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Inverse of pack_weights.  A new `out` belongs to the launch stream."""
    _need(w_packed, "w_packed", torch.uint8, (None, None, None))
    E, n, kb = w_packed.shape
    if out is None:
        with _on(stream):
            out = torch.empty_like(w_packed)
    _need(out, "out", torch.uint8, (E, n, kb))
    dev = _same_cuda("w_packed out", w_packed, out)
    st = lib().moe_fp4_unpack_weights(_ptr(w_packed), _ptr(out), E, n, 2 * kb, _stream(stream, dev))
    if st != OK:
        raise MoeFp4Error(st, "moe_fp4_unpack_weights")
    return out


def quantize(x: torch.Tensor, tensor_scale: torch.Tensor | None = None, q=None, sf=None,
             stream=None, dynamic: bool | None = None):
    """NVFP4-quantise a 2-D BF16 or FP32 CUDA tensor [rows][k].

    tensor_scale None -> dynamic: a new 1-element float32 tensor receives g.
    Otherwise a 1-element float32 CUDA tensor: by default it holds a calibrated g
    (static); with dynamic=True it receives the computed g instead.
    Returns (q uint8[rows][k/2], sf uint8[rows][k/16], tensor_scale float32[1]); new ones
    belong to the launch stream.
    """
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    if x.dtype == torch.bfloat16:
        dt = IN_BF16
    elif x.dtype == torch.float32:
        dt = IN_FP32
    else:
        raise ValueError("x must be bfloat16 or float32")
    rows, k = x.shape
    dev = x.device
    if dynamic is None:
        dynamic = tensor_scale is None
    mode = SCALE_DYNAMIC if dynamic else SCALE_STATIC
    if tensor_scale is None and not dynamic:
        raise ValueError("a static quantisation needs tensor_scale")
    with _on(stream):
        if q is None:
            q = torch.empty((rows, k // 2), dtype=torch.uint8, device=dev)
        if sf is None:
            sf = torch.empty((rows, k // 16), dtype=torch.uint8, device=dev)
        if tensor_scale is None:
            tensor_scale = torch.empty(1, dtype=torch.float32, device=dev)
    _need(q, "q", torch.uint8, (_AtLeast(rows), k // 2))
    _need(sf, "sf", torch.uint8, (_AtLeast(rows), k // 16))
    _need(tensor_scale, "tensor_scale", torch.float32, (_AtLeast(1),))
    dev = _same_cuda("x q sf tensor_scale", x, q, sf, tensor_scale)
    st = lib().moe_fp4_quantize(_ptr(x), dt, rows, k, x.stride(0), _ptr(q), _ptr(sf),
                                _ptr(tensor_scale), mode, _stream(stream, dev))
    if st != OK:
        raise MoeFp4Error(st, "moe_fp4_quantize")
    return q, sf, tensor_scale


def _gemm_operands(a_q, a_sf, a_scale, w_q, w_sf, w_scale, offsets, a_row_index, m_total):
    """Check the operands shared by the grouped-GEMM entry points; returns
    (E, n, k, a_rows, m_total)."""
    _need(w_q, "w_q", torch.uint8, (None, None, None))
    E, n, kb = w_q.shape
    _need(a_q, "a_q", torch.uint8, (None, kb))
    a_rows = a_q.shape[0]
    _need(a_sf, "a_sf", torch.uint8, (a_rows, kb // 8))
    _need(a_scale, "a_scale", torch.float32, (_AtLeast(1),))
    _need(w_sf, "w_sf", torch.uint8, (E, n, kb // 8))
    _need(w_scale, "w_scale", torch.float32, (E,))
    _need(offsets, "offsets", torch.int32, (E + 1,))
    if m_total is None:
        m_total = a_row_index.shape[0] if a_row_index is not None else a_rows
    if a_row_index is not None:
        _need(a_row_index, "a_row_index", torch.int32, (m_total,))
    return E, n, 2 * kb, a_rows, m_total


def grouped_gemm(a_q, a_sf, a_scale, w_q, w_sf, w_scale, offsets, a_row_index=None, out=None,
                 m_total: int | None = None, stream=None, packed: bool = False):
    """NVFP4 grouped GEMM.  Shapes: a_q [a_rows][k/2], a_sf [a_rows][k/16], a_scale [1],
    w_q [E][n][k/2], w_sf [E][n][k/16], w_scale [E], offsets int32 [E+1],
    a_row_index int32 [m_total] or None.  m_total defaults to a_row_index's length,
    else a_rows.  packed: w_q is in the packed layout (pack_weights).  Returns out,
    a BF16 tensor [m_total][n] that belongs to the launch stream (or the given `out`)."""
    E, n, k, a_rows, m_total = _gemm_operands(a_q, a_sf, a_scale, w_q, w_sf, w_scale, offsets,
                                              a_row_index, m_total)
    if out is None:
        with _on(stream):
            out = torch.empty((m_total, n), dtype=torch.bfloat16, device=w_q.device)
    _need(out, "out", torch.bfloat16, (_AtLeast(m_total), _AtLeast(n)), rows=True)
    dev = _same_cuda("a_q a_sf a_scale w_q w_sf w_scale offsets a_row_index out", a_q, a_sf, a_scale, w_q, w_sf, w_scale, offsets, a_row_index, out)
    fn = lib().moe_grouped_gemm_fp4_packed if packed else lib().moe_grouped_gemm_fp4
    st = fn(_ptr(a_q), _ptr(a_sf), _ptr(a_scale), a_rows, _ptr(a_row_index), _ptr(w_q), _ptr(w_sf),
            _ptr(w_scale), _ptr(offsets), E, m_total, n, k, _ptr(out), out.stride(0), _stream(stream, dev))
    if st != OK:
        raise MoeFp4Error(st, "moe_grouped_gemm_fp4_packed" if packed else "moe_grouped_gemm_fp4")
    return out


def finalize_raw(*args):
    """moe_grouped_gemm_fp4_finalize with raw pointers (C argument order); returns the status."""
    return lib().moe_grouped_gemm_fp4_finalize(*args)


def grouped_gemm_finalize(a_q, a_sf, a_scale, w_q, w_sf, w_scale, offsets, out_token, row_weight,
                          out, a_row_index=None, m_total: int | None = None, packed: bool = False,
                          stream=None):
    """Grouped GEMM with the finalize epilogue: routed row r adds row_weight[r] times its
    result into row out_token[r] of `out` (float32 CUDA tensor [num_tokens][ldo],
    accumulated into).  Other arguments as grouped_gemm.  Returns out."""
    E, n, k, a_rows, m_total = _gemm_operands(a_q, a_sf, a_scale, w_q, w_sf, w_scale, offsets,
                                              a_row_index, m_total)
    _need(out_token, "out_token", torch.int32, (m_total,))
    _need(row_weight, "row_weight", torch.float32, (m_total,))
    _need(out, "out", torch.float32, (None, _AtLeast(n)), rows=True)
    dev = _same_cuda("a_q a_sf a_scale w_q w_sf w_scale offsets a_row_index out_token row_weight out", a_q, a_sf, a_scale, w_q, w_sf, w_scale, offsets, a_row_index, out_token, row_weight, out)
    st = lib().moe_grouped_gemm_fp4_finalize(
        _ptr(a_q), _ptr(a_sf), _ptr(a_scale), a_rows, _ptr(a_row_index), _ptr(w_q), _ptr(w_sf),
        _ptr(w_scale), 1 if packed else 0, _ptr(offsets), E, m_total, n, k, _ptr(out_token),
        _ptr(row_weight), _ptr(out), out.stride(0), out.shape[0], _stream(stream, dev))
    if st != OK:
        raise MoeFp4Error(st, "moe_grouped_gemm_fp4_finalize")
    return out


def swiglu_raw(*args):
    """moe_grouped_gemm_fp4_swiglu with raw pointers (C argument order); returns the status."""
    return lib().moe_grouped_gemm_fp4_swiglu(*args)


def grouped_gemm_swiglu(a_q, a_sf, a_scale, w_q, w_sf, w_scale, offsets, h_scale,
                        a_row_index=None, h_q=None, h_sf=None, m_total: int | None = None,
                        packed: bool = False, stream=None):
    """Gate+up grouped GEMM with the SwiGLU + NVFP4 epilogue.  w_q [E][2I][k/2]: rows
    0..I-1 the gate, I..2I-1 the up projection; h_scale float32 CUDA tensor [1], the
    intermediate's static tensor scale.  Other arguments as grouped_gemm.  Returns
    (h_q uint8 [m_total][I/2], h_sf uint8 [m_total][I/16]), the down projection's
    activations; new ones belong to the launch stream."""
    E, n, k, a_rows, m_total = _gemm_operands(a_q, a_sf, a_scale, w_q, w_sf, w_scale, offsets,
                                              a_row_index, m_total)
    dev = w_q.device
    with _on(stream):
        if h_q is None:
            h_q = torch.empty((m_total, n // 4), dtype=torch.uint8, device=dev)
        if h_sf is None:
            h_sf = torch.empty((m_total, n // 32), dtype=torch.uint8, device=dev)
    _need(h_scale, "h_scale", torch.float32, (_AtLeast(1),))
    _need(h_q, "h_q", torch.uint8, (_AtLeast(m_total), n // 4))
    _need(h_sf, "h_sf", torch.uint8, (_AtLeast(m_total), n // 32))
    dev = _same_cuda("a_q a_sf a_scale w_q w_sf w_scale offsets a_row_index h_scale h_q h_sf", a_q, a_sf, a_scale, w_q, w_sf, w_scale, offsets, a_row_index, h_scale, h_q, h_sf)
    st = lib().moe_grouped_gemm_fp4_swiglu(
        _ptr(a_q), _ptr(a_sf), _ptr(a_scale), a_rows, _ptr(a_row_index), _ptr(w_q), _ptr(w_sf),
        _ptr(w_scale), 1 if packed else 0, _ptr(offsets), E, m_total, n, k, _ptr(h_scale),
        _ptr(h_q), _ptr(h_sf), _stream(stream, dev))
    if st != OK:
        raise MoeFp4Error(st, "moe_grouped_gemm_fp4_swiglu")
    return h_q, h_sf


def combine_raw(*args):
    """moe_fp4_combine with raw pointers (C argument order); returns the status."""
    return lib().moe_fp4_combine(*args)


def combine(rows, token_rows, token_weights, out=None, residual=None, out_dtype=torch.bfloat16,
            stream=None):
    """Token-order combine: out[t] = (residual[t] +) sum_s token_weights[t][s] * rows[token_rows[t][s]]
    in FP32, slots in order.  rows: BF16 CUDA tensor [m_total][>= n] (the grouped GEMM's
    output); token_rows int32 / token_weights float32 [num_tokens][topk].  Returns out
    ([num_tokens][n] of out_dtype, bfloat16 or float32); a new one belongs to the launch
    stream."""
    _need(rows, "rows", torch.bfloat16, (None, None), rows=True)
    m_total, n = rows.shape
    _need(token_rows, "token_rows", torch.int32, (None, None))
    T, topk = token_rows.shape
    _need(token_weights, "token_weights", torch.float32, (T, topk))
    if residual is not None:
        _need(residual, "residual", torch.float32, (T, _AtLeast(n)), rows=True)
    if out is None:
        with _on(stream):
            out = torch.empty((T, n), dtype=out_dtype, device=rows.device)
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"out: dtype {out.dtype}, expected bfloat16 or float32")
    _need(out, "out", out.dtype, (T, _AtLeast(n)), rows=True)
    dev = _same_cuda("rows token_rows token_weights residual out", rows, token_rows, token_weights, residual, out)
    dt = OUT_FP32 if out.dtype == torch.float32 else OUT_BF16
    st = lib().moe_fp4_combine(_ptr(rows), rows.stride(0), m_total, _ptr(token_rows),
                               _ptr(token_weights), topk, T, n, _ptr(residual),
                               residual.stride(0) if residual is not None else 0, _ptr(out), dt,
                               out.stride(0), _stream(stream, dev))
    if st != OK:
        raise MoeFp4Error(st, "moe_fp4_combine")
    return out


_IN_TYPES = {torch.bfloat16: IN_BF16, torch.float32: IN_FP32, torch.float16: IN_FP16}
_OUT_TYPES = {torch.bfloat16: OUT_BF16, torch.float32: OUT_FP32, torch.float16: OUT_FP16}


# The calls below are short on the GPU (a few microseconds), so their host time counts.
# Plain calls (tensors on the current device and its current stream) go through _calls,
# which checks and allocates in C++ and returns None where anything is out of the
# ordinary; the Python code then does the call or names what is wrong.  Here, tensors are
# checked with the three plain comparisons that almost always hold, and _need runs only
# where one of them fails.

def _exact(t, name, dtype, shape):
    """A contiguous tensor of this dtype and shape."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        _need(t, name, dtype, shape)


def _pitch(t, name, dtype, shape):
    """A matrix of this dtype and shape with unit column stride; returns its row pitch."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape):
        _need(t, name, dtype, shape)
    row, col = t.stride()
    if col != 1 and shape[1] > 1 and shape[0] > 0:  # (an empty tensor may have any strides)
        raise ValueError(f"{name}: rows must have unit column stride")
    return row if shape[0] > 1 else shape[1]


def _current_device():
    return torch._C._cuda_getDevice()


def _raw_stream(dev):
    """The current stream of device `dev`, as the number the C entry points take."""
    return torch._C._cuda_getCurrentRawStream(dev)


def _launch_stream(stream, dev):
    """_stream, without a stream object for the default."""
    if stream is not None:
        return _stream(stream, dev)
    if _current_device() != dev:
        raise ValueError(f"stream on cuda:{_current_device()}, tensors on cuda:{dev}")
    return _raw_stream(dev)


def _few_rows(x, residual, out, out_dtype, m, k, cols, stream):
    """Check the activations, residual and output of a few-token call; returns
    (x type, x pitch, residual pitch, out, out type, out pitch)."""
    dt = x.dtype
    ld = _pitch(x, "x", dt, (m, k))
    ld_res = 0 if residual is None else _pitch(residual, "residual", dt, (m, cols))
    if out is None:
        with _on(stream):
            out = x.new_empty((m, cols)) if out_dtype is None else x.new_empty((m, cols), dtype=out_dtype)
        if out.dtype not in _OUT_TYPES:
            raise ValueError(f"out_dtype: {out_dtype}, expected bfloat16, float16 or float32")
        return _IN_TYPES[dt], ld, ld_res, out, _OUT_TYPES[out.dtype], cols
    if not isinstance(out, torch.Tensor) or out.dtype not in _OUT_TYPES or \
            (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out: expected a " + ("bfloat16, float16 or float32" if out_dtype is None
                                               else str(out_dtype)) + " tensor")
    ldo = _pitch(out, "out", out.dtype, (m, cols))
    return _IN_TYPES[dt], ld, ld_res, out, _OUT_TYPES[out.dtype], ldo


def _x_ok(x):
    if not isinstance(x, torch.Tensor) or x.dtype not in (torch.bfloat16, torch.float16) or x.dim() != 2:
        raise ValueError("x: expected a 2-D bfloat16 or float16 tensor")
    return x.shape


def linear_raw(*args):
    """moe_fp4_linear with raw pointers (C argument order); returns the status."""
    return lib().moe_fp4_linear(*args)


def linear(x, w_q, w_sf, w_scale, swiglu: bool = False, residual=None, out=None, out_dtype=None,
           stream=None):
    """Few-token linear layer: x (bfloat16 or float16 CUDA tensor [m][k], unit column
    stride) times NVFP4 weights w_q uint8 [n][k/2], w_sf uint8 [n][k/16], w_scale
    float32 [1].  Returns out [m][n] = x W^T (+ residual, x's type [m][n]), or with swiglu
    [m][n/2] = silu(first half) * second half; of out_dtype (default: x's type).  A new out
    belongs to the launch stream."""
    if (_calls or lib() and _calls) and stream is None and isinstance(x, torch.Tensor) and x.is_cuda:
        dev = _current_device()
        got = _calls.linear(x, w_q, w_sf, w_scale, swiglu, residual, out,
                            -1 if out_dtype is None else _OUT_TYPES.get(out_dtype, 3), dev, _raw_stream(dev))
        if got is not None:
            return got
    m, k = _x_ok(x)
    _need(w_q, "w_q", torch.uint8, (None, k // 2))
    n = w_q.shape[0]
    if swiglu and (n % 2 or residual is not None):
        raise ValueError("swiglu: needs an even number of weight rows and no residual")
    _exact(w_sf, "w_sf", torch.uint8, (n, k // 16))
    _exact(w_scale, "w_scale", torch.float32, (1,))
    dt, ld, ld_res, out, odt, ldo = _few_rows(x, residual, out, out_dtype, m, k, n // 2 if swiglu else n, stream)
    dev = _same_cuda("x w_q w_sf w_scale residual out", x, w_q, w_sf, w_scale, residual, out)
    st = (_lib or lib()).moe_fp4_linear(
        x.data_ptr(), dt, m, ld, w_q.data_ptr(), w_sf.data_ptr(), w_scale.data_ptr(), n, k,
        1 if swiglu else 0, None if residual is None else residual.data_ptr(), ld_res, out.data_ptr(),
        odt, ldo, _launch_stream(stream, dev))
    if st != OK:
        raise MoeFp4Error(st, "moe_fp4_linear")
    return out


def ffn_raw(*args):
    """moe_fp4_ffn with raw pointers (C argument order); returns the status."""
    return lib().moe_fp4_ffn(*args)


def ffn_workspace_size(tokens: int, topk: int, num_experts: int, inter: int) -> int:
    """Device workspace bytes of moe_ffn for these sizes (0 where it does not run)."""
    return (_lib or lib()).moe_fp4_ffn_workspace_size(tokens, topk, num_experts, inter)


def moe_ffn(x, ids, weights, w13_q, w13_sf, w13_scale, w2_q, w2_sf, w2_scale, residual=None,
            out=None, out_dtype=None, workspace=None, stream=None):
    """A whole Mixture-of-Experts layer for up to 64 tokens: x (bfloat16 or float16 CUDA
    tensor [tokens][hidden]), ids int32 / weights float32 [tokens][topk] (an id outside
    [0, E) is skipped), NVFP4 weights w13 [E][2I][hidden] (gate rows, then up rows) and
    w2 [E][hidden][I] with scales float32 [E].  Returns out [tokens][hidden] = (residual +)
    the routing-weighted sum of the experts, of out_dtype (default: x's type).
    workspace: uint8 CUDA tensor of ffn_workspace_size bytes (default: a new one).  A new out
    or workspace belongs to the launch stream."""
    if (_calls or lib() and _calls) and stream is None and workspace is None and \
            isinstance(x, torch.Tensor) and x.is_cuda:
        dev = _current_device()
        got = _calls.ffn(x, ids, weights, w13_q, w13_sf, w13_scale, w2_q, w2_sf, w2_scale, residual, out,
                         -1 if out_dtype is None else _OUT_TYPES.get(out_dtype, 3), dev, _raw_stream(dev))
        if got is not None:
            return got
    u8, f32 = torch.uint8, torch.float32
    T, H = _x_ok(x)
    _need(w13_q, "w13_q", u8, (None, None, H // 2))
    E, rows, _ = w13_q.shape
    I = rows // 2
    if rows % 2:
        raise ValueError(f"w13_q: shape {tuple(w13_q.shape)}, expected an even number of rows")
    _need(ids, "ids", torch.int32, (T, None))
    K = ids.shape[1]
    _exact(weights, "weights", f32, (T, K))
    _exact(w13_sf, "w13_sf", u8, (E, rows, H // 16))
    _exact(w13_scale, "w13_scale", f32, (E,))
    _exact(w2_q, "w2_q", u8, (E, H, I // 2))
    _exact(w2_sf, "w2_sf", u8, (E, H, I // 16))
    _exact(w2_scale, "w2_scale", f32, (E,))
    dt, ld, ld_res, out, odt, ldo = _few_rows(x, residual, out, out_dtype, T, H, H, stream)
    if workspace is None:
        with _on(stream):
            workspace = w13_q.new_empty(ffn_workspace_size(T, K, E, I))
    else:
        _need(workspace, "workspace", u8, (_AtLeast(ffn_workspace_size(T, K, E, I)),))
    dev = _same_cuda("x ids weights w13_q w13_sf w13_scale w2_q w2_sf w2_scale residual out workspace",
                     x, ids, weights, w13_q, w13_sf, w13_scale, w2_q, w2_sf, w2_scale, residual, out,
                     workspace)
    st = (_lib or lib()).moe_fp4_ffn(
        x.data_ptr(), dt, T, ld, ids.data_ptr(), weights.data_ptr(), K, w13_q.data_ptr(),
        w13_sf.data_ptr(), w13_scale.data_ptr(), w2_q.data_ptr(), w2_sf.data_ptr(), w2_scale.data_ptr(),
        E, H, I, None if residual is None else residual.data_ptr(), ld_res, out.data_ptr(), odt, ldo,
        workspace.data_ptr(), workspace.numel(), _launch_stream(stream, dev))
    if st != OK:
        raise MoeFp4Error(st, "moe_fp4_ffn")
    return out


class Routing(NamedTuple):
    """What the router leaves on the GPU: ids / weights / token_rows [tokens][topk],
    offsets [E + 1], row_token [tokens * topk] (moe_fp4_route)."""
    ids: torch.Tensor
    weights: torch.Tensor
    offsets: torch.Tensor
    row_token: torch.Tensor
    token_rows: torch.Tensor


def route_raw(*args):
    """moe_fp4_route with raw pointers (C argument order); returns the status."""
    return lib().moe_fp4_route(*args)


def route_workspace_size(tokens: int, num_experts: int) -> int:
    """Device workspace bytes of route for these sizes."""
    return (_lib or lib()).moe_fp4_route_workspace_size(tokens, num_experts)


_SCORES = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}


def route(logits, topk: int, score: str = "softmax", bias=None, renormalize: bool = True,
          num_groups: int = 1, topk_groups: int | None = None, out: Routing | None = None,
          workspace=None, stream=None) -> Routing:
    """The router: gate logits (float32, bfloat16 or float16 CUDA tensor [tokens][E], unit
    column stride) to each token's topk experts, their weights and the routed rows
    grouped by expert.  score "softmax" or "sigmoid" (ranked by score + bias, float32
    [E]); num_groups / topk_groups limit the choice to the best groups of experts.
    Routing.offsets and .row_token are grouped_gemm's offsets and a_row_index,
    .token_rows and .weights combine's; .ids and .weights moe_ffn's.  New results and a new
    workspace belong to the launch stream; without a stream, workspace or out the five results
    share one allocation, which lives as long as any of them (clone one that is kept or saved
    alone)."""
    if (_calls or lib() and _calls) and stream is None and workspace is None and out is None and \
            isinstance(logits, torch.Tensor) and logits.is_cuda and score in _SCORES:
        dev = _current_device()
        got = _calls.route(logits, topk, _SCORES[score], bias, renormalize, num_groups,
                           num_groups if topk_groups is None else topk_groups, dev, _raw_stream(dev))
        if got is not None:
            return Routing(*got)
    if not isinstance(logits, torch.Tensor) or logits.dtype not in _IN_TYPES or logits.dim() != 2:
        raise ValueError("logits: expected a 2-D float32, bfloat16 or float16 tensor")
    if score not in _SCORES:
        raise ValueError(f"score: {score!r}, expected 'softmax' or 'sigmoid'")
    if topk < 1:
        raise ValueError(f"topk: {topk}, expected at least 1")
    T, E = logits.shape
    i32, f32 = torch.int32, torch.float32
    ld = _pitch(logits, "logits", logits.dtype, (T, E))
    if bias is not None:
        _exact(bias, "bias", f32, (E,))
    if out is None:
        new = logits.new_empty
        with _on(stream):
            ids, offsets = new((T, topk), dtype=i32), new(E + 1, dtype=i32)
            out = Routing(ids, new((T, topk), dtype=f32), offsets, new(T * topk, dtype=i32),
                          new((T, topk), dtype=i32))
    else:
        for t, name, dtype, shape in zip(out, Routing._fields, (i32, f32, i32, i32, i32),
                                         ((T, topk), (T, topk), (E + 1,), (T * topk,), (T, topk))):
            _exact(t, name, dtype, shape)
    need = route_workspace_size(T, E)
    if workspace is None:
        if need:
            with _on(stream):
                workspace = logits.new_empty(need, dtype=torch.uint8)
    else:
        _need(workspace, "workspace", torch.uint8, (_AtLeast(need),))
    dev = _same_cuda("logits bias ids weights offsets row_token token_rows workspace", logits, bias,
                     *out, workspace)
    st = (_lib or lib()).moe_fp4_route(
        logits.data_ptr(), _IN_TYPES[logits.dtype], T, E, ld, _SCORES[score],
        None if bias is None else bias.data_ptr(), 1 if renormalize else 0, topk, num_groups,
        num_groups if topk_groups is None else topk_groups, out.ids.data_ptr(), out.weights.data_ptr(),
        out.offsets.data_ptr(), out.row_token.data_ptr(), out.token_rows.data_ptr(),
        None if workspace is None else workspace.data_ptr(), need, _launch_stream(stream, dev))
    if st != OK:
        raise MoeFp4Error(st, "moe_fp4_route")
    return out
