"""Binding of the training-step operators: the gated linear recurrence, the RMS
norm and the AdamW step, with their adjoints (``include/libchol.h``).

Like ``_lib``: argument marshalling only.  Outputs and workspaces that are not
given are allocated on the stream the call runs on.  A call runs on the device
of its tensors.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from ._lib import CHOL_F32, _check, lib

CHOL_BF16, CHOL_F16 = 4, 5
GATES = {"linear": 0, "log": 1}
_CODES = {torch.float32: CHOL_F32, torch.bfloat16: CHOL_BF16, torch.float16: CHOL_F16}


class AdamwTensor(ctypes.Structure):
    """chol_adamw_tensor"""
    _fields_ = [(k, ctypes.c_void_p) for k in ("p", "g", "m", "v", "master", "m_scale", "v_scale")] + \
               [(k, ctypes.c_int64) for k in ("n", "first")]


def _bind():
    i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    rows = [vp, i64, i64]
    lib.chol_recurrence.argtypes = [i32, i32, i64, i64, i64, *rows, *rows, vp, vp, *rows, vp, sz, vp]
    lib.chol_recurrence_adjoint.argtypes = [i32, i32, i64, i64, i64, *rows, *rows, *rows, vp, vp, *rows, *rows, vp,
                                            vp, sz, vp]
    lib.chol_recurrence_workspace_size.argtypes = [i32, i64, i64, i64, ctypes.POINTER(sz)]
    lib.chol_rmsnorm.argtypes = [i32, i64, i64, vp, i64, vp, i64, vp, ctypes.c_float, vp, i64, vp, i64, vp]
    lib.chol_rmsnorm_quant.argtypes = [i32, i64, i64, i64, vp, i64, vp, i64, vp, ctypes.c_float, vp, i64, vp, i64, vp,
                                       i64, vp]
    lib.chol_rmsnorm_adjoint.argtypes = [i32, i64, i64, vp, i64, vp, vp, i64, vp, i64, ctypes.c_float, vp, i64, vp,
                                         i32, vp, sz, vp]
    lib.chol_rmsnorm_adjoint_workspace_size.argtypes = [i32, i64, i64, ctypes.POINTER(sz)]
    f64 = ctypes.c_double
    lib.chol_adamw_list.argtypes = [i32, i32, i64, ctypes.POINTER(AdamwTensor), vp, sz, ctypes.POINTER(i64),
                                    ctypes.POINTER(sz)]
    lib.chol_adamw.argtypes = [i32, i32, i32, i64, vp, vp, f64, f64, f64, f64, f64, i64, ctypes.c_uint32, vp]


_bind()


def _code(t) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"expected float32, bfloat16 or float16, got {t.dtype}")
    return code


def _same(t, name: str, like, shape=None, dtype=None):
    """t is on like's device and has the given shape (default like's) and type (default like's)."""
    if t.shape == (like.shape if shape is None else shape) and t.dtype is (like.dtype if dtype is None else dtype) \
            and t.device == like.device:
        return
    if t.device != like.device:
        raise ValueError(f"{name} must live on {like.device}, got {t.device}")
    if t.dtype != (like.dtype if dtype is None else dtype):
        raise TypeError(f"{name} must be {like.dtype if dtype is None else dtype}, got {t.dtype}")
    if t.shape != (like.shape if shape is None else shape):
        raise ValueError(f"{name} must have shape {tuple(like.shape if shape is None else shape)}, got {tuple(t.shape)}")


@contextlib.contextmanager
def _switched(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


_HERE = contextlib.nullcontext()


def _on(t, stream):
    """Context in which allocations and launches go to t's device and to `stream` (default: its current stream)."""
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    if stream is None and t.get_device() == torch.cuda.current_device():
        return _HERE
    return _switched(t.device, stream)


def _raw_stream(t) -> int:
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _scratch(need: int, device, workspace):
    """(tensor to keep until the call returns, pointer, bytes)"""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif workspace.device != device:
        raise ValueError(f"workspace must live on {device}")
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


# ------------------------------------------------------------- recurrence ----

def _seq(t, name: str):
    """(pointer, ld, stride) of a [batch, len, dim] array with unit channel stride."""
    batch, length, dim = t.shape
    if t.is_contiguous():
        return t.data_ptr(), dim, length * dim
    sb, st, sc = t.stride()
    if dim > 1 and sc != 1:
        raise ValueError(f"{name} must have unit channel stride")
    if length <= 1:
        st = max(dim, 1)
    if batch <= 1:
        sb = st * max(length, 1)
    return t.data_ptr(), st, sb


def _state(t, name: str, like, shape):
    if t is None:
        return None
    _same(t, name, like, shape, torch.float32)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _gate(gate: str) -> int:
    code = GATES.get(gate)
    if code is None:
        raise ValueError(f"gate must be 'linear' or 'log', got {gate!r}")
    return code


def chol_recurrence_workspace_size(dtype_code: int, batch: int, length: int, dim: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib.chol_recurrence_workspace_size(dtype_code, batch, length, dim, ctypes.byref(out)))
    return int(out.value)


def chol_recurrence(a, b, h0=None, hlast=None, h=None, gate: str = "linear", workspace=None, stream=None):
    """h_t = a_t h_{t-1} + b_t over [batch, len, dim]: returns (h, hlast).

    ``gate`` "log": a holds log a_t.  ``h0`` (fp32 [batch, dim], None is zero) is
    the state before the first step; ``hlast`` may be ``h0`` (a kept state,
    updated in place); ``h`` may be ``a`` or ``b``."""
    if a.dim() != 3:
        raise ValueError("a must be [batch, len, dim]")
    code, g = _code(a), _gate(gate)
    _same(b, "b", a)
    batch, length, dim = a.shape
    with _on(a, stream):
        if h is None:
            h = torch.empty_like(a)
        else:
            _same(h, "h", a)
        if hlast is None:
            hlast = a.new_empty((batch, dim), dtype=torch.float32)
        ph0, pl = _state(h0, "h0", a, (batch, dim)), _state(hlast, "hlast", a, (batch, dim))
        need = chol_recurrence_workspace_size(code, batch, length, dim) if length > 1 else 0
        keep, ws, wbytes = _scratch(need, a.device, workspace)
        _check(lib.chol_recurrence(code, g, batch, length, dim, *_seq(a, "a"), *_seq(b, "b"), ph0, pl, *_seq(h, "h"),
                                   ws, wbytes, _raw_stream(a)))
    return h, hlast


def chol_recurrence_adjoint(a, h, adjH, h0=None, adjHlast=None, adjA=None, adjB=None, adjH0=None,
                            gate: str = "linear", workspace=None, stream=None):
    """Adjoint of chol_recurrence: returns (adjA, adjB, adjH0).

    ``h`` is what the forward call wrote; ``adjA`` is the gradient of a as it is
    stored (of log a_t for gate "log").  ``adjA`` and ``adjB`` may be ``a`` or
    ``adjH``; ``adjH0`` may be ``adjHlast``."""
    if a.dim() != 3:
        raise ValueError("a must be [batch, len, dim]")
    code, g = _code(a), _gate(gate)
    _same(h, "h", a)
    _same(adjH, "adjH", a)
    batch, length, dim = a.shape
    with _on(a, stream):
        if adjA is None:
            adjA = torch.empty_like(a)
        else:
            _same(adjA, "adjA", a)
        if adjB is None:
            adjB = torch.empty_like(a)
        else:
            _same(adjB, "adjB", a)
        if adjH0 is None:
            adjH0 = a.new_empty((batch, dim), dtype=torch.float32)
        ph0 = _state(h0, "h0", a, (batch, dim))
        pl, p0 = _state(adjHlast, "adjHlast", a, (batch, dim)), _state(adjH0, "adjH0", a, (batch, dim))
        need = chol_recurrence_workspace_size(code, batch, length, dim) if length > 1 else 0
        keep, ws, wbytes = _scratch(need, a.device, workspace)
        _check(lib.chol_recurrence_adjoint(code, g, batch, length, dim, *_seq(a, "a"), *_seq(h, "h"),
                                           *_seq(adjH, "adjH"), ph0, pl, *_seq(adjA, "adjA"), *_seq(adjB, "adjB"), p0,
                                           ws, wbytes, _raw_stream(a)))
    return adjA, adjB, adjH0


# ---------------------------------------------------------------- RMS norm ----

RMSNORM_GROUPS = (0, 32, 64, 128, 256)


def _rows(t, name: str):
    """(pointer, ld) of a [rows, cols] array with unit column stride, or of any
    contiguous array taken as rows of its last dimension."""
    if t.is_contiguous():
        return t.data_ptr(), t.shape[-1]
    if t.dim() == 2:
        ld, sc = t.stride()
        rows, cols = t.shape
        if cols > 1 and sc != 1:
            raise ValueError(f"{name} must have unit column stride")
        return t.data_ptr(), ld if rows > 1 else cols
    raise ValueError(f"{name} must be [rows, cols] or contiguous")


def _row_shape(x, w):
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    cols = x.shape[-1]
    _same(w, "w", x, (cols,))
    if not w.is_contiguous():
        raise ValueError("w must be contiguous")
    return (x.shape[0] if x.dim() == 2 else x.numel() // cols if cols else 0), cols


def chol_rmsnorm(x, w, residual=None, eps: float = 1e-6, y=None, h=None, stream=None):
    """y = h w / sqrt(mean(h^2) + eps) over the last dimension, h = x + residual:
    returns (y, h), where h is x itself without a residual.  ``y`` or ``h`` may
    be ``x`` or ``residual`` (in place)."""
    code = _code(x)
    rows, cols = _row_shape(x, w)
    with _on(x, stream):
        px, ldx = _rows(x, "x")
        if y is None:
            y = torch.empty_like(x)
        else:
            _same(y, "y", x)
        py, ldy = _rows(y, "y")
        pr = ph = None
        ldr = ldh = cols
        if residual is None:
            h = x
        else:
            _same(residual, "residual", x)
            pr, ldr = _rows(residual, "residual")
            if h is None:
                h = torch.empty_like(x)
            else:
                _same(h, "h", x)
            ph, ldh = _rows(h, "h")
        _check(lib.chol_rmsnorm(code, rows, cols, px, ldx, pr, ldr, w.data_ptr(), eps, py, ldy, ph, ldh,
                                _raw_stream(x)))
    return y, h


def chol_rmsnorm_quant(x, w, residual=None, group: int = 0, eps: float = 1e-6, q=None, scale=None, h=None,
                       stream=None):
    """chol_rmsnorm with y as float8_e4m3fn and fp32 scales, one for every
    ``group`` columns (0: one a row): returns (q, scale, h) with y ~ q * scale.
    ``scale`` is [rows, ceil(cols / group)]."""
    code = _code(x)
    rows, cols = _row_shape(x, w)
    if group not in RMSNORM_GROUPS:
        raise ValueError(f"group must be one of {RMSNORM_GROUPS}, got {group}")
    groups = -(-cols // group) if group else 1
    with _on(x, stream):
        px, ldx = _rows(x, "x")
        if q is None:
            q = torch.empty_like(x, dtype=torch.float8_e4m3fn)
        else:
            _same(q, "q", x, dtype=torch.float8_e4m3fn)
        if scale is None:
            scale = x.new_empty((rows, groups), dtype=torch.float32)
        else:
            _same(scale, "scale", x, (rows, groups), torch.float32)
        pq, ldq = _rows(q, "q")
        ps, lds = _rows(scale, "scale")
        pr = ph = None
        ldr = ldh = cols
        if residual is None:
            h = x
        else:
            _same(residual, "residual", x)
            pr, ldr = _rows(residual, "residual")
            if h is None:
                h = torch.empty_like(x)
            else:
                _same(h, "h", x)
            ph, ldh = _rows(h, "h")
        _check(lib.chol_rmsnorm_quant(code, rows, cols, group, px, ldx, pr, ldr, w.data_ptr(), eps, pq, ldq, ps, lds,
                                      ph, ldh, _raw_stream(x)))
    return q, scale, h


def chol_rmsnorm_adjoint_workspace_size(dtype_code: int, rows: int, cols: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib.chol_rmsnorm_adjoint_workspace_size(dtype_code, rows, cols, ctypes.byref(out)))
    return int(out.value)


def chol_rmsnorm_adjoint(h, w, adj, adjH=None, eps: float = 1e-6, adjX=None, adjW=None, accumulate: bool = False,
                         workspace=None, stream=None):
    """Adjoint of chol_rmsnorm: returns (adjX, adjW).  ``adj`` is the gradient of
    y, ``adjH`` the one that reaches h past the norm; adjX is the gradient of h, so
    of x and of the residual.  ``adjW`` (fp32) is added to with ``accumulate``."""
    code = _code(h)
    rows, cols = _row_shape(h, w)
    _same(adj, "adj", h)
    with _on(h, stream):
        if adjX is None:
            adjX = torch.empty_like(h)
        else:
            _same(adjX, "adjX", h)
        if adjW is None:
            adjW = (h.new_zeros if accumulate else h.new_empty)((cols,), dtype=torch.float32)
        else:
            _state(adjW, "adjW", h, (cols,))
        ph, ldh = _rows(h, "h")
        pa, lda = _rows(adj, "adj")
        pg, ldg = None, cols
        if adjH is not None:
            _same(adjH, "adjH", h)
            pg, ldg = _rows(adjH, "adjH")
        px, ldx = _rows(adjX, "adjX")
        keep, ws, wbytes = _scratch(chol_rmsnorm_adjoint_workspace_size(code, rows, cols), h.device, workspace)
        _check(lib.chol_rmsnorm_adjoint(code, rows, cols, ph, ldh, w.data_ptr(), pa, lda, pg, ldg, eps, px, ldx,
                                        adjW.data_ptr(), 1 if accumulate else 0, ws, wbytes, _raw_stream(h)))
    return adjX, adjW


# ------------------------------------------------------------------- AdamW ----

ADAMW_TILE = 256


class AdamwList:
    """The tensors of an AdamW step and their work list on the device.  Holds the
    tensors, whose memory the list addresses."""

    def __init__(self, code, bits, master, chunks, table, tensors):
        self.code, self.bits, self.master, self.chunks = code, bits, master, chunks
        self.table, self.tensors = table, tensors


def chol_adamw_list(p, g, m, v, master=None, m_scale=None, v_scale=None, first=None) -> AdamwList:
    """The work list of chol_adamw, made once for lists of contiguous tensors.

    p, g: weights and gradients of one type.  m, v: states, all float32, or all
    float8_e4m3fn with ``m_scale`` and ``v_scale`` (fp32, one for every 256
    elements; v then holds the root of the second moment).  ``master``: fp32
    weights that p is the rounding of.  ``first``: each tensor's position in the
    random sequence (default: one after the other, each rounded up to 256)."""
    p, g, m, v = list(p), list(g), list(m), list(v)
    if not p:
        raise ValueError("the list has no tensors")
    if len(m) != len(p):
        raise ValueError(f"m has {len(m)} tensors for {len(p)}")
    bits = {torch.float32: 32, torch.float8_e4m3fn: 8}.get(m[0].dtype)
    if bits is None:
        raise TypeError(f"states must be float32 or float8_e4m3fn, got {m[0].dtype}")
    if bits == 8 and (m_scale is None or v_scale is None):
        raise ValueError("8-bit states need m_scale and v_scale")
    if bits == 32 and (m_scale is not None or v_scale is not None):
        raise ValueError("32-bit states take no scales")
    code = _code(p[0])
    if not p[0].is_cuda:
        raise ValueError("tensors must live on the GPU")
    columns = {"p": (p, p[0].dtype), "g": (g, p[0].dtype), "m": (m, m[0].dtype), "v": (v, m[0].dtype)}
    for name, given in (("master", master), ("m_scale", m_scale), ("v_scale", v_scale)):
        if given is not None:
            columns[name] = (list(given), torch.float32)
    if first is not None:
        first = list(first)
        if len(first) != len(p):
            raise ValueError(f"first has {len(first)} entries for {len(p)} tensors")
    device, sizes = p[0].device, [t.numel() for t in p]
    tiles = [-(-n // ADAMW_TILE) for n in sizes]
    for name, (tensors, dtype) in columns.items():
        if len(tensors) != len(p):
            raise ValueError(f"{name} has {len(tensors)} tensors for {len(p)}")
        counts = tiles if name.endswith("_scale") else sizes
        for i, t in enumerate(tensors):
            if t.dtype is not dtype or t.device != device:
                _same(t, f"{name}[{i}]", p[0], t.shape, dtype)
            if t.numel() != counts[i]:
                raise ValueError(f"{name}[{i}] has {t.numel()} elements for {sizes[i]} weights")
            if not t.is_contiguous():
                raise ValueError(f"{name}[{i}] must be contiguous")
    if first is None:
        first, at = [], 0
        for n in tiles:
            first.append(at)
            at += n * ADAMW_TILE
    none = [None] * len(p)
    pointers = [[t.data_ptr() for t in columns[k][0]] if k in columns else none
                for k in ("p", "g", "m", "v", "master", "m_scale", "v_scale")]
    items = (AdamwTensor * len(p))(*zip(*pointers, sizes, first))
    chunks, size = ctypes.c_int64(0), ctypes.c_size_t(0)
    _check(lib.chol_adamw_list(code, bits, len(p), items, None, 0, ctypes.byref(chunks), ctypes.byref(size)))
    host = torch.empty(max(size.value, 8), dtype=torch.uint8)
    _check(lib.chol_adamw_list(code, bits, len(p), items, host.data_ptr(), host.numel(), ctypes.byref(chunks),
                               ctypes.byref(size)))
    return AdamwList(code, bits, int(master is not None), chunks.value, host.to(p[0].device),
                     [c[0] for c in columns.values()])


def chol_adamw(tensors: AdamwList, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
               weight_decay: float = 0.0, grad_scale=None, seed: int = 0, stream=None) -> None:
    """One AdamW step over the list, in place.  ``grad_scale``: fp32 device tensor
    of one element that gradients are multiplied by.  ``seed``: this step's random
    roundings of 8-bit states (another one each step)."""
    if grad_scale is not None:
        if grad_scale.numel() != 1:
            raise ValueError("grad_scale must have one element")
        _same(grad_scale, "grad_scale", tensors.table, grad_scale.shape, torch.float32)
    with _on(tensors.table, stream):
        _check(lib.chol_adamw(tensors.code, tensors.bits, tensors.master, tensors.chunks, tensors.table.data_ptr(),
                              _ptr(grad_scale), lr, beta1, beta2, eps, weight_decay, step, seed & 0xFFFFFFFF,
                              _raw_stream(tensors.table)))
