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


def _bind():
    i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    rows = [vp, i64, i64]
    lib.chol_recurrence.argtypes = [i32, i32, i64, i64, i64, *rows, *rows, vp, vp, *rows, vp, sz, vp]
    lib.chol_recurrence_adjoint.argtypes = [i32, i32, i64, i64, i64, *rows, *rows, *rows, vp, vp, *rows, *rows, vp,
                                            vp, sz, vp]
    lib.chol_recurrence_workspace_size.argtypes = [i32, i64, i64, i64, ctypes.POINTER(sz)]


_bind()


def _code(t) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"expected float32, bfloat16 or float16, got {t.dtype}")
    return code


def _same(t, name: str, like, shape=None, dtype=None):
    """t is on like's device and has the given shape (default like's) and type (default like's)."""
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
            h = torch.empty((batch, length, dim), dtype=a.dtype, device=a.device)
        else:
            _same(h, "h", a)
        if hlast is None:
            hlast = torch.empty((batch, dim), dtype=torch.float32, device=a.device)
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
            adjA = torch.empty((batch, length, dim), dtype=a.dtype, device=a.device)
        else:
            _same(adjA, "adjA", a)
        if adjB is None:
            adjB = torch.empty((batch, length, dim), dtype=a.dtype, device=a.device)
        else:
            _same(adjB, "adjB", a)
        if adjH0 is None:
            adjH0 = torch.empty((batch, dim), dtype=torch.float32, device=a.device)
        ph0 = _state(h0, "h0", a, (batch, dim))
        pl, p0 = _state(adjHlast, "adjHlast", a, (batch, dim)), _state(adjH0, "adjH0", a, (batch, dim))
        need = chol_recurrence_workspace_size(code, batch, length, dim) if length > 1 else 0
        keep, ws, wbytes = _scratch(need, a.device, workspace)
        _check(lib.chol_recurrence_adjoint(code, g, batch, length, dim, *_seq(a, "a"), *_seq(h, "h"),
                                           *_seq(adjH, "adjH"), ph0, pl, *_seq(adjA, "adjA"), *_seq(adjB, "adjB"), p0,
                                           ws, wbytes, _raw_stream(a)))
    return adjA, adjB, adjH0
