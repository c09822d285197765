"""Binding of the operators of a selective state space language model: the short
causal convolution, the selective scan and the log probabilities of given tokens,
with their adjoints (``include/libchol.h``).

Like ``_train``: argument marshalling only.  Outputs and workspaces that are not
given are allocated on the stream the call runs on.  A call runs on the device
of its tensors.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import NamedTuple, Optional

import torch

from ._lib import _check, lib
from ._train import _code, _on, _ptr, _raw_stream, _rows, _same, _scratch, _seq

CONV_WIDTHS = (2, 3, 4)
SCAN_MAX_STATES = 64
LOGPROB_MAX_TOP = 32


def _bind():
    i64, i32, vp, sz, f32 = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
    rows, size = [vp, i64, i64], ctypes.POINTER(sz)
    lib.chol_causal_conv.argtypes = [i32, i32, i64, i64, i64, i64, *rows, vp, vp, vp, vp, *rows, vp]
    lib.chol_causal_conv_adjoint.argtypes = [i32, i32, i64, i64, i64, i64, *rows, vp, vp, vp, *rows, vp, *rows, vp, vp,
                                             i32, vp, vp, sz, vp]
    lib.chol_causal_conv_adjoint_workspace_size.argtypes = [i32, i64, i64, i64, i64, size]
    lib.chol_selective_scan.argtypes = [i32, ctypes.c_char_p, vp, sz, vp]
    lib.chol_selective_scan_adjoint.argtypes = [i32, ctypes.c_char_p, vp, sz, vp]
    lib.chol_selective_scan_workspace_size.argtypes = [i32, i64, i64, i64, i64, i64, size]
    lib.chol_selective_scan_block.argtypes = [i64]
    lib.chol_selective_scan_block.restype = i64
    lib.chol_token_logprob.argtypes = [i32, i64, i64, vp, i64, vp, f32, vp, vp, vp, i64, vp, vp, vp, sz, vp]
    lib.chol_token_logprob_workspace_size.argtypes = [i32, i64, i64, i64, size]
    lib.chol_token_logprob_adjoint.argtypes = [i32, i64, i64, vp, i64, vp, f32, vp, vp, vp, vp, vp, i64, vp]


_bind()


def _like(t, name, like, shape=None, dtype=None):
    """t, checked, or a new tensor of that shape (default like's) and type (default like's)."""
    if t is None:
        return torch.empty_like(like) if shape is None else like.new_empty(shape, dtype=dtype)
    _same(t, name, like, shape, dtype)
    return t


def _whole(t, name, like, shape, dtype=None):
    """Pointer of a contiguous tensor of that shape and type (default like's); 0 for None."""
    if t is None:
        return 0
    if dtype is None:
        dtype = like.dtype
    if t.dtype is dtype and t.shape == shape and t.get_device() == like.get_device() and t.is_contiguous():
        return t.data_ptr()
    _same(t, name, like, shape, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _f32(t, name, like, shape):
    return _whole(t, name, like, shape, torch.float32)


def _steps(t, name, like):
    """(pointer, ld, stride) of a [batch, len, dim] array of like's shape and type."""
    if t is like or (t.dtype is like.dtype and t.shape == like.shape and t.get_device() == like.get_device()):
        return _seq(t, name)
    _same(t, name, like)
    return _seq(t, name)


# ------------------------------------------------------------- convolution ----

def _conv_sizes(x, w):
    if x.dim() != 3:
        raise ValueError("x must be [batch, len, dim]")
    if w.dim() != 2 or w.shape[1] not in CONV_WIDTHS:
        raise ValueError(f"w must be [dim, width] with a width of {CONV_WIDTHS}, got {tuple(w.shape)}")
    return (*x.shape, w.shape[1])


@functools.lru_cache(maxsize=1024)
def chol_causal_conv_adjoint_workspace_size(dtype_code: int, batch: int, length: int, dim: int, width: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib.chol_causal_conv_adjoint_workspace_size(dtype_code, batch, length, dim, width, ctypes.byref(out)))
    return int(out.value)


def chol_causal_conv(x, w, bias=None, state=None, last=None, y=None, silu: bool = True, stream=None):
    """y_t = silu(bias + sum_k w_k x_{t-width+1+k}) over [batch, len, dim]: returns (y, last).

    ``w`` [dim, width], width 2 to 4.  ``state`` ([batch, width - 1, dim], None is
    zeros) holds the rows before the first; ``last``, the last rows, may be ``state``
    (kept rows, updated in place).  ``silu`` False leaves out the activation."""
    code = _code(x)
    batch, length, dim, width = _conv_sizes(x, w)
    pw, pb = _whole(w, "w", x, (dim, width)), _whole(bias, "bias", x, (dim,))
    kept = (batch, width - 1, dim)
    with _on(x, stream):
        if y is None:
            y = torch.empty_like(x)
        if last is None:
            last = x.new_empty(kept)
        _check(lib.chol_causal_conv(code, silu, batch, length, dim, width, *_seq(x, "x"), pw, pb,
                                    _whole(state, "state", x, kept), _whole(last, "last", x, kept), *_steps(y, "y", x),
                                    _raw_stream(x)))
    return y, last


def chol_causal_conv_adjoint(x, w, adj, bias=None, state=None, adjLast=None, silu: bool = True, adjX=None, adjW=None,
                             adjBias=None, adjState=None, accumulate: bool = False, workspace=None, stream=None):
    """Adjoint of chol_causal_conv: returns (adjX, adjW, adjBias, adjState); adjBias is
    None without a bias and adjState None without a state, unless they are given.

    adjW and adjBias are fp32 and added to with ``accumulate``."""
    code = _code(x)
    batch, length, dim, width = _conv_sizes(x, w)
    pw, pb = _whole(w, "w", x, (dim, width)), _whole(bias, "bias", x, (dim,))
    _same(adj, "adj", x)
    kept = (batch, width - 1, dim)
    with _on(x, stream):
        adjX = _like(adjX, "adjX", x)
        new = x.new_zeros if accumulate else x.new_empty
        if adjW is None:
            adjW = new((dim, width), dtype=torch.float32)
        if adjBias is None and bias is not None:
            adjBias = new((dim,), dtype=torch.float32)
        if adjState is None and state is not None:
            adjState = torch.empty_like(state)
        keep, ws, wbytes = _scratch(chol_causal_conv_adjoint_workspace_size(code, batch, length, dim, width), x.device,
                                    workspace)
        _check(lib.chol_causal_conv_adjoint(
            code, silu, batch, length, dim, width, *_seq(x, "x"), pw, pb, _whole(state, "state", x, kept),
            *_seq(adj, "adj"), _whole(adjLast, "adjLast", x, kept), *_seq(adjX, "adjX"),
            _f32(adjW, "adjW", x, (dim, width)), _f32(adjBias, "adjBias", x, (dim,)), accumulate,
            _whole(adjState, "adjState", x, kept), ws, wbytes, _raw_stream(x)))
    return adjX, adjW, adjBias, adjState


# -------------------------------------------------------------------- scan ----

# chol_scan_args: sizes, flags, six arrays, A D bias h0 hlast starts, six arrays, adj_hlast, adj_A adj_D adj_bias adj_h0
_ARGS = struct.Struct("@5q2i" + 6 * "Pqq" + "6P" + 6 * "Pqq" + "5P")
_NO_ROWS = (0, 0, 0)
_NO_ADJOINT = (0,) * 23


@functools.lru_cache(maxsize=1024)
def chol_selective_scan_workspace_size(adjoint: bool, batch: int, length: int, dim: int, groups: int, states: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib.chol_selective_scan_workspace_size(int(adjoint), batch, length, dim, groups, states, ctypes.byref(out)))
    return int(out.value)


@functools.lru_cache(maxsize=1024)
def chol_selective_scan_block(states: int) -> int:
    """Steps between two of the states that a forward call saves."""
    block = int(lib.chol_selective_scan_block(states))
    if block < 0:
        raise ValueError(f"states must be 1 to {SCAN_MAX_STATES}, got {states}")
    return block


def _mixed(t, name):
    """(pointer, ld, stride) of B or C, [batch, len, states] or [batch, len, groups, states]."""
    if t.dim() == 3:
        return _seq(t, name)
    batch, length, groups, states = t.shape
    if t.is_contiguous():
        return t.data_ptr(), groups * states, length * groups * states
    sb, st, sg, sn = t.stride()
    if (states > 1 and sn != 1) or (groups > 1 and sg != states):
        raise ValueError(f"{name} must have its groups and states contiguous")
    if length <= 1:
        st = groups * states
    if batch <= 1:
        sb = st * max(length, 1)
    return t.data_ptr(), st, sb


def _scan_sizes(u, delta, A, B, C):
    if u.dim() != 3:
        raise ValueError("u must be [batch, len, dim]")
    batch, length, dim = u.shape
    if A.dim() != 2 or A.shape[0] != dim:
        raise ValueError(f"A must be [dim, states], got {tuple(A.shape)}")
    states = A.shape[1]
    if not 1 <= states <= SCAN_MAX_STATES:
        raise ValueError(f"A must have 1 to {SCAN_MAX_STATES} states, got {states}")
    if B.dim() == 4:
        groups = B.shape[2]
        if groups < 1 or dim % groups:
            raise ValueError(f"{groups} groups do not divide {dim} channels")
        _same(B, "B", u, (batch, length, groups, states))
    else:
        groups = 1
        _same(B, "B", u, (batch, length, states))
    _same(C, "C", B)
    return batch, length, dim, groups, states


def chol_selective_scan(u, delta, A, B, C, D=None, z=None, bias=None, h0=None, hlast=None, y=None, starts=None,
                        save: bool = False, softplus: bool = True, workspace=None, stream=None):
    """h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t, y_t = (C_t h_t + D u_t) silu(z_t), with dt =
    softplus(delta + bias), over [batch, len, dim]: returns (y, hlast, starts).

    ``A`` fp32 [dim, states]; ``B`` and ``C`` [batch, len, states], or [batch, len, groups,
    states] for groups of dim / groups channels each; ``D`` and ``bias`` fp32 [dim]; ``z``
    gates the output.  ``h0`` (fp32 [batch, dim, states], None is zero) is the state before
    the first step; ``hlast`` may be ``h0`` (a kept state, updated in place); ``y`` may be
    ``u``, ``delta`` or ``z``.  ``save``, or a ``starts`` tensor (fp32 [batch, ceil(len /
    block), dim, states]), keeps the states that the adjoint starts from."""
    code = _code(u)
    batch, length, dim, groups, states = _scan_sizes(u, delta, A, B, C)
    with _on(u, stream):
        if y is None:
            y = torch.empty_like(u)
        shape = (batch, dim, states)
        if hlast is None:
            hlast = u.new_empty(shape, dtype=torch.float32)
        if save or starts is not None:
            starts = _like(starts, "starts", u, (batch, -(-length // chol_selective_scan_block(states)), dim, states),
                           torch.float32)
        args = _ARGS.pack(
            batch, length, dim, groups, states, softplus, 0, *_seq(u, "u"), *_steps(delta, "delta", u), *_mixed(B, "B"),
            *_mixed(C, "C"), *(_NO_ROWS if z is None else _steps(z, "z", u)), *_steps(y, "y", u),
            _f32(A, "A", u, (dim, states)), _f32(D, "D", u, (dim,)), _f32(bias, "bias", u, (dim,)), _f32(h0, "h0", u, shape),
            _f32(hlast, "hlast", u, shape), 0 if starts is None else _f32(starts, "starts", u, starts.shape), *_NO_ADJOINT)
        need = chol_selective_scan_workspace_size(False, batch, length, dim, groups, states) if length > 1 else 0
        keep, ws, wbytes = _scratch(need, u.device, workspace)
        _check(lib.chol_selective_scan(code, args, ws, wbytes, _raw_stream(u)))
    return y, hlast, starts


def chol_selective_scan_adjoint(u, delta, A, B, C, starts, adj, D=None, z=None, bias=None, adjHlast=None, adjU=None,
                                adjDelta=None, adjA=None, adjB=None, adjC=None, adjD=None, adjZ=None, adjBias=None,
                                adjH0=None, accumulate: bool = False, softplus: bool = True, workspace=None,
                                stream=None):
    """Adjoint of chol_selective_scan: returns (adjU, adjDelta, adjA, adjB, adjC, adjD, adjZ,
    adjBias, adjH0).  adjD, adjZ and adjBias are None without D, z and bias.

    ``starts`` is what the forward call saved.  adjU, adjDelta and adjZ may be u, delta and
    z themselves, or one of them ``adj``; adjB and adjC may be B and C; ``adjH0`` may be
    ``adjHlast``.  adjA, adjD and adjBias are fp32 and added to with ``accumulate``."""
    code = _code(u)
    batch, length, dim, groups, states = _scan_sizes(u, delta, A, B, C)
    blocks = -(-length // chol_selective_scan_block(states))
    with _on(u, stream):
        if adjU is None:
            adjU = torch.empty_like(u)
        if adjDelta is None:
            adjDelta = torch.empty_like(u)
        adjB, adjC = _like(adjB, "adjB", B), _like(adjC, "adjC", C)
        if z is not None:
            adjZ = torch.empty_like(u) if adjZ is None else adjZ
        elif adjZ is not None:
            raise ValueError("adjZ needs z")
        new = u.new_zeros if accumulate else u.new_empty
        if adjA is None:
            adjA = new((dim, states), dtype=torch.float32)
        if adjD is None and D is not None:
            adjD = new((dim,), dtype=torch.float32)
        if adjBias is None and bias is not None:
            adjBias = new((dim,), dtype=torch.float32)
        shape = (batch, dim, states)
        if adjH0 is None:
            adjH0 = u.new_empty(shape, dtype=torch.float32)
        args = _ARGS.pack(
            batch, length, dim, groups, states, softplus, accumulate, *_seq(u, "u"), *_steps(delta, "delta", u),
            *_mixed(B, "B"), *_mixed(C, "C"), *(_NO_ROWS if z is None else _steps(z, "z", u)), *_NO_ROWS,
            _f32(A, "A", u, (dim, states)), _f32(D, "D", u, (dim,)), _f32(bias, "bias", u, (dim,)), 0, 0,
            _f32(starts, "starts", u, (batch, blocks, dim, states)), *_steps(adj, "adj", u), *_steps(adjU, "adjU", u),
            *_steps(adjDelta, "adjDelta", u), *_mixed(adjB, "adjB"), *_mixed(adjC, "adjC"),
            *(_NO_ROWS if z is None else _steps(adjZ, "adjZ", u)), _f32(adjHlast, "adjHlast", u, shape),
            _f32(adjA, "adjA", u, (dim, states)), _f32(adjD, "adjD", u, (dim,)), _f32(adjBias, "adjBias", u, (dim,)),
            _f32(adjH0, "adjH0", u, shape))
        need = chol_selective_scan_workspace_size(True, batch, length, dim, groups, states)
        keep, ws, wbytes = _scratch(need, u.device, workspace)
        _check(lib.chol_selective_scan_adjoint(code, args, ws, wbytes, _raw_stream(u)))
    return adjU, adjDelta, adjA, adjB, adjC, adjD, adjZ, adjBias, adjH0


# ------------------------------------------------------- log probabilities ----

class TokenLogprob(NamedTuple):
    """Of every row: the given token's log probability, the logarithm of the sum over
    the vocabulary, the entropy, and the most likely columns with their log probabilities."""
    logp: torch.Tensor
    lse: torch.Tensor
    entropy: Optional[torch.Tensor]
    top_ids: Optional[torch.Tensor]
    top_logp: Optional[torch.Tensor]


def _logits(x, tokens):
    if x.dim() != 2:
        raise ValueError("logits must be [rows, vocab]")
    _same(tokens, "tokens", x, (x.shape[0],), torch.int64)
    if not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous")
    return x.shape


@functools.lru_cache(maxsize=1024)
def chol_token_logprob_workspace_size(dtype_code: int, rows: int, vocab: int, top: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib.chol_token_logprob_workspace_size(dtype_code, rows, vocab, top, ctypes.byref(out)))
    return int(out.value)


def chol_token_logprob(logits, tokens, scale: float = 1.0, top: int = 0, entropy: bool = True, workspace=None,
                       stream=None) -> TokenLogprob:
    """Log probabilities of ``tokens`` (int64 [rows]; outside the vocabulary: none, 0) under
    the rows of ``scale`` times ``logits`` [rows, vocab], with the entropy (unless False)
    and the ``top`` most likely columns, the lowest first among equal ones."""
    code = _code(logits)
    rows, vocab = _logits(logits, tokens)
    if not 0 <= top <= min(vocab, LOGPROB_MAX_TOP):
        raise ValueError(f"top must be 0 to {min(vocab, LOGPROB_MAX_TOP)}, got {top}")
    with _on(logits, stream):
        px, ldx = _rows(logits, "logits")
        logp, lse, *h = logits.new_empty((3 if entropy else 2, rows), dtype=torch.float32).unbind(0)
        h = h[0] if entropy else None
        ids = top_logp = None
        if top:
            ids = logits.new_empty((rows, top), dtype=torch.int64)
            top_logp = logits.new_empty((rows, top), dtype=torch.float32)
        keep, ws, wbytes = _scratch(chol_token_logprob_workspace_size(code, rows, vocab, top), logits.device, workspace)
        _check(lib.chol_token_logprob(code, rows, vocab, px, ldx, tokens.data_ptr(), scale, logp.data_ptr(),
                                      lse.data_ptr(), _ptr(h), top, _ptr(top_logp), _ptr(ids), ws, wbytes,
                                      _raw_stream(logits)))
    return TokenLogprob(logp, lse, h, ids, top_logp)


def chol_token_logprob_adjoint(logits, tokens, lse, adjLogp=None, entropy=None, adjEntropy=None, scale: float = 1.0,
                               adjLogits=None, stream=None):
    """Gradient of chol_token_logprob's logp and entropy with respect to the logits.

    ``lse`` and ``entropy`` (needed with ``adjEntropy``) are what the forward call
    returned; ``adjLogits`` may be ``logits``."""
    code = _code(logits)
    rows, vocab = _logits(logits, tokens)
    if adjEntropy is not None and entropy is None:
        raise ValueError("adjEntropy needs entropy")
    with _on(logits, stream):
        adjLogits = _like(adjLogits, "adjLogits", logits)
        px, ldx = _rows(logits, "logits")
        pa, lda = _rows(adjLogits, "adjLogits")
        _check(lib.chol_token_logprob_adjoint(
            code, rows, vocab, px, ldx, tokens.data_ptr(), scale, _f32(lse, "lse", logits, (rows,)),
            _f32(entropy, "entropy", logits, (rows,)), _f32(adjLogp, "adjLogp", logits, (rows,)),
            _f32(adjEntropy, "adjEntropy", logits, (rows,)), pa, lda, _raw_stream(logits)))
    return adjLogits
