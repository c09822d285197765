"""Argument checks of the training-step operators, on the CPU: the C-ABI refuses
on the host before anything is launched, and the binding refuses what it cannot
pass on."""
import ctypes

import pytest

dc = pytest.importorskip("differentiable_cholesky_amd")
torch = pytest.importorskip("torch")
from differentiable_cholesky_amd import _lib  # noqa: E402

lib = _lib.lib
F32, F64, BF16, F16 = _lib.CHOL_F32, _lib.CHOL_F64, dc.CHOL_BF16, dc.CHOL_F16
OK, INVALID, NOTSUP, WS = (_lib.CHOL_OK, _lib.CHOL_ERR_INVALID_VALUE, _lib.CHOL_ERR_NOT_SUPPORTED,
                           _lib.CHOL_ERR_WORKSPACE)
P = [k << 32 for k in range(1, 12)]   # addresses that are never read: every call below fails a check first


def need(dt, batch, length, dim):
    out = ctypes.c_size_t(0)
    s = lib.chol_recurrence_workspace_size(dt, batch, length, dim, ctypes.byref(out))
    return s, out.value


def forward(dt=BF16, gate=0, batch=2, length=100, dim=64, a=(P[0], 64, 6400), b=(P[1], 64, 6400), h0=P[2], last=P[3],
            h=(P[4], 64, 6400), ws=P[5], wbytes=1 << 40):
    return lib.chol_recurrence(dt, gate, batch, length, dim, *a, *b, h0, last, *h, ws, wbytes, None)


def adjoint(dt=BF16, gate=0, batch=2, length=100, dim=64, a=(P[0], 64, 6400), h=(P[1], 64, 6400), adj=(P[2], 64, 6400),
            h0=P[3], last=P[4], da=(P[5], 64, 6400), db=(P[6], 64, 6400), d0=P[7], ws=P[8], wbytes=1 << 40):
    return lib.chol_recurrence_adjoint(dt, gate, batch, length, dim, *a, *h, *adj, h0, last, *da, *db, d0, ws, wbytes,
                                       None)


def test_recurrence_workspace_size():
    assert need(BF16, 4, 1, 100) == (OK, 0)
    assert need(F32, 0, 10, 10) == (OK, 0)
    s, n = need(F32, 1, 1 << 16, 64)
    assert s == OK and n > 0
    assert need(F64, 1, 10, 10)[0] == INVALID
    assert need(F32, -1, 10, 10)[0] == INVALID
    assert need(F32, 1 << 20, 10, 1 << 20)[0] == NOTSUP
    assert lib.chol_recurrence_workspace_size(F32, 1, 1, 1, None) == INVALID


@pytest.mark.parametrize("change,expect", [
    (dict(dt=F64), INVALID), (dict(dt=9), INVALID), (dict(gate=2), INVALID),
    (dict(batch=-1), INVALID), (dict(length=-1), INVALID), (dict(dim=-1), INVALID),
    (dict(batch=0), OK), (dict(dim=0), OK),
    (dict(dim=1 << 31), NOTSUP),
    (dict(a=(None, 64, 6400)), INVALID), (dict(h=(None, 64, 6400)), INVALID), (dict(last=None), INVALID),
    (dict(a=(P[0], 63, 6400)), INVALID),                       # rows overlap
    (dict(b=(P[1], 64, 6399)), INVALID),                       # batch elements overlap
    (dict(b=(P[1], 64, 32)), INVALID),
    (dict(b=(P[1], -64, 6400)), INVALID),
    (dict(h=(P[1] + 2, 64, 6400)), INVALID),                   # partly over b
    (dict(h=(P[1], 65, 6500)), INVALID),                       # b's buffer in another layout
    (dict(h=(P[1] + 64 * 2, 128, 12800), b=(P[1], 127, 12700)), INVALID),
    (dict(last=P[2] + 4), INVALID),                            # partly over h0
    (dict(last=P[1]), INVALID),                                # over b
    (dict(h0=P[4]), INVALID),                                  # h over h0
])
def test_recurrence_refusals(change, expect):
    assert forward(**change) == expect


def test_recurrence_workspace_refusals():
    big = dict(batch=1, length=1 << 16, a=(P[0], 64, 0), b=(P[1], 64, 0), h=(P[4], 64, 0))
    n = need(BF16, 1, 1 << 16, 64)[1]
    assert forward(**big, ws=None, wbytes=0) == WS
    assert forward(**big, wbytes=n - 1) == WS
    assert forward(**big, ws=P[5] + 4) == INVALID
    assert forward(**big, ws=P[1], wbytes=n) == INVALID
    assert forward(**big, ws=P[3], wbytes=n) == INVALID


@pytest.mark.parametrize("change", [
    dict(dt=F64), dict(gate=-1), dict(h=(None, 64, 6400)), dict(adj=(None, 64, 6400)), dict(da=(None, 64, 6400)),
    dict(db=(None, 64, 6400)), dict(d0=None),
    dict(da=(P[1], 64, 6400)), dict(db=(P[1], 64, 6400)),       # over h, which is read a step ahead
    dict(da=(P[6], 64, 6400)), dict(da=(P[6] + 64, 64, 6400)),  # adjA and adjB share elements
    dict(da=(P[5], 127, 12700), db=(P[5] + 128, 127, 12700)),   # slices that wrap into each other
    dict(d0=P[3]), dict(d0=P[4] + 4), dict(d0=P[5]),
])
def test_recurrence_adjoint_refusals(change):
    assert adjoint(**change) == INVALID


def test_binding_refuses():
    a = torch.zeros(2, 3, 4)
    with pytest.raises(ValueError):
        dc.chol_recurrence(a, a)                               # not on the GPU
    with pytest.raises(ValueError):
        dc.chol_recurrence(a[0], a[0])
    with pytest.raises(TypeError):
        dc.chol_recurrence(a.double(), a.double())
    with pytest.raises(TypeError):
        dc.chol_recurrence(a, a.half())
    with pytest.raises(ValueError):
        dc.chol_recurrence(a, a[:1])
    with pytest.raises(ValueError):
        dc.chol_recurrence(a, a, gate="tanh")
    with pytest.raises(ValueError):
        dc.chol_recurrence_adjoint(a, a, a[:, :2])
