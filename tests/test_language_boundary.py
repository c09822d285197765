"""Argument checks of the convolution, the scan and the token log probabilities, on the CPU:
the C-ABI refuses on the host before anything is launched, and the binding refuses what it
cannot pass on."""
import ctypes
import random

import pytest

dc = pytest.importorskip("differentiable_cholesky_amd")
torch = pytest.importorskip("torch")
from differentiable_cholesky_amd import _language, _lib  # noqa: E402

lib = _lib.lib
F32, F64, BF16, F16 = _lib.CHOL_F32, _lib.CHOL_F64, dc.CHOL_BF16, dc.CHOL_F16
OK, INVALID, NOTSUP, WS = (_lib.CHOL_OK, _lib.CHOL_ERR_INVALID_VALUE, _lib.CHOL_ERR_NOT_SUPPORTED,
                           _lib.CHOL_ERR_WORKSPACE)
P = [k << 32 for k in range(1, 40)]   # addresses that are never read: every call below fails a check first


# ------------------------------------------------------------- convolution ----

def conv(dt=BF16, batch=2, length=100, dim=64, width=4, x=(P[0], 64, 6400), w=P[1], bias=P[2], state=P[3], last=P[4],
         y=(P[5], 64, 6400)):
    return lib.chol_causal_conv(dt, 1, batch, length, dim, width, *x, w, bias, state, last, *y, None)


def conv_adjoint(dt=BF16, batch=2, length=100, dim=64, width=4, x=(P[0], 64, 6400), w=P[1], bias=P[2], state=P[3],
                 adj=(P[5], 64, 6400), adj_last=P[6], dx=(P[7], 64, 6400), dw=P[8], db=P[9], ds=P[10], ws=P[11],
                 wbytes=1 << 40):
    return lib.chol_causal_conv_adjoint(dt, 1, batch, length, dim, width, *x, w, bias, state, *adj, adj_last, *dx, dw, db, 0,
                                        ds, ws, wbytes, None)


@pytest.mark.parametrize("change,expect", [
    (dict(dt=F64), INVALID), (dict(dt=9), INVALID), (dict(batch=-1), INVALID), (dict(length=-1), INVALID), (dict(dim=-1), INVALID),
    (dict(width=0), INVALID), (dict(width=1), NOTSUP), (dict(width=5), NOTSUP), (dict(batch=0), OK), (dict(dim=0), OK),
    (dict(batch=1 << 20, dim=1 << 20), NOTSUP), (dict(length=1 << 31), NOTSUP), (dict(batch=1 << 25, dim=1), NOTSUP),
    (dict(x=(None, 64, 6400)), INVALID), (dict(w=None), INVALID), (dict(y=(None, 64, 6400)), INVALID),
    (dict(x=(P[0], 63, 6400)), INVALID), (dict(x=(P[0], 64, 6399)), INVALID), (dict(y=(P[5], 64, 32)), INVALID),
    (dict(x=(P[0] + 1, 64, 6400)), INVALID), (dict(w=P[1] + 1), INVALID),
    (dict(y=(P[0], 64, 6400)), INVALID), (dict(y=(P[0] + 2, 64, 6400)), INVALID), (dict(y=(P[1], 64, 6400)), INVALID),
    (dict(y=(P[3], 64, 6400)), INVALID), (dict(last=P[3] + 2), INVALID), (dict(last=P[5]), INVALID), (dict(last=P[0]), INVALID),
    (dict(last=P[2]), INVALID), (dict(length=0, x=(None, 0, 0), y=(None, 0, 0), last=None), OK),
])
def test_conv_refusals(change, expect):
    assert conv(**change) == expect


@pytest.mark.parametrize("change,expect", [
    (dict(dt=F64), INVALID), (dict(width=5), NOTSUP), (dict(dim=0), OK), (dict(adj=(None, 64, 6400)), INVALID),
    (dict(dx=(None, 64, 6400)), INVALID), (dict(dw=None), INVALID), (dict(dw=P[8] + 2), INVALID),
    (dict(dx=(P[5], 64, 6400)), INVALID), (dict(dx=(P[0], 64, 6400)), INVALID), (dict(ds=P[6]), INVALID), (dict(ds=P[7]), INVALID),
    (dict(db=P[8] + 4), INVALID), (dict(dw=P[3]), INVALID), (dict(ws=None), WS), (dict(wbytes=16), WS),
    (dict(ws=P[11] + 2), INVALID), (dict(ws=P[0]), INVALID), (dict(ws=P[8]), INVALID),
])
def test_conv_adjoint_refusals(change, expect):
    assert conv_adjoint(**change) == expect


def test_conv_workspace_size():
    out = ctypes.c_size_t(1)
    size = lib.chol_causal_conv_adjoint_workspace_size
    assert size(BF16, 0, 10, 10, 4, ctypes.byref(out)) == OK and out.value == 0
    assert size(BF16, 1, 10, 10, 4, ctypes.byref(out)) == OK and out.value == 10 * 5 * 4
    assert size(BF16, 1, 10, 10, 7, ctypes.byref(out)) == NOTSUP
    assert size(F64, 1, 10, 10, 4, ctypes.byref(out)) == INVALID
    assert size(F32, 1, 10, 10, 4, None) == INVALID


# -------------------------------------------------------------------- scan ----

ROWS, MIXED = (64, 6400), (32, 3200)


def scan_args(batch=2, length=100, dim=64, groups=2, states=16, **change):
    rows = {"u": (P[0], *ROWS), "delta": (P[1], *ROWS), "B": (P[2], *MIXED), "C": (P[3], *MIXED), "z": (P[4], *ROWS),
            "y": (P[5], *ROWS), "adj": (P[12], *ROWS), "adj_u": (P[13], *ROWS), "adj_delta": (P[14], *ROWS),
            "adj_B": (P[15], *MIXED), "adj_C": (P[16], *MIXED), "adj_z": (P[17], *ROWS)}
    one = {"A": P[6], "D": P[7], "bias": P[8], "h0": P[9], "hlast": P[10], "starts": P[11], "adj_hlast": P[18], "adj_A": P[19],
           "adj_D": P[20], "adj_bias": P[21], "adj_h0": P[22]}
    for k, x in change.items():
        (rows if k in rows else one)[k] = x
    get = lambda *names: [v or 0 for n in names for v in (rows[n] if n in rows else (one[n],))]  # noqa: E731
    return _language._ARGS.pack(
        batch, length, dim, groups, states, 1, 0, *get("u", "delta", "B", "C", "z", "y", "A", "D", "bias", "h0", "hlast", "starts",
                                                       "adj", "adj_u", "adj_delta", "adj_B", "adj_C", "adj_z", "adj_hlast",
                                                       "adj_A", "adj_D", "adj_bias", "adj_h0"))


def scan(dt=BF16, ws=P[25], wbytes=1 << 40, **change):
    return lib.chol_selective_scan(dt, scan_args(**change), ws, wbytes, None)


def scan_adjoint(dt=BF16, ws=P[25], wbytes=1 << 40, **change):
    return lib.chol_selective_scan_adjoint(dt, scan_args(**change), ws, wbytes, None)


@pytest.mark.parametrize("change,expect", [
    (dict(dt=F64), INVALID), (dict(batch=-1), INVALID), (dict(length=-1), INVALID), (dict(dim=-2), INVALID), (dict(groups=0), INVALID),
    (dict(groups=3), INVALID), (dict(states=0), INVALID), (dict(states=65), NOTSUP), (dict(batch=0), OK), (dict(dim=0), OK),
    (dict(batch=1 << 20, dim=1 << 10), NOTSUP), (dict(length=(1 << 30) + 1), NOTSUP),
    (dict(batch=1, length=2, u=(P[0], (1 << 25) + 1, 0)), NOTSUP), (dict(batch=1, length=2, y=(P[5], 1 << 26, 0)), NOTSUP),
    (dict(batch=1, length=2, C=(P[3], 1 << 30, 0)), NOTSUP), (dict(batch=1, B=(P[2], 1 << 41, 0)), INVALID),
    (dict(u=(0, *ROWS)), INVALID), (dict(delta=(0, *ROWS)), INVALID), (dict(B=(0, *MIXED)), INVALID), (dict(C=(0, *MIXED)), INVALID),
    (dict(y=(0, *ROWS)), INVALID), (dict(A=0), INVALID), (dict(hlast=0), INVALID),
    (dict(u=(P[0], 63, 6400)), INVALID), (dict(B=(P[2], 31, 3200)), INVALID), (dict(C=(P[3], 32, 3199)), INVALID),
    (dict(A=P[6] + 2), INVALID), (dict(u=(P[0] + 1, *ROWS)), INVALID), (dict(h0=P[9] + 2), INVALID),
    (dict(y=(P[0] + 2, *ROWS)), INVALID), (dict(y=(P[2], *ROWS)), INVALID), (dict(y=(P[0], 65, 6500)), INVALID),
    (dict(y=(P[6], *ROWS)), INVALID), (dict(hlast=P[9] + 4), INVALID), (dict(hlast=P[6]), INVALID), (dict(starts=P[9]), INVALID),
    (dict(starts=P[10]), INVALID), (dict(starts=P[5]), INVALID),
    (dict(ws=0), WS), (dict(wbytes=64), WS), (dict(ws=P[25] + 2), INVALID), (dict(ws=P[3]), INVALID), (dict(ws=P[10]), INVALID),
])
def test_scan_refusals(change, expect):
    assert scan(**change) == expect


@pytest.mark.parametrize("change,expect", [
    (dict(batch=1, length=2, adj_z=(P[17], 1 << 26, 0)), NOTSUP), (dict(batch=1, length=2, adj=(P[12], 1 << 26, 0)), NOTSUP),
    (dict(dt=F64), INVALID), (dict(states=65), NOTSUP), (dict(dim=0), OK), (dict(starts=0), INVALID), (dict(adj=(0, *ROWS)), INVALID),
    (dict(adj_u=(0, *ROWS)), INVALID), (dict(adj_z=(0, *ROWS)), INVALID), (dict(adj_B=(0, *MIXED)), INVALID), (dict(adj_A=0), INVALID),
    (dict(adj_A=P[19] + 1), INVALID), (dict(adj_delta=(P[0], *ROWS)), INVALID), (dict(adj_u=(P[4], *ROWS)), INVALID),
    (dict(adj_u=(P[12], *ROWS), adj_z=(P[12], *ROWS)), INVALID), (dict(adj_B=(P[3], *MIXED)), INVALID),
    (dict(adj_B=(P[16], *MIXED)), INVALID), (dict(adj_h0=P[11]), INVALID), (dict(adj_h0=P[18] + 4), INVALID),
    (dict(adj_D=P[19]), INVALID), (dict(adj_bias=P[6]), INVALID),
    (dict(ws=0), WS), (dict(wbytes=1024), WS), (dict(ws=P[25] + 2), INVALID), (dict(ws=P[12]), INVALID), (dict(ws=P[22]), INVALID),
])
def test_scan_adjoint_refusals(change, expect):
    assert scan_adjoint(**change) == expect


def test_scan_no_arguments():
    assert lib.chol_selective_scan(BF16, None, None, 0, None) == INVALID
    assert lib.chol_selective_scan_adjoint(BF16, None, None, 0, None) == INVALID


def test_launches_that_a_call_of_no_elements_makes_still_fit():
    """Without a batch the gradients of the weights are written all the same, a thread or more each."""
    out = ctypes.c_size_t(1)
    conv, scan_ = lib.chol_causal_conv_adjoint_workspace_size, lib.chol_selective_scan_workspace_size
    for batch in (0, 1):
        assert conv(BF16, batch, 1, 1 << 25, 4, ctypes.byref(out)) == OK
        assert conv(BF16, batch, 1, 1 << 28, 4, ctypes.byref(out)) == NOTSUP
        assert scan_(1, batch, 0, 1 << 20, 1, 16, ctypes.byref(out)) == OK
        assert scan_(1, batch, 0, 1 << 28, 1, 16, ctypes.byref(out)) == NOTSUP


def test_scan_sizes():
    block = lib.chol_selective_scan_block
    assert [block(n) for n in (-1, 0, 1, 16, 17, 32, 33, 64, 65)] == [-1, -1, 64, 64, 32, 32, 16, 16, -1]
    out = ctypes.c_size_t(1)
    size = lib.chol_selective_scan_workspace_size
    assert size(0, 4, 1, 100, 1, 16, ctypes.byref(out)) == OK and out.value == 0
    assert size(0, 64, 1000, 4096, 1, 16, ctypes.byref(out)) == OK and out.value == 0     # waves enough without segments
    assert size(0, 1, 10000, 64, 1, 16, ctypes.byref(out)) == OK and out.value > 0
    assert size(1, 1, 0, 64, 1, 16, ctypes.byref(out)) == OK and out.value == 0
    assert size(0, 1, 10, 64, 3, 16, ctypes.byref(out)) == INVALID
    assert size(0, 1, 10, 64, 1, 16, None) == INVALID


def shared(one, other, batch, length):
    import numpy as np
    at = lambda a: (a[0] + np.arange(batch)[:, None, None] * a[3] + np.arange(length)[:, None] * a[2] + np.arange(a[1])).ravel()  # noqa: E731
    return bool(np.isin(at(one), at(other)).any())


def test_slices_of_different_widths_are_apart_where_no_element_is_shared():
    """y and B in one buffer with the same distances, at every kind of offset, against the sets of their elements.
    The missing workspace is found after the arrays have been compared."""
    rng, seen = random.Random(0), {False: 0, True: 0}
    length = 70                                                 # (more than a segment, so that there is a workspace)
    for k in range(400):
        batch, dim, states = rng.choice([1, 2, 3]), rng.choice([1, 2, 5]), rng.choice([1, 3, 8])
        most = max(dim, states)
        ld = most + rng.choice([0, 1, dim, dim + states])
        stride = ld * (length - 1) + most + rng.choice([0, 3, 2 * ld])
        if k % 2:                                               # sequence-major
            stride = most + rng.choice([0, 1, dim, dim + states])
            ld = stride * (batch - 1) + most + rng.choice([0, 3, 2 * stride])
        d = rng.choice([0, 1, 2]) * stride + rng.choice([0, 1, 2, length]) * ld + rng.randint(-most - 2, most + 3)
        d *= rng.choice([-1, 1])
        same = shared((0, dim, ld, stride), (d, states, ld, stride), batch, length)
        seen[same] += 1
        at = 1 << 38
        got = scan(batch=batch, length=length, dim=dim, groups=1, states=states, u=(P[0], 64, 6400), delta=(P[1], 64, 6400),
                   z=(P[4], 64, 6400), C=(P[3], 64, 6400), y=(at, ld, stride), B=(at + 2 * d, ld, stride), ws=None, wbytes=0)
        assert got == (INVALID if same else WS), (batch, dim, states, ld, stride, d)
    assert min(seen.values()) > 50


# ------------------------------------------------------- log probabilities ----

def logprob(dt=BF16, rows=10, vocab=100000, x=(P[0], 100000), tokens=P[1], scale=1.0, logp=P[2], lse=P[3], entropy=P[4], top=4,
            top_logp=P[5], ids=P[6], ws=P[7], wbytes=1 << 40):
    return lib.chol_token_logprob(dt, rows, vocab, *x, tokens, scale, logp, lse, entropy, top, top_logp, ids, ws, wbytes, None)


def logprob_adjoint(dt=BF16, rows=10, vocab=100000, x=(P[0], 100000), tokens=P[1], scale=1.0, lse=P[2], entropy=P[3], gl=P[4],
                    ge=P[5], dx=(P[6], 100000)):
    return lib.chol_token_logprob_adjoint(dt, rows, vocab, *x, tokens, scale, lse, entropy, gl, ge, *dx, None)


@pytest.mark.parametrize("change,expect", [
    (dict(dt=F64), INVALID), (dict(rows=-1), INVALID), (dict(vocab=-1), INVALID), (dict(vocab=0), INVALID), (dict(rows=0), OK),
    (dict(rows=0, vocab=0, top=0), OK), (dict(vocab=524289, x=(P[0], 524289)), NOTSUP), (dict(rows=1 << 31), NOTSUP),
    (dict(rows=1 << 29), NOTSUP), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(top=-1), INVALID), (dict(top=33), INVALID), (dict(vocab=3, top=4), INVALID),
    (dict(x=(None, 100000)), INVALID), (dict(x=(P[0], 99999)), INVALID), (dict(x=(P[0] + 1, 100000)), INVALID),
    (dict(tokens=None), INVALID), (dict(tokens=P[1] + 4), INVALID), (dict(logp=None), INVALID), (dict(lse=None), INVALID),
    (dict(top_logp=None), INVALID), (dict(ids=None), INVALID), (dict(ids=P[6] + 4), INVALID), (dict(logp=P[3]), INVALID),
    (dict(entropy=P[2] + 4), INVALID), (dict(ids=P[1]), INVALID), (dict(lse=P[0]), INVALID), (dict(top_logp=P[6]), INVALID),
    (dict(ws=None), WS), (dict(wbytes=100), WS), (dict(ws=P[7] + 4), INVALID), (dict(ws=P[0]), INVALID), (dict(ws=P[6]), INVALID),
])
def test_logprob_refusals(change, expect):
    assert logprob(**change) == expect


@pytest.mark.parametrize("change,expect", [
    (dict(dt=F64), INVALID), (dict(vocab=0), INVALID), (dict(rows=0), OK), (dict(scale=0.0), INVALID), (dict(x=(None, 100000)), INVALID),
    (dict(tokens=None), INVALID), (dict(lse=None), INVALID), (dict(entropy=None), INVALID), (dict(dx=(None, 100000)), INVALID),
    (dict(dx=(P[6], 99999)), INVALID), (dict(dx=(P[0] + 2, 100000)), INVALID), (dict(dx=(P[0], 100001)), INVALID),
    (dict(dx=(P[2], 100000)), INVALID), (dict(dx=(P[1], 100000)), INVALID), (dict(vocab=1 << 20), NOTSUP),
])
def test_logprob_adjoint_refusals(change, expect):
    assert logprob_adjoint(**change) == expect


# ----------------------------------------------------------------- binding ----

def test_binding_refuses():
    x, w = torch.zeros(2, 3, 4), torch.zeros(4, 4)
    for call in (lambda: dc.chol_causal_conv(x, w),                                  # not on the GPU
                 lambda: dc.chol_causal_conv(x[0], w),
                 lambda: dc.chol_causal_conv(x, w[:, :1]),
                 lambda: dc.chol_causal_conv(x, w[:3]),
                 lambda: dc.chol_causal_conv(x, w.t()[:, :3]),
                 lambda: dc.chol_causal_conv(x, w, bias=w[0, :3]),
                 lambda: dc.chol_causal_conv_adjoint(x, w, x[:1])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        dc.chol_causal_conv(x, w.half())
    with pytest.raises(TypeError):
        dc.chol_causal_conv(x.double(), w.double())
    A, B = torch.zeros(4, 16), torch.zeros(2, 3, 16)
    for call in (lambda: dc.chol_selective_scan(x, x, A, B, B),
                 lambda: dc.chol_selective_scan(x[0], x[0], A, B, B),
                 lambda: dc.chol_selective_scan(x, x[:1], A, B, B),
                 lambda: dc.chol_selective_scan(x, x, A[:3], B, B),
                 lambda: dc.chol_selective_scan(x, x, A, B[..., :8], B),
                 lambda: dc.chol_selective_scan(x, x, A, B.view(2, 3, 1, 16), B),
                 lambda: dc.chol_selective_scan(x, x, A, *[torch.zeros(2, 3, 3, 16)] * 2),
                 lambda: dc.chol_selective_scan(x, x, *[torch.zeros(4, 65)], *[torch.zeros(2, 3, 65)] * 2),
                 lambda: dc.chol_selective_scan_block(65)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        dc.chol_selective_scan(x, x, A, B.half(), B.half())
    y, t = torch.zeros(3, 8), torch.zeros(3, dtype=torch.int64)
    for call in (lambda: dc.chol_token_logprob(y, t),
                 lambda: dc.chol_token_logprob(y[0], t),
                 lambda: dc.chol_token_logprob(y, t[:2]),
                 lambda: dc.chol_token_logprob(y, t, top=9),
                 lambda: dc.chol_token_logprob(y, t, top=-1),
                 lambda: dc.chol_token_logprob_adjoint(y, t, y[:, 0], adjEntropy=y[:, 0])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        dc.chol_token_logprob(y, t.int())
