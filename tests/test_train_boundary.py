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
    assert need(F32, 1 << 24, 1, 1)[0] == NOTSUP              # more threads than a grid holds
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


def shared(length, dim, batch, ld, stride, d):
    """Whether two such arrays, d elements apart, have an element in common."""
    import numpy as np
    one = (np.arange(batch)[:, None, None] * stride + np.arange(length)[:, None] * ld + np.arange(dim)).ravel()
    return bool(np.isin(one, one + d).any())


def test_slices_of_one_buffer_are_apart_where_no_element_is_shared():
    """Two arrays with the same distances, at every kind of offset, against the sets of their elements.  The missing
    workspace is found after the arrays have been compared."""
    import random
    rng = random.Random(0)
    seen = {False: 0, True: 0}
    length, at = 1100, 1 << 36                                 # more than one workgroup along the sequence
    for k in range(300):
        batch, dim = rng.choice([1, 2, 3]), rng.choice([1, 2, 5])
        ld = dim + rng.choice([0, 1, dim, dim + 3])
        stride = ld * (length - 1) + dim + rng.choice([0, ld - dim, 3, 2 * ld])
        if k % 2:                                              # sequence-major
            stride = dim + rng.choice([0, 1, dim, dim + 3])
            ld = stride * (batch - 1) + dim + rng.choice([0, stride - dim, 3, 2 * stride])
        d = abs(rng.choice([0, 1, 2]) * stride + rng.choice([0, 1, 2, length]) * ld + rng.randint(-dim - 2, 2 * dim + 3))
        if d == 0:
            continue
        same = shared(length, dim, batch, ld, stride, d)
        seen[same] += 1
        got = forward(batch=batch, length=length, dim=dim, a=(1 << 40, ld, stride), b=(at, ld, stride),
                      h=(at + 2 * d, ld, stride), ws=None, wbytes=0)
        assert got == (INVALID if same else WS), (batch, dim, ld, stride, d)
    assert min(seen.values()) > 50
    # halves of a joint buffer, sequence-major, and batch-major with padding that is no multiple of a row
    for ld, stride in ((4 * 128, 128), (128, 128 * 1100 + 5)):
        rows = dict(batch=4, length=1100, dim=64, ws=None, wbytes=0)
        one, other = (P[0], ld, stride), (P[0] + 64 * 2, ld, stride)
        assert forward(**rows, a=one, b=(P[1], ld, stride), h=other) == WS
        assert forward(**rows, a=one, b=(P[1], ld, stride), h=(P[0] + 63 * 2, ld, stride)) == INVALID
        far = {k: (P[i], ld, stride) for i, k in enumerate(("a", "h", "adj"), 8)}
        assert adjoint(**rows, **far, da=one, db=other) == WS
        assert adjoint(**rows, **far, da=one, db=(P[0] + 65 * 2 - 4, ld, stride)) == INVALID
        assert adjoint(**rows, **dict(far, h=one), da=(P[1], ld, stride), db=other) == WS


def test_an_empty_sequence_has_the_limits_of_one_step():
    """It copies the states, with as many threads."""
    none = (None, 0, 0)
    for batch, dim in ((1 << 24, 1), (1 << 20, 1 << 20), (1 << 31, 1)):
        assert need(BF16, batch, 0, dim)[0] == need(BF16, batch, 1, dim)[0] == NOTSUP
        assert forward(batch=batch, length=0, dim=dim, a=none, b=none, h=none) == NOTSUP
        assert adjoint(batch=batch, length=0, dim=dim, a=none, h=none, adj=none, da=none, db=none) == NOTSUP
    assert need(BF16, 1 << 22, 0, 16) == (OK, 0)
    assert forward(length=0, a=none, b=none, h=none, last=None) == INVALID


@pytest.mark.parametrize("length,ld", [((1 << 24) + 1, 1 << 40), ((1 << 31) - 1, 1 << 40), ((1 << 22) + 1, 1 << 40)])
def test_spans_beyond_64_bits_are_refused(length, ld):
    """Rows of ld elements whose byte offsets pass 64 bits; 2^24 of 2^40 come out as no offset at all."""
    rows = dict(batch=1, length=length, dim=1, a=(P[0], 1, 0), b=(P[1], 1, 0), h=(P[4], 1, 0))
    assert forward(**dict(rows, h=(P[1], ld, 0))) == INVALID
    assert forward(**dict(rows, a=(P[0], ld, 0), b=(P[1], ld, 0), h=(P[0] + (1 << 20), ld, 0))) == INVALID
    assert forward(**dict(rows, batch=2, length=3, a=(P[0], 1, ld), b=(P[1], 1, ld), h=(P[0] + 64, 1, ld * 2))) == INVALID
    assert norm(rows=length, x=(P[0], ld), r=(None, 0), y=(P[0] + (1 << 20), ld)) == INVALID
    assert norm_adjoint(rows=length, h=(P[0], ld), dx=(P[0] + (1 << 20), ld)) == INVALID


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


# ------------------------------------------------------------------- norm ----

def norm(dt=BF16, rows=10, cols=64, x=(P[0], 64), r=(P[1], 64), w=P[2], eps=1e-6, y=(P[3], 64), h=(P[4], 64)):
    return lib.chol_rmsnorm(dt, rows, cols, *x, *r, w, eps, *y, *h, None)


def quant(dt=BF16, rows=10, cols=64, group=32, x=(P[0], 64), r=(P[1], 64), w=P[2], eps=1e-6, q=(P[3], 64),
          scale=(P[4], 2), h=(P[5], 64)):
    return lib.chol_rmsnorm_quant(dt, rows, cols, group, *x, *r, w, eps, *q, *scale, *h, None)


def norm_adjoint(dt=BF16, rows=2000, cols=64, h=(P[0], 64), w=P[1], adj=(P[2], 64), past=(P[3], 64), eps=1e-6,
                 dx=(P[4], 64), dw=P[5], acc=0, ws=P[6], wbytes=1 << 40):
    return lib.chol_rmsnorm_adjoint(dt, rows, cols, *h, w, *adj, *past, eps, *dx, dw, acc, ws, wbytes, None)


@pytest.mark.parametrize("change,expect", [
    (dict(dt=F64), INVALID), (dict(rows=-1), INVALID), (dict(cols=-1), INVALID), (dict(rows=0), OK), (dict(cols=0), OK),
    (dict(cols=16385), NOTSUP), (dict(rows=1 << 31), NOTSUP), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(x=(None, 64)), INVALID), (dict(w=None), INVALID), (dict(y=(None, 64)), INVALID), (dict(h=(None, 64)), INVALID),
    (dict(x=(P[0], 63)), INVALID), (dict(y=(P[3], 63)), INVALID), (dict(r=(P[1], -64)), INVALID),
    (dict(y=(P[0] + 2, 64)), INVALID), (dict(y=(P[0], 65)), INVALID), (dict(y=(P[4], 64)), INVALID),
    (dict(h=(P[2], 64)), INVALID), (dict(y=(P[2] - 64, 64)), INVALID), (dict(h=(P[1] + 2, 64)), INVALID),
])
def test_norm_refusals(change, expect):
    assert norm(**change) == expect


@pytest.mark.parametrize("change,expect", [
    (dict(group=16), INVALID), (dict(group=96), INVALID), (dict(group=512), INVALID), (dict(group=-32), INVALID),
    (dict(rows=0), OK), (dict(q=(P[0], 64)), INVALID), (dict(scale=(P[4], 1)), INVALID), (dict(scale=(None, 2)), INVALID),
    (dict(scale=(P[3], 2)), INVALID), (dict(q=(P[5], 64)), INVALID), (dict(scale=(P[1], 2)), INVALID),
])
def test_quant_refusals(change, expect):
    assert quant(**change) == expect


@pytest.mark.parametrize("change,expect", [
    (dict(dt=F64), INVALID), (dict(cols=16385), NOTSUP), (dict(cols=0), OK), (dict(eps=-1e-9), INVALID),
    (dict(dw=None), INVALID), (dict(w=None), INVALID), (dict(h=(None, 64)), INVALID), (dict(adj=(None, 64)), INVALID),
    (dict(dx=(None, 64)), INVALID), (dict(dx=(P[2] + 2, 64)), INVALID), (dict(dw=P[4]), INVALID), (dict(dw=P[0]), INVALID),
    (dict(dw=P[1]), INVALID), (dict(dx=(P[1], 64)), INVALID),
    (dict(ws=None, wbytes=0), WS), (dict(wbytes=100), WS), (dict(ws=P[6] + 2), INVALID), (dict(ws=P[4]), INVALID),
    (dict(ws=P[2]), INVALID), (dict(ws=P[5]), INVALID), (dict(past=(P[3], 3)), INVALID),
])
def test_norm_adjoint_refusals(change, expect):
    assert norm_adjoint(**change) == expect


def test_norm_adjoint_workspace_size():
    """A row of partial sums for every workgroup but a single one; a workgroup takes the rows that its threads hold."""
    def size(dt, rows, cols):
        out = ctypes.c_size_t(0)
        assert lib.chol_rmsnorm_adjoint_workspace_size(dt, rows, cols, ctypes.byref(out)) == OK
        return out.value

    for dt, width in ((BF16, 8), (F16, 8), (F32, 4)):
        for cols in (1, 64, 100, 128, 250, 300, 511, 512, 1000, 1024, 1025, 2000, 2047, 2048, 3000, 4096, 5000, 8192, 16384):
            vectors = -(-cols // width)
            together = 1 if vectors > 256 else 256 // min(t for t in (8, 16, 32, 64) if t >= min(vectors, 64))
            assert size(dt, 1, cols) == size(dt, together, cols) == 0
            assert size(dt, together + 1, cols) == 2 * cols * 4
            assert size(dt, 1 << 20, cols) in (256 * cols * 4, 512 * cols * 4)


def test_norm_binding_refuses():
    x, w = torch.zeros(3, 8), torch.ones(8)
    with pytest.raises(ValueError):
        dc.chol_rmsnorm(x, w)
    with pytest.raises(ValueError):
        dc.chol_rmsnorm(x, w[:7])
    with pytest.raises(TypeError):
        dc.chol_rmsnorm(x, w.half())
    with pytest.raises(ValueError):
        dc.chol_rmsnorm_quant(x, w, group=48)
    with pytest.raises(ValueError):
        dc.chol_rmsnorm_adjoint(x, w, x[:2])


# ------------------------------------------------------------------ AdamW ----

def adamw_list(dt=BF16, bits=8, table=None, room=0, **change):
    items = (dc._train.AdamwTensor * 2)()
    for i in range(2):
        fields = dict(p=P[0], g=P[1], m=P[2], v=P[3], master=P[4], m_scale=P[5], v_scale=P[6], n=5000, first=0)
        for k in fields:
            if k not in ("n", "first"):
                fields[k] += i << 20
        if i == 1:
            fields.update(change)
        for k, x in fields.items():
            setattr(items[i], k, x)
    chunks, size = ctypes.c_int64(-1), ctypes.c_size_t(0)
    s = lib.chol_adamw_list(dt, bits, 2, items, table, room, ctypes.byref(chunks), ctypes.byref(size))
    return s, chunks.value, size.value


def test_adamw_list():
    s, chunks, size = adamw_list()
    assert s == OK and chunks == 4 and size == 4 * 64
    buf = ctypes.create_string_buffer(size)
    at = ctypes.addressof(buf)
    assert adamw_list(table=at, room=size - 1)[0] == WS
    assert adamw_list(table=at, room=size)[0] == OK
    words = (ctypes.c_uint64 * 32).from_buffer(buf)
    assert words[0] == P[0] and words[8] == P[0] + 2 * 4096 and words[10] == P[2] + 4096 and words[13] == P[5] + 4 * 16
    assert words[7] == 4096 and words[15] == 904 + (4096 << 32)
    assert adamw_list(n=0)[:2] == (OK, 2)
    assert adamw_list(g=P[1])[0] == OK             # a gradient that two tensors share is only read


@pytest.mark.parametrize("change", [
    dict(dt=F64), dict(bits=16), dict(n=-1), dict(p=None), dict(g=None), dict(m=None), dict(v=None), dict(m_scale=None),
    dict(master=None), dict(p=P[0] + 1 + (1 << 20)), dict(master=P[4] + 2 + (1 << 20)), dict(p=P[0]), dict(p=P[0] + 9998),
    dict(g=P[0] + 100), dict(m=P[2] + 4999), dict(v=P[2]), dict(m_scale=P[6]), dict(master=P[1] + 4),
])
def test_adamw_list_refusals(change):
    assert adamw_list(**change)[0] == INVALID


@pytest.mark.parametrize("change,expect", [
    (dict(dt=F64), INVALID), (dict(bits=4), INVALID), (dict(chunks=-1), INVALID), (dict(chunks=0), OK),
    (dict(table=None), INVALID), (dict(table=P[0] + 4), INVALID), (dict(clip=P[1] + 2), INVALID),
    (dict(beta1=1.0), INVALID), (dict(beta2=-0.1), INVALID), (dict(beta1=float("nan")), INVALID), (dict(eps=-1.0), INVALID),
    (dict(lr=float("inf")), INVALID), (dict(wd=float("nan")), INVALID), (dict(step=0), INVALID),
])
def test_adamw_refusals(change, expect):
    a = dict(dt=BF16, bits=8, master=1, chunks=4, table=P[0], clip=P[1], lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, wd=0.1,
             step=1, seed=0, stream=None)
    a.update(change)
    assert lib.chol_adamw(*a.values()) == expect


def test_adamw_binding_refuses():
    t = [torch.zeros(8)]
    with pytest.raises(ValueError):
        dc.chol_adamw_list([], [], [], [])
    with pytest.raises(ValueError):
        dc.chol_adamw_list(t, t, t, t)                 # not on the GPU
    with pytest.raises(TypeError):
        dc.chol_adamw_list(t, t, [x.half() for x in t], t)
    with pytest.raises(ValueError):
        dc.chol_adamw_list(t, t, t, t, m_scale=t)
    with pytest.raises(ValueError):
        dc.chol_adamw_list(t, t, [], t)
    e = [torch.zeros(8, dtype=torch.uint8).view(torch.float8_e4m3fn)]
    with pytest.raises(ValueError):
        dc.chol_adamw_list(t, t, e, e)
