"""chol_causal_conv and chol_causal_conv_adjoint against 64 bits, on the GPU."""
import pytest

import language_util as lu
import train_util as tu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def make(batch, length, dim, width, dtype, bias=True, state=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, w, b, adj = r(batch, length, dim), r(dim, width), r(dim), r(batch, length, dim)
    s, last = r(batch, width - 1, dim), r(batch, width - 1, dim)
    return tuple(t.to(dtype).cuda() if t is not None else None for t in
                 (x, w, b if bias else None, s if state else None, adj, last if state else None))


def check(x, w, bias, state, adj, adj_last, silu, what):
    import differentiable_cholesky_amd as dc
    y, last = dc.chol_causal_conv(x, w, bias=bias, state=state, silu=silu)
    ref, kept, bound = lu.conv_forward(x, w, bias, state, silu)
    tu.near(y, ref, bound, what + " y")
    assert torch.equal(last.double(), kept)
    got = dc.chol_causal_conv_adjoint(x, w, adj, bias=bias, state=state, adjLast=adj_last, silu=silu)
    refs, bounds = lu.conv_adjoint(x, w, adj, bias, state, adj_last, silu)
    for name, a, b, c in zip(("adjX", "adjW", "adjBias", "adjState"), got, refs, bounds):
        if a is not None:
            tu.near(a, b, c, f"{what} {name}")
    assert (got[2] is None) == (bias is None) and (got[3] is None) == (state is None)


SIZES = [(1, 1, 1), (2, 1, 5), (3, 2, 64), (2, 3, 7), (1, 4, 513), (2, 7, 130), (1, 8, 8), (3, 9, 33), (1, 63, 1), (2, 64, 3),
         (2, 65, 256), (1, 300, 100), (5, 517, 17), (1, 5000, 12), (2, 1100, 1032), (70, 3, 4)]


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("batch,length,dim", SIZES)
def test_forward_and_adjoint(batch, length, dim, width, dtype, silu):
    odd = batch + length + dim + width
    check(*make(batch, length, dim, width, dtype, bias=odd % 3 > 0, state=odd % 2 > 0, seed=odd), silu, "conv")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("length", [1, 70])
def test_layouts(dtype, length):
    """Sequence-major storage and column slices of a joint buffer at odd offsets."""
    import differentiable_cholesky_amd as dc
    batch, dim, width = 3, 67, 4
    x, w, bias, state, adj, adj_last = make(batch, length, dim, width, dtype)
    y, _ = dc.chol_causal_conv(x, w, bias=bias, state=state)
    grads = dc.chol_causal_conv_adjoint(x, w, adj, bias=bias, state=state, adjLast=adj_last)
    joint = torch.full((batch, length, 3 * dim + 5), 7.0, dtype=dtype, device="cuda")
    xj, yj, dj = (joint[..., k + k * dim:k + (k + 1) * dim] for k in (1, 2, 0))
    xj.copy_(x)
    dc.chol_causal_conv(xj, w, bias=bias, state=state, y=yj)
    assert torch.equal(yj, y) and torch.equal(xj, x)
    major = adj.transpose(0, 1).contiguous().transpose(0, 1)
    got = dc.chol_causal_conv_adjoint(xj, w, major, bias=bias, state=state, adjLast=adj_last, adjX=dj)
    for p, q in zip(got, grads):
        assert torch.equal(p, q)
    for k in (dim, 2 * dim + 1, 3 * dim + 2, 3 * dim + 4):
        assert (joint[..., k] == 7).all()


@pytest.mark.parametrize("length", [1, 2, 5, 200])
def test_kept_rows_in_place_and_in_pieces(length):
    """A sequence in two pieces, or a token at a time, is the sequence."""
    import differentiable_cholesky_amd as dc
    x, w, bias, state, adj, adj_last = make(2, length + 6, 100, 4, torch.bfloat16, seed=3)
    y, last = dc.chol_causal_conv(x, w, bias=bias, state=state)
    kept = state.clone()
    parts = [dc.chol_causal_conv(x[:, :length], w, bias=bias, state=kept, last=kept)[0]]
    parts += [dc.chol_causal_conv(x[:, t:t + 1], w, bias=bias, state=kept, last=kept)[0] for t in range(length, length + 6)]
    assert torch.equal(torch.cat(parts, 1), y) and torch.equal(kept, last)


def test_empty_sequences_and_accumulated_gradients():
    import differentiable_cholesky_amd as dc
    x, w, bias, state, adj, adj_last = make(2, 40, 30, 3, torch.float32)
    e = x[:, :0]
    y, last = dc.chol_causal_conv(e, w, bias=bias, state=state)
    assert y.shape == e.shape and torch.equal(last, state)
    assert not dc.chol_causal_conv(e, w)[1].any()
    _, dw, db, ds = dc.chol_causal_conv_adjoint(e, w, e, bias=bias, state=state, adjLast=adj_last)
    assert torch.equal(ds, adj_last) and not dw.any() and not db.any()
    z = x[:0]
    assert dc.chol_causal_conv(z, w)[0].shape == z.shape
    _, dw, db, _ = dc.chol_causal_conv_adjoint(z, w, z, bias=bias)
    assert not dw.any() and not db.any()
    _, dw, db, _ = dc.chol_causal_conv_adjoint(x, w, adj, bias=bias)
    dw2, db2 = torch.full_like(dw, 2.0), torch.full_like(db, 3.0)
    dc.chol_causal_conv_adjoint(x, w, adj, bias=bias, adjW=dw2, adjBias=db2, accumulate=True)
    assert torch.equal(dw2, 2.0 + dw) and torch.equal(db2, 3.0 + db)


@pytest.mark.parametrize("width", [2, 3, 4])
def test_non_finite_inputs_reach_their_window_only(width):
    import differentiable_cholesky_amd as dc
    x, w, bias, _, adj, _ = make(1, 200, 20, width, torch.float32, state=False)
    clean, _ = dc.chol_causal_conv(x, w, bias=bias)
    x[0, 70, 3], x[0, 71, 11] = float("nan"), float("inf")
    y, _ = dc.chol_causal_conv(x, w, bias=bias)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[0, 70:70 + width, 3] = bad[0, 71:71 + width, 11] = True
    assert torch.equal(y[~bad], clean[~bad]) and torch.isnan(y[0, 70:70 + width, 3]).all()
    dx = dc.chol_causal_conv_adjoint(x, w, adj, bias=bias)[0]
    reach = torch.zeros_like(bad)
    reach[0, 71 - width:70 + width, 3] = reach[0, 72 - width:71 + width, 11] = True
    assert torch.isfinite(dx[~reach]).all()


@pytest.mark.parametrize("length", [1, 130])
def test_captured_and_replayed(length):
    """Kept rows carried on by a graph as by eager calls, and gradients of changed inputs."""
    import differentiable_cholesky_amd as dc
    x, w, bias, state, adj, _ = make(2, length, 70, 4, torch.bfloat16, seed=9)
    a, b = state.clone(), state.clone()
    dc.chol_causal_conv(x, w, bias=bias, state=state)
    dc.chol_causal_conv_adjoint(x, w, adj, bias=bias, state=state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = dc.chol_causal_conv_adjoint(x, w, adj, bias=bias, state=a)
        y, _ = dc.chol_causal_conv(x, w, bias=bias, state=a, last=a)
    for _ in range(4):
        graph.replay()
        want = dc.chol_causal_conv_adjoint(x, w, adj, bias=bias, state=b)
        z, _ = dc.chol_causal_conv(x, w, bias=bias, state=b, last=b)
        torch.cuda.synchronize()
        assert torch.equal(y, z) and torch.equal(a, b)
        for p, q in zip(grads, want):
            assert torch.equal(p, q)
        x.mul_(-0.5)


def test_other_streams_and_workspaces():
    import differentiable_cholesky_amd as dc
    x, w, bias, state, adj, _ = make(2, 300, 70, 4, torch.bfloat16)
    want = dc.chol_causal_conv_adjoint(x, w, adj, bias=bias, state=state)
    need = dc.chol_causal_conv_adjoint_workspace_size(dc.CHOL_BF16, 2, 300, 70, 4)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = dc.chol_causal_conv_adjoint(x, w, adj, bias=bias, state=state, workspace=ws, stream=side)
    y, _ = dc.chol_causal_conv(x, w, bias=bias, state=state, stream=side)
    side.synchronize()
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    assert torch.equal(y, dc.chol_causal_conv(x, w, bias=bias, state=state)[0])


def test_gradients_against_differences():
    import differentiable_cholesky_amd as dc
    x, w, bias, state, adj, _ = make(1, 20, 6, 3, torch.float32)
    f = lambda x, w, bias, state: (lu.conv_forward(x, w, bias, state, True)[0] * adj.double()).sum()  # noqa: E731
    got = dc.chol_causal_conv_adjoint(x, w, adj, bias=bias, state=state)
    args = [t.double() for t in (x, w, bias, state)]
    g = torch.Generator().manual_seed(1)
    for k in range(4):
        way = torch.randn(args[k].shape, generator=g).double().cuda()
        step = 1e-5
        ends = [f(*(a + s * step * way if i == k else a for i, a in enumerate(args))) for s in (1, -1)]
        slope = (ends[0] - ends[1]) / (2 * step)
        size = (got[k].double() * way).abs().sum()
        # fp32 gradients of sums of at most 20 terms, and a difference of order step^2
        assert abs((got[k].double() * way).sum() - slope) <= 200 * tu.U * size + 1e-8 * size
