"""chol_rmsnorm, chol_rmsnorm_quant and chol_rmsnorm_adjoint against 64 bits, on the GPU."""
import pytest

import train_util as tu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
EPS = 1e-6
E4M3 = torch.float8_e4m3fn
# A row's sum of squares passes at most 16384 / 1024 * 2 = 32 sums in a thread, 6 in the wave and 16 across waves (54
# roundings, halved by the root); division, eps, root and two products add 6.
NORM_U = (54 / 2 + 6) * tu.U


def make(rows, cols, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x, r, adj, adj_h = (torch.randn(rows, cols, generator=g).to(dtype).cuda() for _ in range(4))
    w = (1 + 0.2 * torch.randn(cols, generator=g)).to(dtype).cuda()
    return x, 3 * r, w, adj, adj_h


def unit64(h):
    h = h.double()
    return h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)


SIZES = [(1, 1), (3, 7), (5, 64), (2, 511), (4, 512), (7, 1003), (3, 1024), (2, 2047), (3, 4096), (2, 4100), (1, 8192),
         (2, 16383), (3, 16384), (600, 136), (100, 32), (77, 33), (50, 128), (33, 129), (19, 256)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_norm(rows, cols, dtype, residual):
    import differentiable_cholesky_amd as dc
    x, r, w, _, _ = make(rows, cols, dtype)
    y, h = dc.chol_rmsnorm(x, w, residual=r if residual else None, eps=EPS)
    assert torch.equal(h, (x.float() + r.float()).to(dtype) if residual else x)
    ref = unit64(h) * w.double()
    tu.near(y, ref, (NORM_U + tu.HALF[dtype] * (1 + NORM_U)) * ref.abs() + tu.TINY[dtype], "y")


def check_quant(y, q, scale, group, what):
    rows, cols = y.shape
    size = group or cols
    full = torch.nn.functional.pad(y, (0, -cols % size)).view(rows, -1, size)
    most = full.abs().amax(2)
    want = torch.where(most > 0, most / 448, 1.0)
    tu.near(scale, want, (NORM_U + 3 * tu.U) * want, what + " scale")
    s = scale.double().repeat_interleave(size, 1)[:, :cols]
    # half a step: relative 2^-4 of the value, or 2^-10 below the normal codes
    bound = 2.0 ** -4 * y.abs() * (1 + 2 * NORM_U) + 2.0 ** -10 * s + 2 * NORM_U * y.abs()
    tu.near(q.float().double() * s, y, bound, what + " q")
    codes = torch.nn.functional.pad(q.float(), (0, -cols % size)).view(rows, -1, size).abs().amax(2)
    assert (codes == torch.where(most > 0, 448.0, 0.0)).all()


@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (5, 64), (2, 200), (7, 1003), (3, 4096), (2, 4100), (2, 16383)])
def test_quant(rows, cols, dtype, group):
    import differentiable_cholesky_amd as dc
    residual = cols % 2 == 0
    x, r, w, _, _ = make(rows, cols, dtype, seed=1)
    q, scale, h = dc.chol_rmsnorm_quant(x, w, residual=r if residual else None, group=group, eps=EPS)
    assert torch.equal(h, (x.float() + r.float()).to(dtype) if residual else x)
    check_quant(unit64(h) * w.double(), q, scale, group, "quant")


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(500, 1003), (64, 4096), (3000, 130)])
def test_codes_are_those_of_64_bits(rows, cols, dtype, group):
    """A code is rounded from a value that is right to half a step of fp32."""
    import differentiable_cholesky_amd as dc
    x, _, w, _, _ = make(rows, cols, dtype, seed=8)
    q, _, _ = dc.chol_rmsnorm_quant(x, w, group=group, eps=EPS)
    p = x.double() * w.double()
    size = group or cols
    most = torch.nn.functional.pad(p.abs(), (0, -cols % size)).view(rows, -1, size).amax(2)
    code = (p * (448 / most).repeat_interleave(size, 1)[:, :cols]).float().to(E4M3)
    assert torch.equal(q.view(torch.uint8), code.view(torch.uint8))


def test_quant_of_zeros_nan_and_tiny_rows():
    import differentiable_cholesky_amd as dc
    x, _, w, _, _ = make(5, 300, torch.float32, seed=2)
    x[0] = 0
    x[1, 7] = float("nan")
    x[2, 130:200] = 0
    x[3] = 1e-38
    x[4, 250] = float("inf")
    q, scale, _ = dc.chol_rmsnorm_quant(x, w, group=64, eps=EPS)
    f = q.float()
    assert (scale[0] == 1).all() and not f[0].any()
    assert (scale[1] == 1).all() and torch.isnan(f[1]).all()
    assert torch.isfinite(f[2]).all() and not f[2, 130:200].any()
    assert torch.isfinite(f[3]).all() and torch.isfinite(scale[3]).all()
    # an infinite mean leaves 0 for finite elements and NaN for the infinite one
    assert torch.isnan(f[4, 250]) and not f[4, :250].any() and (scale[4] == 1).all()
    w[9] = float("inf")
    q, scale, _ = dc.chol_rmsnorm_quant(x[2:3], w, group=64, eps=EPS)
    assert torch.isinf(scale[0, 0]) and torch.isfinite(scale[0, 1:]).all()
    assert torch.isfinite(q.float()[0, 64:]).all()


ADJ_SIZES = SIZES + [(513, 520), (2100, 130), (1025, 2050), (20000, 60), (9000, 90), (5000, 250)]


@pytest.mark.parametrize("past", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", ADJ_SIZES)
def test_adjoint(rows, cols, dtype, past):
    import differentiable_cholesky_amd as dc
    h, _, w, adj, adj_h = make(rows, cols, dtype, seed=3)
    dx, dw = dc.chol_rmsnorm_adjoint(h, w, adj, adjH=adj_h if past else None, eps=EPS)
    f, a, g = h.double(), adj.double(), adj.double() * w.double()
    s = 1 / torch.sqrt(f.square().mean(1, keepdim=True) + EPS)
    along = (g * f).mean(1, keepdim=True)
    ref = s * (g - f * s * s * along)
    size = s * (g.abs() + f.abs() * s * s * (g * f).abs().mean(1, keepdim=True))
    if past:
        ref, size = ref + adj_h.double(), size + adj_h.double().abs()
    # three powers of s, the sum of g h (54 roundings and 2 products) and 6 more
    u = 3 * NORM_U + 64 * tu.U
    tu.near(dx, ref, u * size + tu.HALF[dtype] * (ref.abs() + u * size) + tu.TINY[dtype], "adjX")
    terms = a * f * s
    tu.near(dw, terms.sum(0), (NORM_U + (rows + 8) * tu.U) * terms.abs().sum(0), "adjW")
    base = torch.ones_like(dw)
    _, dw2 = dc.chol_rmsnorm_adjoint(h, w, adj, adjH=adj_h if past else None, eps=EPS, adjW=base, accumulate=True)
    assert dw2 is base and torch.equal(dw2, 1 + dw)


def test_adjoint_against_differences():
    import differentiable_cholesky_amd as dc
    h, _, w, adj, adj_h = make(4, 70, torch.float32, seed=4)
    dx, dw = dc.chol_rmsnorm_adjoint(h, w, adj, adjH=adj_h, eps=EPS)

    def loss(h, w):
        unit = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
        return (unit * w * adj.double()).sum() + (h * adj_h.double()).sum()

    g = torch.Generator().manual_seed(5)
    for k, (x, d) in enumerate(((h, dx), (w, dw))):
        v = torch.randn(x.shape, generator=g).cuda().double()
        up, down = [h.double(), w.double()], [h.double(), w.double()]
        up[k] = up[k] + 1e-5 * v
        down[k] = down[k] - 1e-5 * v
        slope = (loss(*up) - loss(*down)) / 2e-5
        scale = (d.double() * v).abs().sum()
        assert abs((d.double() * v).sum() - slope) <= 200 * tu.U * scale + 1e-6 * (1 + slope.abs())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layouts_and_in_place(dtype):
    import differentiable_cholesky_amd as dc
    rows, cols = 37, 515
    x, r, w, adj, adj_h = make(rows, cols, dtype, seed=6)
    y, h = dc.chol_rmsnorm(x, w, residual=r, eps=EPS)
    wide = torch.full((rows, 2 * cols + 5), 7.0, dtype=dtype, device="cuda")
    xs, rs = wide[:, 1:1 + cols], wide[:, 2 + cols:2 + 2 * cols]
    xs.copy_(x), rs.copy_(r)
    dc.chol_rmsnorm(xs, w, residual=rs, eps=EPS, y=xs, h=rs)
    assert torch.equal(xs, y) and torch.equal(rs, h)
    assert (wide[:, 0] == 7).all() and (wide[:, 1 + cols] == 7).all() and (wide[:, 2 + 2 * cols:] == 7).all()
    y3, h3 = dc.chol_rmsnorm(x.view(1, rows, cols), w, residual=r.view(1, rows, cols), eps=EPS)
    assert y3.shape == (1, rows, cols) and torch.equal(y3[0], y) and torch.equal(h3[0], h)
    dx, dw = dc.chol_rmsnorm_adjoint(h, w, adj, adjH=adj_h, eps=EPS)
    for over in (0, 1, 2):
        args = [h.clone(), adj.clone(), adj_h.clone()]
        got, _ = dc.chol_rmsnorm_adjoint(args[0], w, args[1], adjH=args[2], eps=EPS, adjX=args[over])
        assert torch.equal(got, dx)
    q, scale, _ = dc.chol_rmsnorm_quant(x, w, group=128, eps=EPS)
    qw = torch.zeros(rows, cols + 3, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    q2, s2, _ = dc.chol_rmsnorm_quant(x, w, group=128, eps=EPS, q=qw[:, 1:1 + cols])
    assert torch.equal(q2.float(), q.float()) and torch.equal(s2, scale)
    assert not qw.view(torch.uint8)[:, [0, cols + 1, cols + 2]].any()


def test_empty():
    import differentiable_cholesky_amd as dc
    w = torch.ones(8, device="cuda")
    e = torch.empty(0, 8, device="cuda")
    assert dc.chol_rmsnorm(e, w)[0].shape == (0, 8)
    q, scale, _ = dc.chol_rmsnorm_quant(e, w, group=32)
    assert q.shape == (0, 8) and scale.shape == (0, 1)
    dx, dw = dc.chol_rmsnorm_adjoint(e, w, e)
    assert dx.shape == (0, 8) and not dw.any()
    keep = torch.ones(8, device="cuda")
    dc.chol_rmsnorm_adjoint(e, w, e, adjW=keep, accumulate=True)
    assert (keep == 1).all()


def test_captured_into_a_graph():
    import differentiable_cholesky_amd as dc
    h, r, w, adj, adj_h = make(700, 1030, torch.bfloat16, seed=7)
    dc.chol_rmsnorm_adjoint(h, w, adj)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, s = dc.chol_rmsnorm(h, w, residual=r)
        dx, dw = dc.chol_rmsnorm_adjoint(s, w, adj, adjH=adj_h)
    for _ in range(4):
        h.mul_(0.5)
        adj.mul_(2)
        want = dc.chol_rmsnorm(h, w, residual=r)
        grads = dc.chol_rmsnorm_adjoint(want[1], w, adj, adjH=adj_h)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((y, s, dx, dw), (*want, *grads)):
            assert torch.equal(a, b)


def test_more_rows_than_one_launch_takes():
    import differentiable_cholesky_amd as dc
    rows, cols = (1 << 26) + 5, 3
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-6:] = torch.randn(6, cols, device="cuda").bfloat16()
    w = torch.tensor([1.0, 2.0, 0.5], device="cuda").bfloat16()
    y, _ = dc.chol_rmsnorm(x, w, eps=EPS)
    assert torch.equal(y[-6:], dc.chol_rmsnorm(x[-6:].clone(), w, eps=EPS)[0])
    assert torch.equal(y[:-6].amin(0), w) and torch.equal(y[:-6].amax(0), w)


def test_rows_beyond_the_caches():
    """A call that moves more than the last cache holds gives what its slices give."""
    import differentiable_cholesky_amd as dc
    rows, cols = 9000, 4100
    x, r, w, adj, adj_h = (t.cuda() for t in make(rows, cols, torch.bfloat16, seed=9))
    y, h = dc.chol_rmsnorm(x, w, residual=r)
    q, scale, _ = dc.chol_rmsnorm_quant(x, w, residual=r, group=64)
    dx, _ = dc.chol_rmsnorm_adjoint(h, w, adj, adjH=adj_h)
    for part in (slice(0, 2500), slice(2500, 5000), slice(5000, 7500), slice(7500, rows)):
        y1, h1 = dc.chol_rmsnorm(x[part], w, residual=r[part])
        assert torch.equal(y1, y[part]) and torch.equal(h1, h[part])
        q1, s1, _ = dc.chol_rmsnorm_quant(x[part], w, residual=r[part], group=64)
        assert torch.equal(q1.float(), q[part].float()) and torch.equal(s1, scale[part])
        assert torch.equal(dc.chol_rmsnorm_adjoint(h1, w, adj[part], adjH=adj_h[part])[0], dx[part])


def test_more_elements_than_32_bits_count():
    import differentiable_cholesky_amd as dc
    rows, cols = 1100000, 2048                                # 2.3e9 elements
    g = torch.Generator(device="cuda").manual_seed(10)
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.empty(cols, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    part = x[-100:].clone()
    q, scale, _ = dc.chol_rmsnorm_quant(x, w, group=64)
    q1, s1, _ = dc.chol_rmsnorm_quant(part, w, group=64)
    assert torch.equal(q[-100:].float(), q1.float()) and torch.equal(scale[-100:], s1)
    y, _ = dc.chol_rmsnorm(x, w)
    assert torch.equal(y[-100:], dc.chol_rmsnorm(part, w)[0])
    dx, _ = dc.chol_rmsnorm_adjoint(x, w, y, adjX=y)
    assert torch.equal(dx[-100:], dc.chol_rmsnorm_adjoint(part, w, dc.chol_rmsnorm(part, w)[0])[0])
