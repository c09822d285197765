"""chol_recurrence and chol_recurrence_adjoint against 64 bits, on the GPU."""
import pytest

import train_util as tu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def make(batch, length, dim, dtype, gate, state, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = torch.exp(torch.randn(batch, length, dim, generator=g) - 2.0)
    a = (-r if gate == "log" else torch.exp(-r) * torch.sign(torch.randn(batch, length, dim, generator=g))).to(dtype)
    b = torch.randn(batch, length, dim, generator=g).to(dtype)
    adj = torch.randn(batch, length, dim, generator=g).to(dtype)
    h0 = torch.randn(batch, dim, generator=g) if state else None
    last = torch.randn(batch, dim, generator=g) if state else None
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    return tuple(cuda(t) for t in (a, b, adj, h0, last))


def check_forward(a, b, h0, gate, h, last, what):
    h64, l64, size, lsize = tu.recurrence64(a, b, h0, gate)
    u = tu.steps_u(a.shape[1], gate)
    t = a.dtype
    tu.near(h, h64, (1 + tu.HALF[t]) * u * size + tu.HALF[t] * h64.abs() + tu.TINY[t], what + " h")
    tu.near(last, l64, u * lsize + tu.TINY[torch.float32], what + " last")


def check_adjoint(a, h, adj, h0, adj_last, gate, got, what):
    ref, size = tu.recurrence_adjoint64(a, h, adj, h0, adj_last, gate)
    u = tu.steps_u(a.shape[1], gate) + 4 * tu.U
    for name, x, r, s, t in zip(("adjA", "adjB", "adjH0"), got, ref, size, (a.dtype, a.dtype, torch.float32)):
        half = tu.HALF[t] if name != "adjH0" else 0.0
        tu.near(x, r, (1 + half) * u * s + half * r.abs() + tu.TINY[t], f"{what} {name}")


SIZES = [(1, 1, 1), (2, 1, 5), (1, 2, 64), (3, 15, 65), (2, 16, 128), (1, 17, 130), (2, 127, 33), (1, 129, 256), (5, 300, 7),
         (1, 1025, 100), (2, 2049, 66), (1, 5000, 31), (2, 3000, 16), (1, 2100, 32), (3, 700, 64), (1, 9000, 3), (9, 257, 17)]


@pytest.mark.parametrize("gate", ["linear", "log"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,length,dim", SIZES)
def test_forward_and_adjoint(batch, length, dim, dtype, gate):
    import differentiable_cholesky_amd as dc
    state = (batch + length + dim) % 2 == 0
    a, b, adj, h0, adj_last = make(batch, length, dim, dtype, gate, state)
    h, last = dc.chol_recurrence(a, b, h0=h0, gate=gate)
    check_forward(a, b, h0, gate, h, last, "forward")
    got = dc.chol_recurrence_adjoint(a, h, adj, h0=h0, adjHlast=adj_last, gate=gate)
    check_adjoint(a, h, adj, h0, adj_last, gate, got, "adjoint")


@pytest.mark.parametrize("dtype", TYPES)
def test_one_sequence_longer_than_any_run_kept_at_once(dtype):
    import differentiable_cholesky_amd as dc
    a, b, adj, h0, adj_last = make(1, 40000, 130, dtype, "linear", True)
    h, last = dc.chol_recurrence(a, b, h0=h0)
    check_forward(a, b, h0, "linear", h, last, "long")
    got = dc.chol_recurrence_adjoint(a, h, adj, h0=h0, adjHlast=adj_last)
    check_adjoint(a, h, adj, h0, adj_last, "linear", got, "long")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("length", [1, 70, 1500])
def test_layouts(dtype, length):
    """Sequence-major storage, column slices of a joint buffer at odd offsets, padded rows."""
    import differentiable_cholesky_amd as dc
    batch, dim = 3, 67
    a, b, adj, h0, adj_last = make(batch, length, dim, dtype, "log", True, seed=3)
    h, last = dc.chol_recurrence(a, b, h0=h0, gate="log")
    grads = dc.chol_recurrence_adjoint(a, h, adj, h0=h0, adjHlast=adj_last, gate="log")

    joint = torch.full((batch, length, 2 * dim + 3), 7.0, dtype=dtype, device="cuda")
    aj, bj = joint[..., 1:1 + dim], joint[..., 1 + dim:1 + 2 * dim]
    aj.copy_(a), bj.copy_(b)
    major = torch.full((length, batch, dim), 7.0, dtype=dtype, device="cuda").transpose(0, 1)
    h2, last2 = dc.chol_recurrence(aj, bj, h0=h0, h=major, gate="log")
    assert torch.equal(h2, h) and torch.equal(last2, last)
    out = torch.full((batch, length, 2 * dim + 3), 7.0, dtype=dtype, device="cuda")
    da, db = out[..., 1:1 + dim], out[..., 1 + dim:1 + 2 * dim]
    got = dc.chol_recurrence_adjoint(aj, major, adj, h0=h0, adjHlast=adj_last, adjA=da, adjB=db, gate="log")
    for x, y in zip(got, grads):
        assert torch.equal(x, y)
    assert (out[..., 0] == 7).all() and (out[..., 1 + 2 * dim:] == 7).all()
    assert (joint[..., 0] == 7).all() and (joint[..., 1 + 2 * dim:] == 7).all()


@pytest.mark.parametrize("length", [1, 33, 2500])
def test_in_place(length):
    import differentiable_cholesky_amd as dc
    a, b, adj, h0, adj_last = make(2, length, 129, torch.bfloat16, "linear", True, seed=4)
    h, last = dc.chol_recurrence(a, b, h0=h0)
    x, s = b.clone(), h0.clone()
    dc.chol_recurrence(a, x, h0=s, hlast=s, h=x)
    assert torch.equal(x, h) and torch.equal(s, last)
    grads = dc.chol_recurrence_adjoint(a, h, adj, h0=h0, adjHlast=adj_last)
    da, db, d0 = a.clone(), adj.clone(), adj_last.clone()
    dc.chol_recurrence_adjoint(da, h, db, h0=h0, adjHlast=d0, adjA=da, adjB=db, adjH0=d0)
    for p, q in zip((da, db, d0), grads):
        assert torch.equal(p, q)


def test_steps_one_at_a_time_continue_a_sequence():
    import differentiable_cholesky_amd as dc
    a, b, _, h0, _ = make(4, 20, 300, torch.float32, "log", True, seed=5)
    state = h0.clone()
    rows = [dc.chol_recurrence(a[:, t:t + 1], b[:, t:t + 1], h0=state, hlast=state, gate="log")[0] for t in range(20)]
    check_forward(a, b, h0, "log", torch.cat(rows, 1), state, "stepped")


def test_empty_sequence_and_empty_batch():
    import differentiable_cholesky_amd as dc
    h0 = torch.randn(3, 10, device="cuda")
    e = torch.empty(3, 0, 10, dtype=torch.bfloat16, device="cuda")
    h, last = dc.chol_recurrence(e, e, h0=h0)
    assert h.shape == e.shape and torch.equal(last, h0)
    assert not dc.chol_recurrence(e, e)[1].any()
    _, _, d0 = dc.chol_recurrence_adjoint(e, e, e, adjHlast=h0)
    assert torch.equal(d0, h0)
    z = torch.empty(0, 4, 10, device="cuda")
    assert dc.chol_recurrence(z, z)[0].shape == z.shape


@pytest.mark.parametrize("length", [5, 1200])
def test_closed_gates_and_non_finite_inputs_stay_in_their_channel(length):
    """A gate of zero (log: -inf) cuts the sequence; inf and NaN reach later steps of their channel only."""
    import differentiable_cholesky_amd as dc
    a, b, _, h0, _ = make(1, length, 130, torch.float32, "log", True, seed=6)
    at = length // 2
    a[0, at] = float("-inf")
    h, last = dc.chol_recurrence(a, b, h0=h0, gate="log")
    assert torch.equal(h[0, at], b[0, at])
    check_forward(a, b, h0, "log", h, last, "closed")
    clean = h.clone()
    b[0, at, 3], b[0, at, 70] = float("nan"), float("inf")
    h, last = dc.chol_recurrence(a, b, h0=h0, gate="log")
    assert torch.isnan(h[0, at:, 3]).all() and not torch.isfinite(h[0, at:, 70]).any()
    keep = torch.ones(130, dtype=torch.bool, device="cuda")
    keep[[3, 70]] = False
    assert torch.equal(h[..., keep], clean[..., keep]) and torch.equal(h[:, :at], clean[:, :at])


def test_adjoint_against_differences():
    """The loss is linear in b and h0, so its differences there are exact in 64 bits; for a they are centred."""
    import differentiable_cholesky_amd as dc
    a, b, adj, h0, adj_last = make(2, 40, 9, torch.float32, "log", True, seed=7)
    h, _ = dc.chol_recurrence(a, b, h0=h0, gate="log")
    da, db, d0 = dc.chol_recurrence_adjoint(a, h, adj, h0=h0, adjHlast=adj_last, gate="log")

    def loss(a, b, h0):
        h, last, _, _ = tu.recurrence64(a, b, h0, "log")
        return (h * adj.double()).sum() + (last * adj_last.double()).sum()

    g = torch.Generator().manual_seed(8)
    for k, (x, d) in enumerate(((a, da), (b, db), (h0, d0))):
        v = torch.randn(x.shape, generator=g).cuda().double()
        eps = 1e-5
        args = [t.double() for t in (a, b, h0)]
        up, down = list(args), list(args)
        up[k], down[k] = args[k] + eps * v, args[k] - eps * v
        slope = (loss(*up) - loss(*down)) / (2 * eps)
        along = (d.double() * v).sum()
        # fp32 roundings of every term (40 steps), and the differences' own eps^2 and 1e-16 / eps
        scale = (d.double() * v).abs().sum()
        assert abs(along - slope) <= 400 * tu.U * scale + 1e-6 * (1 + slope.abs())


def test_another_stream():
    import differentiable_cholesky_amd as dc
    a, b, adj, h0, _ = make(2, 3000, 128, torch.bfloat16, "linear", True, seed=9)
    want = dc.chol_recurrence(a, b, h0=h0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dc.chol_recurrence(a, b, h0=h0, stream=side)
    with torch.cuda.stream(side):
        copies = [t.clone() for t in got]
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(copies, want):
        assert torch.equal(x, y)


def test_captured_into_a_graph():
    import differentiable_cholesky_amd as dc
    a, b, adj, h0, adj_last = make(1, 3000, 140, torch.bfloat16, "linear", True, seed=10)
    args = dict(h0=h0)
    h, last = dc.chol_recurrence(a, b, **args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gh, gl = dc.chol_recurrence(a, b, **args)
        gg = dc.chol_recurrence_adjoint(a, gh, adj, h0=h0, adjHlast=adj_last)
    for k in range(4):
        b.mul_(0.5)
        want = dc.chol_recurrence(a, b, **args)
        grads = dc.chol_recurrence_adjoint(a, want[0], adj, h0=h0, adjHlast=adj_last)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((gh, gl, *gg), (*want, *grads)):
            assert torch.equal(x, y), k


@pytest.mark.parametrize("dtype", TYPES)
def test_equal_calls_give_equal_bits(dtype):
    """Whatever order the workgroups of a long sequence finish in."""
    import differentiable_cholesky_amd as dc
    a, b, adj, h0, adj_last = make(2, 20000, 260, dtype, "log", True, seed=11)
    h, last = dc.chol_recurrence(a, b, h0=h0, gate="log")
    grads = dc.chol_recurrence_adjoint(a, h, adj, h0=h0, adjHlast=adj_last, gate="log")
    for k in range(20):
        again = dc.chol_recurrence(a, b, h0=h0, gate="log")
        assert torch.equal(again[0], h) and torch.equal(again[1], last), k
        for x, y in zip(dc.chol_recurrence_adjoint(a, h, adj, h0=h0, adjHlast=adj_last, gate="log"), grads):
            assert torch.equal(x, y), k


def test_more_elements_than_32_bits_count():
    import differentiable_cholesky_amd as dc
    length, dim, tail = 70001, 32768, 8                       # 2.3e9 elements
    g = torch.Generator(device="cuda").manual_seed(12)
    a = torch.empty(1, length, dim, dtype=torch.bfloat16, device="cuda").uniform_(0.5, 0.99, generator=g)
    b = torch.empty_like(a).uniform_(-1, 1, generator=g)
    h, last = dc.chol_recurrence(a, b)
    cut = slice(dim - tail, dim)
    h1, last1 = dc.chol_recurrence(a[..., cut], b[..., cut])
    assert torch.equal(h[..., cut], h1) and torch.equal(last[:, cut], last1)
    adj = b[0, -50:, cut].double()
    da, db, _ = dc.chol_recurrence_adjoint(a, h, b, adjB=b)
    for t in range(length - 50, length):
        want = db[0, t, cut].double() * h[0, t - 1, cut].double()
        # adjB is lam rounded once, and adjA rounds its product with lam once
        assert ((da[0, t, cut].double() - want).abs() <= 2.02 * tu.HALF[torch.bfloat16] * want.abs() + 1e-30).all(), t
        if t + 1 < length:
            after = a[0, t + 1, cut].double() * db[0, t + 1, cut].double()
            lam = adj[t - length + 50] + after
            assert ((db[0, t, cut].double() - lam).abs() <= 1.01 * tu.HALF[torch.bfloat16] * (lam.abs() + after.abs())).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("length", [1, 70, 1500])
def test_joint_buffers_in_either_order(dtype, length):
    """a and h, then adjA and adjB, as column slices of one buffer: sequence-major, and batch elements padded by less
    than a row."""
    import differentiable_cholesky_amd as dc
    batch, dim = 3, 67
    a, b, adj, h0, adj_last = make(batch, length, dim, dtype, "log", True, seed=13)
    h, last = dc.chol_recurrence(a, b, h0=h0, gate="log")
    grads = dc.chol_recurrence_adjoint(a, h, adj, h0=h0, adjHlast=adj_last, gate="log")

    def joint(major):
        wide = 2 * dim + 3
        if major:
            return torch.full((length, batch, wide), 7.0, dtype=dtype, device="cuda").transpose(0, 1)
        flat = torch.full((batch * (length * wide + 5),), 7.0, dtype=dtype, device="cuda")
        return flat.as_strided((batch, length, wide), (length * wide + 5, wide, 1))

    for major in (True, False):
        x, y = joint(major), joint(major)
        one, other = slice(1, 1 + dim), slice(1 + dim, 1 + 2 * dim)
        x[..., one].copy_(a)
        got, end = dc.chol_recurrence(x[..., one], b, h0=h0, h=x[..., other], gate="log")
        assert torch.equal(got, h) and torch.equal(end, last) and torch.equal(x[..., one], a)
        back = dc.chol_recurrence_adjoint(x[..., one], x[..., other], adj, h0=h0, adjHlast=adj_last, adjA=y[..., one],
                                          adjB=y[..., other], gate="log")
        for p, q in zip(back, grads):
            assert torch.equal(p, q)
        for t in (x, y):
            assert (t[..., 0] == 7).all() and (t[..., 1 + 2 * dim:] == 7).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_exponentials_of_every_gate(dtype):
    """One step from a state of one gives the gate in fp32, both ways.  The hardware's 2^y is within a step of fp32
    (2 u), the second part's addition half a step (u), and what the series leaves out (1.5 u) and the roundings of
    that part are within another 2 u."""
    import differentiable_cholesky_amd as dc
    if dtype is torch.float32:
        x = torch.logspace(-8, 2.5, 1 << 15, dtype=torch.float64).float()
        a = torch.cat([x, -x])
    else:
        a = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(dtype)
    a = a.cuda().view(1, 1, -1)
    one = torch.ones(1, a.shape[-1], device="cuda")
    zero = torch.zeros_like(a)
    _, up = dc.chol_recurrence(a, zero, h0=one, gate="log")
    _, _, back = dc.chol_recurrence_adjoint(a, zero, zero, h0=one, adjHlast=one, gate="log")
    x = a.double().view(1, -1)
    want = x.exp()
    for got in (up, back):
        assert torch.isnan(got[torch.isnan(x)]).all()
        assert (got[x < -105] == 0).all() and torch.isinf(got[x > 90]).all()
        usual = (x > -87) & (x < 88.5)
        assert ((got.double() - want).abs() <= 5 * tu.U * want)[usual].all()
