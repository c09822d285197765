"""chol_selective_scan and chol_selective_scan_adjoint against 64 bits, on the GPU."""
import pytest

import language_util as lu
import train_util as tu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
NAMES = ("u", "delta", "A", "B", "C", "D", "z", "bias", "h0")


def make(batch, length, dim, groups, states, dtype, state=True, full=True, seed=0):
    """Inputs as a dict, with gradients `adj` and `adj_last`.  full False: no D, z and bias."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    s = {"u": r(batch, length, dim).to(dtype), "delta": (r(batch, length, dim) - 2).to(dtype),
         "A": -torch.exp(r(dim, states) * 0.7), "B": r(batch, length, groups, states).to(dtype),
         "C": r(batch, length, groups, states).to(dtype), "D": r(dim) if full else None,
         "z": r(batch, length, dim).to(dtype) if full else None, "bias": r(dim) * 0.5 if full else None,
         "h0": r(batch, dim, states) if state else None, "adj": r(batch, length, dim).to(dtype),
         "adj_last": r(batch, dim, states) if state else None}
    if groups == 1 and states % 2:
        s["B"], s["C"] = s["B"][:, :, 0], s["C"][:, :, 0]
    return {k: lu.cuda(t) for k, t in s.items()}


def forward(s, **more):
    import differentiable_cholesky_amd as dc
    return dc.chol_selective_scan(s["u"], s["delta"], s["A"], s["B"], s["C"], **{
        **dict(D=s["D"], z=s["z"], bias=s["bias"], h0=s["h0"]), **more})


def adjoint(s, starts, **more):
    import differentiable_cholesky_amd as dc
    return dc.chol_selective_scan_adjoint(s["u"], s["delta"], s["A"], s["B"], s["C"], starts, s["adj"], **{
        **dict(D=s["D"], z=s["z"], bias=s["bias"], adjHlast=s["adj_last"]), **more})


def check(s, what, softplus=True):
    import differentiable_cholesky_amd as dc
    ref = lu.Scan64(*(s[k] for k in ("u", "delta", "A", "B", "C", "D", "z", "bias", "h0")), softplus=softplus)
    y, last, starts = forward(s, save=True, softplus=softplus)
    (y64, l64), (yb, lb) = ref.forward()
    tu.near(y, y64, yb, what + " y")
    tu.near(last, l64, lb, what + " last")
    block = dc.chol_selective_scan_block(s["A"].shape[1])
    for k in range(starts.shape[1]):
        tu.near(starts[:, k], ref.h[k * block], ref.d[k * block] + 1e-40, f"{what} start {k}")
    plain = forward(s, softplus=softplus)
    assert torch.equal(plain[0], y) and torch.equal(plain[1], last) and plain[2] is None
    if s["u"].shape[1] == 0:
        return
    got = dict(zip(NAMES, adjoint(s, starts, softplus=softplus)))
    out, bounds = ref.adjoint(s["adj"], s["adj_last"])
    for k in NAMES:
        if s.get(k) is None and k != "h0":
            assert got[k] is None, k
        else:
            tu.near(got[k].view(out[k].shape), out[k], bounds[k], f"{what} adjoint {k}")


SIZES = [(1, 1, 1, 1, 1), (2, 1, 5, 1, 16), (3, 2, 16, 1, 16), (1, 3, 17, 1, 4), (2, 15, 40, 2, 16), (1, 16, 64, 1, 3),
         (2, 17, 33, 3, 5), (1, 64, 130, 1, 16), (2, 65, 34, 2, 11), (1, 129, 20, 1, 32), (3, 70, 24, 4, 17), (2, 33, 18, 1, 64),
         (1, 50, 200, 2, 33), (1, 200, 256, 2, 16), (2, 500, 36, 1, 16), (1, 333, 140, 7, 8), (17, 20, 12, 1, 16)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,length,dim,groups,states", SIZES)
def test_forward_and_adjoint(batch, length, dim, groups, states, dtype):
    odd = batch + length + dim
    check(make(batch, length, dim, groups, states, dtype, state=odd % 2 > 0, full=odd % 3 > 0, seed=odd), "scan")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,length,dim,states", [(1, 1500, 48, 16), (1, 1025, 16, 40), (2, 900, 16, 20)])
def test_longer_sequences(batch, length, dim, states, dtype):
    check(make(batch, length, dim, 1, states, dtype, seed=length), "long")


def test_many_channels_take_one_segment():
    check(make(8, 150, 1600, 2, 16, torch.bfloat16, seed=5), "wide")


def test_steps_without_softplus():
    s = make(2, 80, 30, 1, 16, torch.float32, seed=6)
    s["delta"] = torch.exp(s["delta"])
    s["bias"] = s["bias"].abs()
    check(s, "plain steps", softplus=False)


@pytest.mark.parametrize("states", [4, 16, 33])
@pytest.mark.parametrize("length", [1, 100])
def test_layouts(length, states):
    """Slices of joint buffers: u, B and C of one product, u and z of another, gradients in one buffer; sequence-major."""
    batch, dim, dtype = 3, 34, torch.bfloat16
    s = make(batch, length, dim, 1, states, dtype, seed=2)
    s["B"], s["C"] = (s[k].reshape(batch, length, states) for k in "BC")
    y, last, starts = forward(s, save=True)
    grads = adjoint(s, starts)

    def joint(*widths):
        whole = torch.full((batch, length, sum(widths) + 3), 7.0, dtype=dtype, device="cuda")
        return whole, [x for x in whole[..., 1:-2].split(widths, -1)]

    t = dict(s)
    one, (t["u"], t["B"], t["C"]) = joint(dim, states, states)
    two, (out, t["z"]) = joint(dim, dim)
    for k in ("u", "B", "C", "z"):
        t[k].copy_(s[k])
    t["delta"] = s["delta"].transpose(0, 1).contiguous().transpose(0, 1)
    got = forward(t, y=out, save=True)
    assert torch.equal(out, y) and torch.equal(got[1], last) and torch.equal(got[2], starts)
    assert torch.equal(t["z"], s["z"])
    three, (du, db, dc_, dz, dd) = joint(dim, states, states, dim, dim)
    got = adjoint(t, starts, adjU=du, adjB=db, adjC=dc_, adjZ=dz, adjDelta=dd)
    for p, q in zip(got, grads):
        assert torch.equal(p, q)
    for whole in (one, two, three):
        assert (whole[..., 0] == 7).all() and (whole[..., -2:] == 7).all()


@pytest.mark.parametrize("batch,length,dim", [(1, 1, 40), (2, 30, 20), (1, 700, 40), (1, 3000, 20)])
def test_in_place(batch, length, dim):
    """A state replaced in place, the output over an input, gradients over inputs."""
    s = make(batch, length, dim, 1, 16, torch.bfloat16, seed=4)
    y, last, starts = forward(s, save=True)
    grads = adjoint(s, starts)
    for over in ("u", "delta", "z"):
        for _ in range(3):
            t = {k: x.clone() for k, x in s.items()}
            forward(t, y=t[over], hlast=t["h0"])
            assert torch.equal(t[over], y) and torch.equal(t["h0"], last)
    t = {k: x.clone() for k, x in s.items()}
    got = adjoint(t, starts, adjU=t["u"], adjDelta=t["delta"], adjZ=t["adj"], adjB=t["B"], adjC=t["C"], adjH0=t["adj_last"])
    for p, q in zip(got, grads):
        assert torch.equal(p, q)


def test_steps_one_at_a_time_continue_a_sequence():
    s = make(3, 40, 50, 2, 16, torch.float32, seed=8)
    ref = lu.Scan64(*(s[k] for k in ("u", "delta", "A", "B", "C", "D", "z", "bias", "h0")))
    (y64, l64), (yb, lb) = ref.forward()
    kept, rows = s["h0"].clone(), []
    for t in range(40):
        part = {k: x[:, t:t + 1] if k in ("u", "delta", "B", "C", "z") else x for k, x in s.items()}
        if t == 20:       # a longer piece
            part = {k: x[:, 20:] if k in ("u", "delta", "B", "C", "z") else x for k, x in s.items()}
        rows.append(forward(part, h0=kept, hlast=kept)[0])
        if t == 20:
            break
    tu.near(torch.cat(rows, 1), y64, yb, "stepped y")
    tu.near(kept, l64, lb, "stepped last")


def test_empty_sequences_and_accumulated_gradients():
    s = make(2, 30, 20, 1, 16, torch.float32)
    e = {k: x[:, :0] if k in ("u", "delta", "B", "C", "z", "adj") else x for k, x in s.items()}
    y, last, starts = forward(e, save=True)
    assert y.shape == e["u"].shape and torch.equal(last, s["h0"]) and starts.shape == (2, 0, 20, 16)
    assert not forward({**e, "h0": None})[1].any()
    got = dict(zip(NAMES, adjoint(e, starts)))
    assert torch.equal(got["h0"], s["adj_last"]) and not any(got[k].any() for k in ("A", "D", "bias"))
    z = {k: x[:0] if k in ("u", "delta", "B", "C", "z", "adj", "h0", "adj_last") else x for k, x in s.items()}
    assert forward(z)[0].shape == z["u"].shape
    assert not any(x.any() for x in (adjoint(z, starts[:0].new_empty(0, 1, 20, 16))[k] for k in (2, 5, 7)))
    _, _, starts = forward(s, save=True)
    want = dict(zip(NAMES, adjoint(s, starts)))
    into = {k: torch.full_like(want[k], 2.0) for k in ("A", "D", "bias")}
    adjoint(s, starts, adjA=into["A"], adjD=into["D"], adjBias=into["bias"], accumulate=True)
    for k, x in into.items():
        assert torch.equal(x, 2.0 + want[k]), k


@pytest.mark.parametrize("length", [1, 90])
def test_non_finite_inputs_stay_in_their_channel(length):
    """Forward: from their step on.  Backward: the channel, and the gradients that are sums over channels."""
    s = make(1, length, 40, 2, 16, torch.float32, seed=3)
    y, last, starts = forward(s, save=True)
    grads = dict(zip(NAMES, adjoint(s, starts)))
    at = length // 2
    s["u"][0, at, 39] = float("nan")          # the last channel, whose values lanes past the end read as well
    y2, last2, starts2 = forward(s, save=True)
    assert torch.isnan(y2[0, at:, 39]).all() and torch.isnan(last2[0, 39]).all()
    y2[0, at:, 39], y[0, at:, 39] = 0, 0
    last2[0, 39], last[0, 39] = 0, 0
    assert torch.equal(y2, y) and torch.equal(last2, last)
    got = dict(zip(NAMES, adjoint(s, starts2)))
    for k in ("u", "delta", "z"):
        assert torch.equal(got[k][..., :39], grads[k][..., :39]), k
    for k in ("A", "D", "bias"):
        assert torch.equal(got[k][:39], grads[k][:39]), k
    for k in "BC":
        assert torch.equal(got[k][:, :, 0], grads[k][:, :, 0]), k


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("length", [1, 90, 900])
@pytest.mark.parametrize("key", ["delta", "B", "C", "z"])
def test_nan_of_any_input_reaches_the_results(key, length, softplus):
    """A step's NaN is in its results, and from there on in the state (but for C and z)."""
    s = make(1, length, 40, 1, 16, torch.float32, seed=3)
    if not softplus:
        s["delta"], s["bias"] = torch.exp(s["delta"]), s["bias"].abs()
    y, last, _ = forward(s, softplus=softplus)
    at = length // 2
    s[key][0, at, ..., 3] = float("nan")
    y2, last2, _ = forward(s, softplus=softplus)
    kept = key in ("C", "z")
    channels = torch.arange(40, device="cuda") == 3 if key in ("delta", "z") else torch.ones(40, dtype=torch.bool, device="cuda")
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[0, at:at + 1 if kept else length, channels] = True
    assert torch.equal(torch.isnan(y2), bad) and torch.equal(y2[~bad], y[~bad])
    if kept:
        assert torch.equal(last2, last)
    else:
        states = torch.arange(16, device="cuda") == 3 if key == "B" else torch.ones(16, dtype=torch.bool, device="cuda")
        assert torch.equal(torch.isnan(last2[0]), channels[:, None] & states)


def test_closed_and_open_steps():
    """Steps so long that the state is forgotten, and of zero, which leave it as it is."""
    s = make(1, 60, 20, 1, 16, torch.float32, full=False, seed=5)
    s["delta"][0, 30] = 1e4
    s["delta"][0, 40] = float("-inf")
    y, last, starts = forward(s, save=True)
    (y64, _), (yb, _) = lu.Scan64(*(s[k] for k in ("u", "delta", "A", "B", "C", "D", "z", "bias", "h0"))).forward()
    tu.near(y[:, :30], y64[:, :30], yb[:, :30], "before")
    # dt = 1e4: what was before is gone, h = dt u B
    h = 1e4 * s["u"][0, 30, :, None].double() * s["B"][0, 30].view(1, 16).double()
    tu.near(y[0, 30], (h * s["C"][0, 30].view(1, 16).double()).sum(1), 40 * tu.U * h.abs().sum(1) * 10, "closed")
    assert torch.isfinite(y).all() and torch.isfinite(last).all()
    got = adjoint(s, starts)
    assert all(torch.isfinite(x).all() for x in got if x is not None)
    assert not got[0][0, 40].any()            # no step, no gradient of its input


@pytest.mark.parametrize("length", [1, 400])
def test_captured_and_replayed(length):
    """A kept state carried on by a graph as by eager calls; two captured calls with workspaces of their own."""
    s = make(2, length, 50, 1, 16, torch.bfloat16, seed=11)
    _, _, starts = forward(s, save=True)
    adjoint(s, starts)
    a, b = s["h0"].clone(), s["h0"].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _, kept = forward(s, h0=a, hlast=a, save=True)
        grads = adjoint(s, kept)
    for _ in range(4):
        graph.replay()
        y2, _, kept2 = forward(s, h0=b, hlast=b, save=True)
        want = adjoint(s, kept2)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(a, b)
        for p, q in zip(grads, want):
            assert torch.equal(p, q)
        s["u"].mul_(-0.5)


def test_other_streams_and_workspaces():
    import differentiable_cholesky_amd as dc
    s = make(1, 1000, 50, 1, 16, torch.bfloat16, seed=12)
    y, _, starts = forward(s, save=True)
    want = adjoint(s, starts)
    sizes = [dc.chol_selective_scan_workspace_size(k, 1, 1000, 50, 1, 16) for k in (False, True)]
    ws = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = forward(s, workspace=ws[0], stream=side)
    grads = adjoint(s, starts, workspace=ws[1], stream=side)
    side.synchronize()
    assert torch.equal(got[0], y)
    for p, q in zip(grads, want):
        assert torch.equal(p, q)


def test_equal_calls_give_equal_bits():
    s = make(2, 700, 300, 1, 16, torch.bfloat16, seed=13)
    y, last, starts = forward(s, save=True)
    want = adjoint(s, starts)
    for _ in range(5):
        for p, q in zip(forward(s, save=True), (y, last, starts)):
            assert torch.equal(p, q)
        for p, q in zip(adjoint(s, starts), want):
            assert torch.equal(p, q)


def test_gradients_against_differences():
    s = make(1, 30, 6, 2, 5, torch.float32, seed=14)
    keys = ("u", "delta", "A", "B", "C", "D", "z", "bias", "h0")

    def f(*args):
        (y, last), _ = lu.Scan64(*args).forward()
        return (y * s["adj"].double()).sum() + (last * s["adj_last"].double()).sum()

    _, _, starts = forward(s, save=True)
    got = dict(zip(NAMES, adjoint(s, starts)))
    args = [s[k].double() for k in keys]
    g = torch.Generator().manual_seed(1)
    for i, k in enumerate(keys):
        way = torch.randn(args[i].shape, generator=g).double().cuda()
        step = 1e-5
        ends = [f(*(a + w * step * way if j == i else a for j, a in enumerate(args))) for w in (1, -1)]
        slope = (ends[0] - ends[1]) / (2 * step)
        size = (got[k].double() * way).abs().sum()
        # fp32 gradients through at most 30 steps of some 20 roundings, and a difference of order step^2
        assert abs((got[k].double() * way).sum() - slope) <= 600 * tu.U * size + 1e-7 * size, k
