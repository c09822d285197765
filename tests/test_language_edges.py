"""Infinite values, padding, offsets and extreme scales of the convolution's, the scan's and the token log
probabilities' inputs, on the GPU."""
import math

import pytest

import language_util as lu
import train_util as tu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
KEYS = ("u", "delta", "A", "B", "C", "D", "z", "bias", "h0")
STEPWISE = ("u", "delta", "B", "C", "z", "adj")


# -------------------------------------------------------------------- scan ----

def scan_inputs(batch, length, dim, groups, states, dtype=torch.float32, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    s = {"u": r(batch, length, dim).to(dtype), "delta": (r(batch, length, dim) - 2).to(dtype),
         "A": -torch.exp(r(dim, states) * 0.7), "B": r(batch, length, groups, states).to(dtype),
         "C": r(batch, length, groups, states).to(dtype), "D": r(dim), "z": r(batch, length, dim).to(dtype),
         "bias": r(dim) * 0.5, "h0": r(batch, dim, states), "adj": r(batch, length, dim).to(dtype),
         "adj_last": r(batch, dim, states)}
    return {k: t.cuda() for k, t in s.items()}


def scan_forward(s, **more):
    import differentiable_cholesky_amd as dc
    return dc.chol_selective_scan(s["u"], s["delta"], s["A"], s["B"], s["C"], **{
        **dict(D=s["D"], z=s["z"], bias=s["bias"], h0=s["h0"]), **more})


def scan_adjoint(s, starts):
    import differentiable_cholesky_amd as dc
    return dict(zip(KEYS, dc.chol_selective_scan_adjoint(s["u"], s["delta"], s["A"], s["B"], s["C"], starts, s["adj"], D=s["D"],
                                                         z=s["z"], bias=s["bias"], adjHlast=s["adj_last"])))


# lengths that are no multiples of the kernels' blocks, one segment and several, channels that fill no wave
ODD = [(1, 1, 5, 1, 16), (2, 2, 20, 1, 16), (1, 37, 40, 2, 16), (1, 90, 34, 1, 5), (1, 905, 24, 1, 16), (2, 70, 18, 1, 32),
       (1, 333, 20, 1, 50), (8, 150, 1600, 2, 16)]


@pytest.mark.parametrize("batch,length,dim,groups,states", ODD)
def test_an_infinite_entry_of_the_last_row(batch, length, dim, groups, states):
    """B infinite in the last step: the state there, and the sums that hold it; nothing else."""
    s = scan_inputs(batch, length, dim, groups, states, seed=length)
    y, last, starts = scan_forward(s, save=True)
    clean = scan_adjoint(s, starts)
    n = states // 2
    s["B"][0, -1, groups - 1, n] = math.inf
    y2, last2, starts2 = scan_forward(s, save=True)
    hit = torch.arange(dim, device="cuda") // (dim // groups) == groups - 1
    assert torch.equal(last2[0, hit, n], s["u"][0, -1, hit].sign() * math.inf)
    last2[0, hit, n] = last[0, hit, n]
    assert torch.equal(last2, last) and torch.equal(starts2, starts)
    assert torch.isinf(y2[0, -1, hit]).all()
    y2[0, -1, hit] = y[0, -1, hit]
    assert torch.equal(y2, y)
    # backward: sums that hold B or the state after the last step are infinite (or not a number), those before are not
    got = scan_adjoint(s, starts2)
    for k in ("B", "D", "h0"):
        assert torch.equal(got[k], clean[k]), k
    for k in ("u", "delta", "z", "C"):
        assert torch.equal(got[k][:, :-1], clean[k][:, :-1]) and torch.equal(got[k][1:], clean[k][1:]), k


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,length,dim,groups,states", ODD)
def test_states_that_forget_at_once(batch, length, dim, groups, states, dtype):
    """A of -inf: exp(dt A) is 0 for any step, and what A multiplies in the gradients is 0 too."""
    s = scan_inputs(batch, length, dim, groups, states, dtype, seed=length)
    gone = torch.rand(dim, states, generator=torch.Generator().manual_seed(1)).cuda() < 0.3
    gone[:, 0] = False
    gone[-1, :] = True
    # (the 64-bit form with steps so long that the exponential is 0: the smallest dt here is above 1e-4)
    s["A"] = torch.where(gone, -1e8, s["A"])
    ref = lu.Scan64(*(s[k] for k in KEYS))
    s["A"] = torch.where(gone, -math.inf, s["A"])
    y, last, starts = scan_forward(s, save=True)
    (y64, l64), (yb, lb) = ref.forward()
    tu.near(y, y64, yb, "y")
    tu.near(last, l64, lb, "last")
    got = scan_adjoint(s, starts)
    out, bounds = ref.adjoint(s["adj"], s["adj_last"])
    for k in KEYS:
        tu.near(got[k].view(out[k].shape), out[k], bounds[k], f"adjoint {k}")
    # the same a token at a time, and NaN stays one
    kept, rows = s["h0"].clone(), []
    for t in range(min(length, 40)):
        part = {k: x[:, t:t + 1] if k in STEPWISE else x for k, x in s.items()}
        rows.append(scan_forward(part, h0=kept, hlast=kept)[0])
    tu.near(torch.cat(rows, 1), y64[:, :40], yb[:, :40], "stepped y")
    s["A"][0, 0] = math.nan
    y2, last2, _ = scan_forward(s)
    assert torch.isnan(y2[:, :, 0]).all() and torch.isnan(last2[:, 0, 0]).all() and torch.equal(last2[:, 1:], last[:, 1:])
