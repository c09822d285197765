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


@pytest.mark.parametrize("batch,length,dim,groups,states", [c for c in ODD if c[1] <= 90])
def test_an_infinite_weight_of_the_last_row(batch, length, dim, groups, states):
    """C infinite in the last step: the gradient of that state is infinite all the way to the first, those of the others
    are as they were."""
    s = scan_inputs(batch, length, dim, groups, states, seed=length)
    _, last, starts = scan_forward(s, save=True)
    clean = scan_adjoint(s, starts)["h0"]
    n = states // 2
    s["C"][0, -1, groups - 1, n] = math.inf
    _, last2, starts2 = scan_forward(s, save=True)
    assert torch.equal(last2, last) and torch.equal(starts2, starts)
    got = scan_adjoint(s, starts2)["h0"]
    hit = torch.arange(dim, device="cuda") // (dim // groups) == groups - 1
    # (silu has the sign of z; these states' steps are short enough that no exponential, of a segment neither, is 0)
    assert torch.equal(got[0, hit, n], (s["adj"][0, -1, hit] * s["z"][0, -1, hit]).sign() * math.inf)
    got[0, hit, n] = clean[0, hit, n]
    assert torch.equal(got, clean)


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


# ------------------------------------------------------- log probabilities ----

def logit_inputs(rows, vocab, dtype, seed=0, std=3.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, vocab, generator=g) * std).to(dtype)
    tokens = torch.randint(0, vocab, (rows,), generator=g)
    gl, ge = torch.randn(rows, generator=g), torch.randn(rows, generator=g)
    return x.cuda(), tokens.cuda(), gl.cuda(), ge.cuda()


def check_logp(x, tokens, scale, top, what):
    """logp and top_logp to what their own size needs: the sum relative to the maximum, its logarithm, and the distance
    from the maximum; no rounding of lse."""
    import differentiable_cholesky_amd as dc
    got = dc.chol_token_logprob(x, tokens, scale=scale, top=top)
    y = x.double() * scale
    d = y - y.amax(1, keepdim=True)
    p = torch.exp(d)
    log_s = torch.log(p.sum(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    # a term is off by its exponent's size (3 U of it), the sum by its depth (lanes, waves, chunks); the logarithm by 2 U
    # and 2 U of itself; the distance by two roundings of its own, the result by one
    sum_err = (p * (3 * d.clamp(min=-1e4).abs() + 64 + 24)).sum(1, keepdim=True) * tu.U
    bound = lambda far: sum_err + 2 * tu.U * (1 + log_s) + 2 * tu.U * far.abs() + tu.U * (far - log_s).abs()  # noqa: E731
    far = d.gather(1, tokens[:, None])
    tu.near(got.logp[:, None], far - log_s, bound(far), what + " logp")
    assert (got.logp <= 0).all()
    if top:
        far = d.gather(1, got.top_ids)
        tu.near(got.top_logp, far - log_s, bound(far), what + " top")
        assert (got.top_logp <= 0).all() and (got.top_logp[:, 0] >= got.logp).all()


LOGITS = [(300, 40), (200, 1000), (100, 5003), (20, 40000), (600, 20000), (3, 131072)]


@pytest.mark.parametrize("scale", [0.7, 1.0, 1.5])
@pytest.mark.parametrize("rows,vocab", LOGITS)
def test_near_certain_tokens_have_no_positive_log_probability(rows, vocab, scale):
    x, tokens, _, _ = logit_inputs(rows, vocab, torch.float32, seed=vocab, std=1.0)
    x[torch.arange(rows), tokens] = 20 + 40 * torch.rand(rows, generator=torch.Generator().manual_seed(1)).cuda()
    check_logp(x, tokens, scale, min(vocab, 5), "certain")


@pytest.mark.parametrize("offset", [-2.0 ** 13, 1024.0, 2.0 ** 16])
@pytest.mark.parametrize("rows,vocab", LOGITS)
def test_an_offset_of_a_row_changes_no_log_probability(rows, vocab, offset):
    import differentiable_cholesky_amd as dc
    x, tokens, _, _ = logit_inputs(rows, vocab, torch.float32, seed=vocab)
    x = torch.round(x * 64) / 64                                     # (so that the sum is exact)
    check_logp(x + offset, tokens, 1.5, min(vocab, 8), "offset")
    a, b = (dc.chol_token_logprob(t, tokens, scale=1.5, top=min(vocab, 8)) for t in (x, x + offset))
    for k in ("logp", "entropy", "top_ids", "top_logp"):
        assert torch.equal(getattr(a, k), getattr(b, k)), k


@pytest.mark.parametrize("rows,vocab", [(5, 60), (3, 5000), (2, 40000), (600, 20000)])
def test_extreme_scales(rows, vocab):
    """Logits whose differences, or the sum of them, pass the largest number of their type, under scales that bring them
    back; and scales near the largest."""
    import differentiable_cholesky_amd as dc
    x, tokens, _, _ = logit_inputs(rows, vocab, torch.float32, seed=vocab, std=1.0)
    x = x.clamp(-3.9, 3.9)
    want = dc.chol_token_logprob(x, tokens, scale=1.0, top=4)
    for power in (-126, -120, -100, 60, 100):
        # y is the same whatever the power: at -126 the logits reach 3.9 2^126 and their differences twice that; at 100 the
        # least of them are still normal numbers
        got = dc.chol_token_logprob(x * 2.0 ** -power, tokens, scale=2.0 ** power, top=4)
        for a, b in zip(got, want):
            assert torch.equal(a, b), power
    flat = torch.zeros_like(x)
    flat[:, ::2] = -2.0 ** 120
    got = dc.chol_token_logprob(flat, tokens, scale=2.0 ** -120)
    same = dc.chol_token_logprob(flat * 2.0 ** -120, tokens)
    assert all(torch.equal(a, b) for a, b in zip(got[:3], same[:3])) and torch.isfinite(got.entropy).all()
    assert (dc.chol_token_logprob(x, tokens, scale=2.0 ** 126).logp <= 0).all()
    for scale in (2.0 ** 126.5, 3.4e38):
        with pytest.raises(dc.CholError):
            dc.chol_token_logprob(x, tokens, scale=scale)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(9, 60), (6, 3001), (5, 70000)])
def test_rows_that_take_no_gradient_have_none(rows, vocab, dtype):
    """Padding's rows hold anything: with no token, or a weight of zero, and no gradient of the entropy they are zero."""
    import differentiable_cholesky_amd as dc
    x, tokens, gl, ge = logit_inputs(rows, vocab, dtype, seed=3)
    clean = dc.chol_token_logprob(x, tokens)
    want = dc.chol_token_logprob_adjoint(x, tokens, clean.lse, adjLogp=gl, entropy=clean.entropy, adjEntropy=ge)
    only = dc.chol_token_logprob_adjoint(x, tokens, clean.lse, adjLogp=gl)
    x[0], x[1, 5], x[2, vocab - 1] = math.nan, math.inf, math.nan
    tokens[0], tokens[1] = -1, vocab
    gl[2] = 0.0
    ge[:3] = 0.0
    got = dc.chol_token_logprob(x, tokens)
    assert torch.isnan(got.lse[:3]).all()
    d = dc.chol_token_logprob_adjoint(x, tokens, got.lse, adjLogp=gl, entropy=got.entropy, adjEntropy=ge)
    assert not d[:3].any() and torch.equal(d[3:], want[3:])
    d = dc.chol_token_logprob_adjoint(x, tokens, got.lse, adjLogp=gl)
    assert not d[:3].any() and torch.equal(d[3:], only[3:])
    # one that takes a gradient has what its definition has
    gl[2] = 1.0
    assert torch.isnan(dc.chol_token_logprob_adjoint(x, tokens, got.lse, adjLogp=gl)[2]).all()
