"""chol_token_logprob and chol_token_logprob_adjoint against 64 bits, on the GPU."""
import math

import pytest

import language_util as lu
import train_util as tu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def make(rows, vocab, dtype, seed=0, std=3.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, vocab, generator=g) * std).to(dtype)
    tokens = torch.randint(0, vocab, (rows,), generator=g)
    gl, ge = torch.randn(rows, generator=g), torch.randn(rows, generator=g)
    return x.cuda(), tokens.cuda(), gl.cuda(), ge.cuda()


def check_forward(x, tokens, scale, top, got, what):
    (logp, lse, entropy, ids, top_logp), bounds = lu.logprob64(x, tokens, scale, top)
    for name, a, b, c in zip(("logp", "lse", "entropy"), got[:3], (logp, lse, entropy), bounds):
        tu.near(a, b, c + 1e-40, f"{what} {name}")
    if top:
        assert torch.equal(got.top_ids, ids), (what, got.top_ids, ids)
        tu.near(got.top_logp, top_logp, bounds[3], what + " top")


def check(x, tokens, gl, ge, scale, top, what):
    import differentiable_cholesky_amd as dc
    got = dc.chol_token_logprob(x, tokens, scale=scale, top=top)
    check_forward(x, tokens, scale, top, got, what)
    d = dc.chol_token_logprob_adjoint(x, tokens, got.lse, adjLogp=gl, entropy=got.entropy, adjEntropy=ge, scale=scale)
    ref, bound = lu.logprob_adjoint64(x, tokens, got.lse, got.entropy, gl, ge, scale)
    tu.near(d, ref, bound, what + " adjoint")


SIZES = [(1, 1), (3, 2), (2, 7), (5, 64), (4, 100), (1, 511), (7, 1024), (3, 2047), (2, 4096), (9, 4099), (3, 10007),
         (1, 16384), (2, 16385), (600, 5001), (5, 50257), (1, 131072), (2, 262145), (530, 33000)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_forward_and_adjoint(rows, vocab, dtype):
    x, tokens, gl, ge = make(rows, vocab, dtype, seed=vocab)
    check(x, tokens, gl, ge, (1.0, 0.7, 1.5)[vocab % 3], min(vocab, (0, 1, 5, 20)[vocab % 4]), "logprob")


@pytest.mark.parametrize("top", [1, 2, 8, 32])
@pytest.mark.parametrize("rows,vocab", [(3, 40), (4, 600), (3, 9000), (2, 40000), (700, 20000)])
def test_alternatives_of_equal_values(rows, vocab, top):
    """Few different values, so that most places are ties; sorted rows; a constant row."""
    import differentiable_cholesky_amd as dc
    g = torch.Generator().manual_seed(top)
    x = torch.randint(-3, 4, (rows, vocab), generator=g).float()
    x[0] = torch.arange(vocab) * 2.0 ** -10
    x[1] = 1.5
    if rows > 2:
        x[2] = torch.where(torch.rand(vocab, generator=g) < 0.5, 0.0, -0.0)
    x = x.cuda()
    tokens = torch.zeros(rows, dtype=torch.int64, device="cuda")
    check_forward(x, tokens, 1.0, top, dc.chol_token_logprob(x, tokens, top=top), "ties")
    y = x.to(torch.bfloat16)
    check_forward(y, tokens, 1.0, top, dc.chol_token_logprob(y, tokens, top=top), "ties in 16 bits")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [50, 3001, 70000])
def test_closed_columns_and_rows(vocab, dtype):
    """-inf, the type's lowest value, rows of nothing, rows without a token, a closed token."""
    import differentiable_cholesky_amd as dc
    x, tokens, gl, ge = make(8, vocab, dtype, seed=1)
    closed = torch.rand(vocab, generator=torch.Generator().manual_seed(2)) < 0.5
    closed[tokens.cpu()] = False
    x[:, closed.cuda()] = -math.inf
    x[1] = torch.where(torch.isinf(x[1]), torch.finfo(dtype).min, x[1].float()).to(dtype)
    tokens[3], tokens[4] = -1, vocab
    check(x, tokens, gl, ge, 1.0, min(8, int((~closed).sum())), "closed")
    x[5] = -math.inf
    x[6], x[6, vocab // 3] = -math.inf, 2.0
    tokens[6] = vocab // 3
    tokens[7] = int(closed.nonzero()[0])
    got = dc.chol_token_logprob(x, tokens, top=2)
    assert got.lse[5] == -math.inf and got.logp[5] == -math.inf and got.entropy[5] == 0
    assert got.top_ids[5].tolist() == [0, 1] and (got.top_logp[5] == -math.inf).all()
    assert got.logp[6] == 0 and got.entropy[6] == 0 and got.lse[6] == 2
    assert got.top_ids[6].tolist() == [vocab // 3, 0] and got.top_logp[6].tolist() == [0, -math.inf]
    assert got.logp[7] == -math.inf and torch.isfinite(got.lse[7])
    assert not got.logp[3:5].any()
    d = dc.chol_token_logprob_adjoint(x, tokens, got.lse, adjLogp=gl, entropy=got.entropy, adjEntropy=ge)
    assert not d[5].any() and torch.isfinite(d).all()
    keep = [0, 1, 2, 3, 4, 6, 7]
    ref, bound = lu.logprob_adjoint64(x[keep], tokens[keep], got.lse[keep], got.entropy[keep], gl[keep], ge[keep], 1.0)
    tu.near(d[keep], ref, bound, "closed adjoint")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(2, 40), (3, 5000), (2, 33000), (600, 33000)])
def test_one_open_column(rows, vocab, dtype):
    """All but one column at the type's lowest value, so that waves and chunks hold nothing else."""
    x, tokens, gl, ge = make(rows, vocab, dtype, seed=vocab)
    row = torch.arange(rows, device="cuda")
    column = row * 7919 % vocab
    open_ = x[row, column]
    x.fill_(torch.finfo(dtype).min)
    x[row, column] = open_
    tokens[::2] = column[::2]
    check(x, tokens, gl, ge, 1.0, 0, "one open")


@pytest.mark.parametrize("rows,vocab", [(2, 900), (2, 40000)])
def test_small_scales_of_large_logits(rows, vocab):
    x, tokens, gl, ge = make(rows, vocab, torch.float32, seed=9)
    import differentiable_cholesky_amd as dc
    x, scale = x * 2.0 ** 117, 2.0 ** -117
    got, want = dc.chol_token_logprob(x, tokens, scale=scale), dc.chol_token_logprob(x * scale, tokens)
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("vocab", [60, 5000, 40000])
def test_non_finite_rows_stay_alone(vocab):
    import differentiable_cholesky_amd as dc
    x, tokens, _, _ = make(6, vocab, torch.float32, seed=3)
    clean = dc.chol_token_logprob(x, tokens, top=3)
    x[1, vocab // 2], x[3, vocab - 1] = math.nan, math.inf
    x[4, 5] = -math.nan
    got = dc.chol_token_logprob(x, tokens, top=3)
    for i in (1, 3, 4):
        assert all(torch.isnan(t[i]) for t in got[:3])
    assert got.top_ids[1, 0] == vocab // 2 and got.top_ids[3, 0] == vocab - 1 and got.top_ids[4, 0] == 5
    for i in (0, 2, 5):
        assert all(torch.equal(a[i], b[i]) for a, b in zip(got, clean))


def test_strides_and_results_in_place():
    import differentiable_cholesky_amd as dc
    x, tokens, gl, ge = make(20, 3001, torch.bfloat16, seed=4)
    want = dc.chol_token_logprob(x, tokens, top=4)
    d = dc.chol_token_logprob_adjoint(x, tokens, want.lse, adjLogp=gl)
    wide = torch.full((20, 3010), 5.0, dtype=x.dtype, device="cuda")
    view = wide[:, 3:3004]
    view.copy_(x)
    got = dc.chol_token_logprob(view, tokens, top=4)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dc.chol_token_logprob_adjoint(view, tokens, want.lse, adjLogp=gl, adjLogits=view)
    assert torch.equal(view, d) and (wide[:, :3] == 5).all() and (wide[:, 3004:] == 5).all()
    bare = dc.chol_token_logprob(x, tokens, entropy=False)
    assert bare.entropy is None and bare.top_ids is None and torch.equal(bare.logp, want.logp)
    only = dc.chol_token_logprob_adjoint(x, tokens, want.lse, entropy=want.entropy, adjEntropy=ge)
    ref, bound = lu.logprob_adjoint64(x, tokens, want.lse, want.entropy, None, ge, 1.0)
    tu.near(only, ref, bound, "entropy alone")


def test_no_rows():
    import differentiable_cholesky_amd as dc
    x = torch.empty(0, 100, device="cuda")
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    got = dc.chol_token_logprob(x, t, top=3)
    assert got.logp.shape == (0,) and got.top_ids.shape == (0, 3)
    assert dc.chol_token_logprob_adjoint(x, t, got.lse).shape == x.shape


@pytest.mark.parametrize("rows,vocab", [(4, 900), (4, 60000)])
def test_captured_and_replayed(rows, vocab):
    import differentiable_cholesky_amd as dc
    x, tokens, gl, ge = make(rows, vocab, torch.bfloat16, seed=5)
    dc.chol_token_logprob(x, tokens, top=4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dc.chol_token_logprob(x, tokens, top=4)
        d = dc.chol_token_logprob_adjoint(x, tokens, got.lse, adjLogp=gl, entropy=got.entropy, adjEntropy=ge)
    for _ in range(4):
        graph.replay()
        want = dc.chol_token_logprob(x, tokens, top=4)
        e = dc.chol_token_logprob_adjoint(x, tokens, want.lse, adjLogp=gl, entropy=want.entropy, adjEntropy=ge)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(d, e)
        x.mul_(-0.75)


def test_other_streams_and_workspaces():
    import differentiable_cholesky_amd as dc
    x, tokens, gl, _ = make(3, 60000, torch.bfloat16, seed=6)
    want = dc.chol_token_logprob(x, tokens, top=4)
    need = dc.chol_token_logprob_workspace_size(dc.CHOL_BF16, 3, 60000, 4)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = dc.chol_token_logprob(x, tokens, top=4, workspace=ws, stream=side)
    d = dc.chol_token_logprob_adjoint(x, tokens, got.lse, adjLogp=gl, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(d, dc.chol_token_logprob_adjoint(x, tokens, want.lse, adjLogp=gl))


def test_gradients_against_differences():
    import differentiable_cholesky_amd as dc
    x, tokens, gl, ge = make(4, 37, torch.float32, seed=7)
    got = dc.chol_token_logprob(x, tokens, scale=0.8)
    d = dc.chol_token_logprob_adjoint(x, tokens, got.lse, adjLogp=gl, entropy=got.entropy, adjEntropy=ge, scale=0.8).double()

    def f(x):
        (logp, _, entropy, _, _), _ = lu.logprob64(x, tokens, 0.8, 0)
        return (logp * gl.double()).sum() + (entropy * ge.double()).sum()

    way = torch.randn(x.shape, generator=torch.Generator().manual_seed(8)).double().cuda()
    step = 1e-5
    slope = (f(x.double() + step * way) - f(x.double() - step * way)) / (2 * step)
    size = (d * way).abs().sum()
    # some 10 roundings of fp32 of terms whose logarithms reach 20, and a difference of order step^2
    assert abs((d * way).sum() - slope) <= 200 * tu.U * size + 1e-8 * size
