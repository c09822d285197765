"""More elements than 32 bits count, and rows as far apart as they may be: the convolution, the scan and the token log
probabilities.  The end of a large call has the bits of a smaller call on it (the same plan, by the sizes)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.slow]


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def normal(*shape, dtype=torch.bfloat16, seed=0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(seed))


def test_convolution_of_more_than_32_bits():
    import differentiable_cholesky_amd as dc
    batch, length, dim, tail = 3, 175_000, 4096 + 8, 333
    assert batch * length * dim > 1 << 31
    x, adj, w, bias = normal(batch, length, dim), normal(batch, length, dim, seed=1), normal(dim, 4), normal(dim, seed=2)
    y, last = dc.chol_causal_conv(x, w, bias=bias)
    end = x[:, -tail:].contiguous()
    kept = x[:, -tail - 3:-tail].contiguous()
    y2, last2 = dc.chol_causal_conv(end, w, bias=bias, state=kept)
    assert torch.equal(y[:, -tail:], y2) and torch.equal(last, last2)
    dx, dw, _, _ = dc.chol_causal_conv_adjoint(x, w, adj, bias=bias, adjX=y)
    dx2, _, _, _ = dc.chol_causal_conv_adjoint(end, w, adj[:, -tail:].contiguous(), bias=bias, state=kept)
    assert torch.equal(dx[:, -tail:], dx2) and torch.isfinite(dw).all()


def test_logits_of_more_than_32_bits():
    import differentiable_cholesky_amd as dc
    rows, vocab, tail = 16_500, 131_072, 64
    assert rows * vocab > 1 << 31
    x = normal(rows, vocab)
    tokens = torch.randint(0, vocab, (rows,), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    gl = normal(rows, dtype=torch.float32, seed=2)
    got = dc.chol_token_logprob(x, tokens, top=3)
    end, t = x[-tail:].clone(), tokens[-tail:].clone()
    want = dc.chol_token_logprob(end, t, top=3)
    assert all(torch.equal(a[-tail:], b) for a, b in zip(got, want))
    d = dc.chol_token_logprob_adjoint(x, tokens, got.lse, adjLogp=gl, entropy=got.entropy, adjEntropy=gl, adjLogits=x)
    e = dc.chol_token_logprob_adjoint(end, t, want.lse, adjLogp=gl[-tail:].clone(), entropy=want.entropy,
                                      adjEntropy=gl[-tail:].clone())
    assert torch.equal(d[-tail:], e)


def scan_inputs(batch, length, dim, states, dtype=torch.bfloat16):
    s = {k: normal(batch, length, dim, dtype=dtype, seed=i) for i, k in enumerate(("u", "delta", "z", "adj"))}
    s["delta"] -= 3
    s.update({k: normal(batch, length, states, dtype=dtype, seed=5 + i) for i, k in enumerate("BC")})
    s["A"] = -torch.exp(normal(dim, states, dtype=torch.float32, seed=8))
    s["D"] = normal(dim, dtype=torch.float32, seed=9)
    return s


def scan_both(s, **more):
    import differentiable_cholesky_amd as dc
    y, last, starts = dc.chol_selective_scan(s["u"], s["delta"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], save=True,
                                             y=more.pop("y", None))
    return y, last, starts, dc.chol_selective_scan_adjoint(s["u"], s["delta"], s["A"], s["B"], s["C"], starts, s["adj"],
                                                           D=s["D"], z=s["z"], **more)


def test_scan_of_more_than_32_bits():
    batch, length, dim = 3, 44_000, 16_384
    assert batch * length * dim > 1 << 31
    s = scan_inputs(batch, length, dim, 16)
    y, last, starts, grads = scan_both(s)
    part = {k: x[1:] if k not in "AD" else x for k, x in s.items()}
    y2, last2, starts2, grads2 = scan_both(part)
    assert torch.equal(y[1:], y2) and torch.equal(last[1:], last2) and torch.equal(starts[1:], starts2)
    for k in (0, 1, 3, 4, 6, 8):      # gradients of u, delta, B, C, z and the first state; the others are sums over the batch
        assert torch.equal(grads[k][1:], grads2[k]), k


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("states", [16, 20, 40])
def test_rows_as_far_apart_as_they_may_be(states, dtype):
    length, dim, ld = 70, 40, 1 << 25
    s = scan_inputs(1, length, dim, states, dtype)
    y, last, starts, grads = scan_both(s)
    wide = torch.empty(1, length, ld, dtype=dtype, device="cuda")
    at, t = 0, dict(s)

    def columns(n, like=None):
        nonlocal at
        x = wide[..., at:at + n]
        at += n + 3
        return x if like is None else x.copy_(like)

    for k in ("u", "delta", "z", "adj", "B", "C"):
        t[k] = columns(s[k].shape[-1], s[k])
    out = {k: columns(n) for k, n in (("y", dim), ("adjU", dim), ("adjDelta", dim), ("adjZ", dim), ("adjB", states), ("adjC", states))}
    y2, last2, starts2, grads2 = scan_both(t, **out)
    assert torch.equal(y, y2) and torch.equal(last, last2) and torch.equal(starts, starts2)
    for a, b in zip(grads, grads2):
        assert (a is None and b is None) or torch.equal(a, b)
