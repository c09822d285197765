"""The selective state space language model of examples/, which runs the convolution, the scan, the norm, the token
log probabilities and AdamW together."""
import importlib.util
import math
import os

import pytest

import train_util as tu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "selective_lm.py")


@pytest.fixture(scope="module")
def lm():
    spec = importlib.util.spec_from_file_location("selective_lm", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def logits64(p, tokens, layers, inner, rank, n, width, eps=1e-6):
    norm = lambda x, w: x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w  # noqa: E731
    silu = torch.nn.functional.silu
    batch, length = tokens.shape
    s, o = p["embed"][tokens], 0
    for i in range(layers):
        s = s + o
        x, z = (norm(s, p[f"norm{i}"]) @ p[f"in{i}"]).split(inner, dim=-1)
        past = torch.cat([torch.zeros(batch, width - 1, inner, dtype=torch.float64), x], 1)
        u = silu(sum(past[:, k:k + length] * p[f"conv{i}"][:, k] for k in range(width)) + p[f"conv_bias{i}"])
        low, B, C = (u @ p[f"x{i}"]).split([rank, n, n], dim=-1)
        dt = torch.nn.functional.softplus(low @ p[f"dt{i}"] + p[f"dt_bias{i}"])
        A, h, rows = -torch.exp(p[f"log_A{i}"]), 0, []
        for t in range(length):
            h = torch.exp(dt[:, t, :, None] * A) * h + (dt * u)[:, t, :, None] * B[:, t, None]
            rows.append((h * C[:, t, None]).sum(-1) + p[f"D{i}"] * u[:, t])
        o = (torch.stack(rows, 1) * silu(z)) @ p[f"out{i}"]
    return norm(s + o, p["norm"]) @ p["embed"].t()


@pytest.mark.parametrize("states,length", [(16, 40), (5, 70)])
def test_loss_and_gradients_against_64_bits(lm, states, length):
    vocab, layers, bonus = 11, 2, 0.3
    model = lm.SelectiveLM(vocab, 24, layers, states=states, rank=3, dtype=torch.float32)
    tokens = lm.sequences(3, length + 1, vocab, torch.Generator().manual_seed(2))
    tokens[1, -5:] = -1                                           # padding: no token to predict
    inputs = tokens.clamp(min=0)
    both = torch.cat([inputs[:, :1], tokens[:, 1:]], 1)
    logits, _ = model.forward(inputs[:, :-1])
    p = {k: t.detach().cpu().double().requires_grad_() for k, t in model.p.items()}
    want = logits64(p, inputs[:, :-1].cpu(), layers, model.inner, model.rank, states, lm.WIDTH)
    # fp32 throughout: as in the recurrent model some 1000 roundings of terms no larger than the largest of a tensor
    assert (logits.cpu().double().view_as(want) - want).abs().max() <= 1000 * tu.U * want.abs().max()
    lp = torch.log_softmax(want, -1)
    wanted = both[:, 1:].cpu()
    given = lp.gather(2, wanted.clamp(min=0)[..., None])[..., 0] * (wanted >= 0)
    loss = -(given.mean() + bonus * -(lp.exp() * lp).sum(-1).mean())
    loss.backward()

    # (the padding's inputs are token 0, its targets none)
    logits, kept = model.forward(inputs[:, :-1])
    r = lm.dc.chol_token_logprob(logits, both[:, 1:].reshape(-1))
    weight = torch.full_like(r.logp, -1.0 / len(r.logp))
    got = -(r.logp.mean() + bonus * r.entropy.mean())
    assert abs(got.item() - loss.item()) <= 1000 * tu.U * abs(loss.item())
    d = lm.dc.chol_token_logprob_adjoint(logits, both[:, 1:].reshape(-1), r.lse, adjLogp=weight, entropy=r.entropy,
                                         adjEntropy=bonus * weight)
    model.backward(d, kept)
    for k, t in p.items():
        err = (model.g[k].cpu().double() - t.grad).abs().max()
        assert err <= 2000 * tu.U * t.grad.abs().max(), (k, err, t.grad.abs().max())


@pytest.mark.parametrize("bits", [32, 8])
def test_training_runs(lm, bits):
    model = lm.SelectiveLM(vocab=32, dim=64, layers=2)
    before = {k: t.clone() for k, t in model.master.items()}
    losses = lm.train(model, 5, bits=bits, bonus=0.01)
    assert all(math.isfinite(x) for x in losses)
    assert all(torch.isfinite(t).all() for t in model.master.values())
    assert all((model.master[k] != t).any() for k, t in before.items())


def test_generation_continues_what_was_read(lm):
    """A prompt in one pass, the next piece in another and the rest token by token give the logits of one pass over all."""
    model = lm.SelectiveLM(vocab=32, dim=64, layers=2, seed=4)
    tokens = lm.sequences(5, 90, 32, torch.Generator().manual_seed(5))
    whole = model.forward(tokens)[0].view(5, 90, -1).float()
    kept, rows = model.kept(5), []
    for part in (tokens[:, :70], tokens[:, 70:80], *tokens[:, 80:].split(1, dim=1)):
        rows.append(model.forward(part, kept)[0].view(5, part.shape[1], -1).float())
    # bf16 activations: 2^-8 a rounding, some tens of them through two blocks
    assert (torch.cat(rows, 1) - whole).abs().max() <= 0.1 * whole.abs().max()


def test_a_captured_step_of_generation(lm):
    """The states and logits of replayed steps are those of eager ones."""
    model = lm.SelectiveLM(vocab=32, dim=64, layers=2, seed=6)
    prompt = lm.sequences(3, 20, 32, torch.Generator().manual_seed(7))
    a, b = model.kept(3), model.kept(3)
    model.forward(prompt, a), model.forward(prompt, b)
    token = torch.zeros(3, 1, dtype=torch.int64, device="cuda")
    warm = model.kept(3)
    for _ in range(2):
        model.forward(token, warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits, _ = model.forward(token, a)
        r = lm.dc.chol_token_logprob(logits, token[:, 0], top=4)
    for k in range(6):
        token.fill_(k)
        graph.replay()
        want, _ = model.forward(token, b)
        w = lm.dc.chol_token_logprob(want, token[:, 0], top=4)
        torch.cuda.synchronize()
        assert torch.equal(logits, want) and all(torch.equal(x, y) for x, y in zip(r, w)), k
        for x, y in zip(a, b):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_sampling_draws_among_the_most_likely(lm):
    model = lm.SelectiveLM(vocab=32, dim=64, layers=1, seed=8)
    prompt = lm.sequences(4, 10, 32, torch.Generator().manual_seed(9))
    first, logp = lm.generate(model, prompt, 3)
    again, _ = lm.generate(model, prompt, 3, uniform=torch.zeros(3, 4, device="cuda"))
    assert torch.equal(first, again) and first.shape == (4, 3) and (logp <= 0).all()
    last, low = lm.generate(model, prompt, 1, uniform=torch.full((1, 4), 0.999999, device="cuda"))
    logits = model.forward(prompt)[0].view(4, 10, -1)[:, -1].float()
    fourth = logits.sort(1, descending=True).values[:, 3]
    assert torch.equal(logits.gather(1, last)[:, 0], fourth)
