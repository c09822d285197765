"""The recurrent language model of examples/, which runs the training-step operators together."""
import importlib.util
import math
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "recurrent_lm.py")


@pytest.fixture(scope="module")
def lm():
    spec = importlib.util.spec_from_file_location("recurrent_lm", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def logits64(p, tokens, layers, dim, eps=1e-6):
    norm = lambda x, w: x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w  # noqa: E731
    s, o = p["embed"][tokens], 0
    for i in range(layers):
        s = s + o
        z, v = (norm(s, p[f"norm{i}"]) @ p[f"in{i}"]).split(dim, dim=-1)
        a, x, rows = torch.sigmoid(-z), 0, []
        for t in range(tokens.shape[1]):
            x = a[:, t] * x + (1 - a[:, t]) * v[:, t]
            rows.append(x)
        o = torch.stack(rows, 1) @ p[f"out{i}"]
    return norm(s + o, p["norm"]) @ p["embed"].t()


def test_gradients_against_64_bits(lm):
    dim, layers, vocab = 24, 2, 11
    model = lm.RecurrentLM(vocab, dim, layers, dtype=torch.float32)
    tokens = lm.sequences(3, 40, vocab, torch.Generator().manual_seed(2))
    weight = torch.randn(3, 40, vocab, generator=torch.Generator().manual_seed(3))
    logits, kept = model.forward(tokens)
    model.backward(weight.cuda(), kept)
    p = {k: t.detach().cpu().double().requires_grad_() for k, t in model.p.items()}
    want = logits64(p, tokens.cpu(), layers, dim)
    (want * weight.double()).sum().backward()
    # fp32 throughout, sums of at most 120 rows or 48 columns through three norms and two recurrences of 40 steps: some
    # 1000 roundings of terms no larger than the largest gradient of a tensor
    assert (logits.cpu().double() - want).abs().max() <= 1000 * 2.0 ** -24 * want.abs().max()
    for k, t in p.items():
        err = (model.g[k].cpu().double() - t.grad).abs().max()
        assert err <= 1000 * 2.0 ** -24 * t.grad.abs().max(), (k, err)


@pytest.mark.parametrize("bits", [32, 8])
def test_it_learns_to_count(lm, bits):
    model = lm.RecurrentLM(vocab=32, dim=128, layers=2)
    losses = lm.train(model, 150, bits=bits)
    assert all(math.isfinite(x) for x in losses)
    # the first token of a sequence does not tell its stride: log(3) / 64 is the least
    assert losses[0] > 3 and losses[-1] < 0.5, (losses[0], losses[-1])


def test_generation_continues_what_was_read(lm):
    """Prompt in one pass and the rest token by token give the logits of one pass over all."""
    model = lm.RecurrentLM(vocab=32, dim=256, layers=2, seed=4)
    tokens = lm.sequences(5, 30, 32, torch.Generator().manual_seed(5))
    whole, _ = model.forward(tokens)
    states = model.states(5)
    model.forward(tokens[:, :20], states)
    for t in range(20, 30):
        got = model.next_logits(tokens[:, t], states)
        # bf16 activations (2^-8 a rounding, some of them) and an 8-bit head: 2^-4 of each of 256 terms at random signs
        assert (got - whole[:, t].float()).abs().max() <= 0.1 * whole[:, t].float().abs().max()
    assert lm.generate(model, tokens, 3).shape == (5, 3)
