"""Padded batches in the selective language model of examples/: tokens below zero are no inputs."""
import importlib.util

import pytest

import train_util as tu
from test_selective_lm import PATH, logits64

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lm():
    pytest.importorskip("differentiable_cholesky_amd")
    spec = importlib.util.spec_from_file_location("selective_lm", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_no_padding_reaches_the_embedding(lm):
    """On the CPU: the tokens that a loss hands to the model's forward pass."""
    class Stop(Exception):
        pass

    model, seen = lm.SelectiveLM(7, 16, 1, device="cpu"), []

    def forward(tokens, kept=None):
        seen.append(tokens)
        raise Stop

    model.forward = forward
    tokens = torch.tensor([[1, 2, 3, 4, 5], [6, 5, -1, -1, -1], [0, -1, -1, -1, -1]])
    before = tokens.clone()
    with pytest.raises(Stop):
        model.loss(tokens)
    assert seen[0].tolist() == [[1, 2, 3, 4], [6, 5, 0, 0], [0, 0, 0, 0]]
    assert torch.equal(tokens, before)


@pytest.mark.gpu
@pytest.mark.parametrize("bonus", [0.0, 0.3])
def test_loss_and_gradients_of_a_padded_batch(lm, bonus):
    vocab, layers, states, length = 11, 2, 16, 40
    model = lm.SelectiveLM(vocab, 24, layers, states=states, rank=3, dtype=torch.float32)
    tokens = lm.sequences(3, length + 1, vocab, torch.Generator().manual_seed(2))
    tokens[1, -5:], tokens[2, 1:] = -1, -1
    got = model.loss(tokens, bonus)
    p = {k: t.detach().cpu().double().requires_grad_() for k, t in model.p.items()}
    host = tokens.cpu()
    lp = torch.log_softmax(logits64(p, host[:, :-1].clamp(min=0), layers, model.inner, model.rank, states, lm.WIDTH), -1)
    want = host[:, 1:]
    given = lp.gather(2, want.clamp(min=0)[..., None])[..., 0] * (want >= 0)
    loss = -(given.mean() + bonus * -(lp.exp() * lp).sum(-1).mean())
    loss.backward()
    # fp32 throughout: some 1000 roundings of terms no larger than the largest of a tensor, twice that for gradients
    assert abs(got.item() - loss.item()) <= 1000 * tu.U * abs(loss.item())
    for k, t in p.items():
        err = (model.g[k].cpu().double() - t.grad).abs().max()
        assert err <= 2000 * tu.U * t.grad.abs().max(), (k, err, t.grad.abs().max())
