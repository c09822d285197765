"""A small selective state space language model on the library's operators: training with
hand-written gradients, then generation token by token from kept rows and states.

Every block is  s += o;  y = norm(s);  (x, z) = y W_in;  u = silu(conv(x));
(low, B, C) = u W_x;  delta = low W_dt;  o = scan(u, delta, A, B, C, gated by z) W_out,
with A = -exp(log_A).  The loss is the tokens' log probability, with a bonus for entropy
if one is asked for; generation samples among the most likely tokens.

    python examples/selective_lm.py [--steps 200] [--bits 8]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import differentiable_cholesky_amd as dc  # noqa: E402
from examples.recurrent_lm import Optimizer, sequences  # noqa: E402

WIDTH = 4   # of the convolution


class SelectiveLM:
    def __init__(self, vocab, dim, layers, inner=None, states=16, rank=None, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.dim, self.layers, self.dtype, self.states = dim, layers, dtype, states
        self.inner, self.rank = inner or 2 * dim, rank or max(1, dim // 16)
        rand = lambda *shape: torch.randn(shape, generator=g) / shape[0] ** 0.5  # noqa: E731
        full = {"embed": torch.randn(vocab, dim, generator=g) * dim ** -0.5, "norm": torch.ones(dim)}
        for i in range(layers):
            full[f"norm{i}"] = torch.ones(dim)
            full[f"in{i}"], full[f"out{i}"] = rand(dim, 2 * self.inner), rand(self.inner, dim)
            full[f"conv{i}"] = torch.randn(self.inner, WIDTH, generator=g) * WIDTH ** -0.5
            full[f"conv_bias{i}"] = torch.zeros(self.inner)
            full[f"x{i}"], full[f"dt{i}"] = rand(self.inner, self.rank + 2 * states), rand(self.rank, self.inner)
            # steps between 0.001 and 0.1 to begin with
            rate = torch.exp(torch.rand(self.inner, generator=g) * math.log(100) + math.log(1e-3))
            full[f"dt_bias{i}"] = torch.log(torch.expm1(rate))
            full[f"log_A{i}"] = torch.log(torch.arange(1.0, states + 1)).repeat(self.inner, 1)
            full[f"D{i}"] = torch.ones(self.inner)
        self.master = {k: t.to(device) for k, t in full.items()}
        self.p = {k: t.to(dtype) for k, t in self.master.items()}
        self.g = {k: torch.zeros_like(t) for k, t in self.p.items()}

    def _mix(self, i):
        """What the scan takes in 32 bits."""
        p = self.p
        return -torch.exp(p[f"log_A{i}"].float()), p[f"D{i}"].float(), p[f"dt_bias{i}"].float()

    def kept(self, batch):
        """Rows and states of every layer, for sequences that have not begun."""
        dev = self.p["embed"].device
        return [(torch.zeros(batch, WIDTH - 1, self.inner, dtype=self.dtype, device=dev),
                 torch.zeros(batch, self.inner, self.states, device=dev)) for _ in range(self.layers)]

    def forward(self, tokens, kept=None):
        """Logits of [batch, len] tokens, [batch * len, vocab], and what the backward pass needs.  ``kept``
        (from kept()) is carried on in place."""
        batch, length = tokens.shape
        p, saved, n = self.p, [], self.states
        s, o = torch.nn.functional.embedding(tokens.reshape(-1), p["embed"]), None
        for i in range(self.layers):
            y, s = dc.chol_rmsnorm(s if o is None else o, p[f"norm{i}"], residual=None if o is None else s)
            x, z = (y @ p[f"in{i}"]).view(batch, length, -1).split(self.inner, dim=-1)
            rows, h = (None, None) if kept is None else kept[i]
            u, _ = dc.chol_causal_conv(x, p[f"conv{i}"], bias=p[f"conv_bias{i}"], state=rows, last=rows)
            low, B, C = (u @ p[f"x{i}"]).split([self.rank, n, n], dim=-1)
            delta = low @ p[f"dt{i}"]
            A, D, bias = self._mix(i)
            v, _, starts = dc.chol_selective_scan(u, delta, A, B, C, D=D, z=z, bias=bias, h0=h, hlast=h, save=kept is None)
            v = v.view(-1, self.inner)
            o = v @ p[f"out{i}"]
            saved.append((s, y, x, z, u, low, B, C, delta, A, D, bias, starts, v))
        y, s = dc.chol_rmsnorm(o, p["norm"], residual=s)
        return y @ p["embed"].t(), (tokens, saved, s, y)

    def backward(self, adj, kept):
        """Gradients of every weight into self.g from that of the logits."""
        tokens, saved, s, y = kept
        p, g, n = self.p, self.g, self.states
        embed = (adj.t() @ y).float()
        ds, dw = dc.chol_rmsnorm_adjoint(s, p["norm"], adj @ p["embed"])
        g["norm"].copy_(dw)
        for i in reversed(range(self.layers)):
            s, y, x, z, u, low, B, C, delta, A, D, bias, starts, v = saved[i]
            torch.mm(v.t(), ds, out=g[f"out{i}"])
            dv = (ds @ p[f"out{i}"].t()).view_as(u)
            # the gradients of x and z, and of the three parts of u W_x, in one buffer each
            joint, mixed = torch.empty(*u.shape[:2], 2 * self.inner, dtype=u.dtype, device=u.device), torch.empty(
                *u.shape[:2], self.rank + 2 * n, dtype=u.dtype, device=u.device)
            dx, dz = joint.split(self.inner, dim=-1)
            dlow, dB, dC = mixed.split([self.rank, n, n], dim=-1)
            du, ddelta, dA, _, _, dD, _, dbias, _ = dc.chol_selective_scan_adjoint(
                u, delta, A, B, C, starts, dv, D=D, z=z, bias=bias, adjB=dB, adjC=dC, adjZ=dz)
            g[f"log_A{i}"].copy_(dA * A), g[f"D{i}"].copy_(dD), g[f"dt_bias{i}"].copy_(dbias)
            ddelta = ddelta.view(-1, self.inner)
            torch.mm(low.reshape(-1, self.rank).t(), ddelta, out=g[f"dt{i}"])
            dlow.copy_((ddelta @ p[f"dt{i}"].t()).view_as(dlow))
            mixed = mixed.view(-1, mixed.shape[-1])
            torch.mm(u.view(-1, self.inner).t(), mixed, out=g[f"x{i}"])
            du += (mixed @ p[f"x{i}"].t()).view_as(du)
            _, dw, db, _ = dc.chol_causal_conv_adjoint(x, p[f"conv{i}"], du, bias=p[f"conv_bias{i}"], adjX=dx)
            g[f"conv{i}"].copy_(dw), g[f"conv_bias{i}"].copy_(db)
            joint = joint.view(-1, 2 * self.inner)
            torch.mm(y.t(), joint, out=g[f"in{i}"])
            ds, dw = dc.chol_rmsnorm_adjoint(s, p[f"norm{i}"], joint @ p[f"in{i}"].t(), adjH=ds)
            g[f"norm{i}"].copy_(dw)
        g["embed"].copy_(embed.index_add_(0, tokens.reshape(-1), ds.float()))

    def loss(self, tokens, bonus=0.0):
        """Mean over all places of the negative log probability of [batch, len + 1] tokens' next ones (below
        zero, padding: none, which counts as 0), less ``bonus`` times the mean entropy; gradients into self.g."""
        logits, kept = self.forward(tokens[:, :-1].clamp(min=0))     # (padding is read as token 0)
        want = tokens[:, 1:].reshape(-1)
        r = dc.chol_token_logprob(logits, want)
        weight = torch.full_like(r.logp, -1.0 / len(want))
        # the logits are not needed again: their gradient takes their place
        dc.chol_token_logprob_adjoint(logits, want, r.lse, adjLogp=weight, entropy=r.entropy,
                                      adjEntropy=bonus * weight if bonus else None, scale=1.0, adjLogits=logits)
        self.backward(logits, kept)
        return -(r.logp.mean() + bonus * r.entropy.mean())


def train(model, steps, bits=8, batch=16, length=64, vocab=32, lr=3e-3, seed=0, bonus=0.0):
    """Returns the loss of every step."""
    opt, gen, losses = Optimizer(model, bits, lr), torch.Generator().manual_seed(seed), []
    for _ in range(steps):
        losses.append(model.loss(sequences(batch, length + 1, vocab, gen), bonus))
        opt.update()
    return torch.stack(losses).tolist()


def generate(model, prompt, count, top=4, temperature=0.7, uniform=None):
    """Continuation of [batch, len] prompts, each token drawn from the `top` most likely (by `uniform`, [count,
    batch] numbers in [0, 1); None: the most likely one).  Returns the tokens and their log probabilities."""
    kept = model.kept(prompt.shape[0])
    logits = model.forward(prompt, kept)[0].view(*prompt.shape, -1)[:, -1]
    tokens, logp = [], []
    for k in range(count):
        none = torch.full((prompt.shape[0],), -1, dtype=torch.int64, device=prompt.device)
        r = dc.chol_token_logprob(logits, none, scale=1.0 / temperature, top=top, entropy=False)
        chance = torch.softmax(r.top_logp, 1).cumsum(1)
        place = torch.zeros_like(none) if uniform is None else (uniform[k, :, None] >= chance[:, :-1]).sum(1)
        tokens.append(r.top_ids.gather(1, place[:, None])[:, 0])
        logp.append(r.top_logp.gather(1, place[:, None])[:, 0])
        logits = model.forward(tokens[-1][:, None], kept)[0]
    return torch.stack(tokens, 1), torch.stack(logp, 1)


if __name__ == "__main__":
    args = argparse.ArgumentParser()
    args.add_argument("--steps", type=int, default=200)
    args.add_argument("--bits", type=int, choices=(8, 32), default=8)
    args = args.parse_args()
    lm = SelectiveLM(vocab=32, dim=128, layers=2)
    losses = train(lm, args.steps, args.bits)
    for k in range(0, args.steps, max(1, args.steps // 10)):
        print(f"step {k:4d}  loss {losses[k]:.4f}")
    print(f"step {args.steps - 1:4d}  loss {losses[-1]:.4f}")
    prompt = sequences(4, 12, 32, torch.Generator().manual_seed(1))
    more, logp = generate(lm, prompt, 12)
    for a, b, c in zip(prompt.tolist(), more.tolist(), logp.tolist()):
        print(*a, "->", *b, " log probability %.3f" % sum(c))
