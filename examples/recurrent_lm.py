"""A small recurrent language model on the training-step operators: training with
hand-written gradients, then generation token by token from kept states.

Every block is  s += o;  y = norm(s);  (z, v) = y W_in;  h = recurrence(a, (1 - a) v)
with the gate a = sigmoid(-z), stored as its logarithm;  o = h W_out.  The residual's
addition is part of the norm, the gates and inputs are column slices of one product,
and one call steps every weight.

    python examples/recurrent_lm.py [--steps 200] [--bits 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import differentiable_cholesky_amd as dc  # noqa: E402

TILE = 256


class RecurrentLM:
    def __init__(self, vocab, dim, layers, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.dim, self.layers, self.dtype = dim, layers, dtype
        rand = lambda *shape: torch.randn(shape, generator=g) / shape[0] ** 0.5  # noqa: E731
        full = {"embed": torch.randn(vocab, dim, generator=g) * dim ** -0.5, "norm": torch.ones(dim)}
        for i in range(layers):
            full[f"norm{i}"] = torch.ones(dim)
            full[f"in{i}"], full[f"out{i}"] = rand(dim, 2 * dim), rand(dim, dim)
        self.master = {k: t.to(device) for k, t in full.items()}
        self.p = {k: t.to(dtype) for k, t in self.master.items()}
        self.g = {k: torch.zeros_like(t) for k, t in self.p.items()}

    def _mix(self, i, u):
        """Gate logarithms and inputs of the recurrence from the product's column halves."""
        z, v = u.split(self.dim, dim=-1)
        log_a = -torch.nn.functional.softplus(z.float())
        return log_a.to(self.dtype), (-torch.expm1(log_a) * v.float()).to(self.dtype)

    def forward(self, tokens, states=None):
        """Logits of [batch, len] tokens and what the backward pass needs.  ``states`` (one fp32
        [batch, dim] tensor a layer) are carried on in place."""
        batch, length = tokens.shape
        p, saved = self.p, []
        s, o = torch.nn.functional.embedding(tokens.reshape(-1), p["embed"]), None
        for i in range(self.layers):
            y, s = dc.chol_rmsnorm(s if o is None else o, p[f"norm{i}"], residual=None if o is None else s)
            u = (y @ p[f"in{i}"]).view(batch, length, -1)
            a, b = self._mix(i, u)
            keep = None if states is None else states[i]
            h, _ = dc.chol_recurrence(a, b, h0=keep, hlast=keep, gate="log")
            h = h.view(-1, self.dim)
            o = h @ p[f"out{i}"]
            saved.append((s, y, u, a, h))
        y, s = dc.chol_rmsnorm(o, p["norm"], residual=s)
        return (y @ p["embed"].t()).view(batch, length, -1), (tokens, saved, s, y)

    def backward(self, adj_logits, kept):
        """Gradients of every weight into self.g."""
        tokens, saved, s, y = kept
        p, g = self.p, self.g
        shape = tokens.shape
        adj = adj_logits.reshape(-1, adj_logits.shape[-1]).to(self.dtype)
        embed = (adj.t() @ y).float()
        ds, dw = dc.chol_rmsnorm_adjoint(s, p["norm"], adj @ p["embed"])
        g["norm"].copy_(dw)
        for i in reversed(range(self.layers)):
            s, y, u, a, h = saved[i]
            torch.mm(h.t(), ds, out=g[f"out{i}"])
            adj_h = (ds @ p[f"out{i}"].t()).view(*shape, self.dim)
            da, db, _ = dc.chol_recurrence_adjoint(a, h.view(*shape, self.dim), adj_h, gate="log")
            z, v = (t.float() for t in u.split(self.dim, dim=-1))
            gate = torch.sigmoid(-z)
            # log a = -softplus(z), whose slope is gate - 1; b = (1 - a) v
            dz = (da.float() - db.float() * v * gate) * (gate - 1)
            du = torch.cat([dz, db.float() * (1 - gate)], -1).to(self.dtype).view(-1, 2 * self.dim)
            torch.mm(y.t(), du, out=g[f"in{i}"])
            ds, dw = dc.chol_rmsnorm_adjoint(s, p[f"norm{i}"], du @ p[f"in{i}"].t(), adjH=ds)
            g[f"norm{i}"].copy_(dw)
        g["embed"].copy_(embed.index_add_(0, tokens.reshape(-1), ds.float()))

    def states(self, batch):
        return [torch.zeros(batch, self.dim, device=self.p["embed"].device) for _ in range(self.layers)]

    def next_logits(self, token, states):
        """One step of generation: the head reads 8-bit rows with a scale for every 128 columns."""
        p = self.p
        s, o = torch.nn.functional.embedding(token, p["embed"]), None
        for i in range(self.layers):
            y, s = dc.chol_rmsnorm(s if o is None else o, p[f"norm{i}"], residual=None if o is None else s)
            a, b = self._mix(i, (y @ p[f"in{i}"])[:, None])
            h, _ = dc.chol_recurrence(a, b, h0=states[i], hlast=states[i], gate="log")
            o = h[:, 0] @ p[f"out{i}"]
        q, scale, _ = dc.chol_rmsnorm_quant(o, p["norm"], residual=s, group=128)
        wide = scale.repeat_interleave(128, 1)[:, :self.dim]
        return (q.float() * wide) @ p["embed"].float().t()


class Optimizer:
    """AdamW with fp32 master weights and states in 32 or 8 bits."""

    def __init__(self, model, bits, lr):
        p, g, master = (list(d.values()) for d in (model.p, model.g, model.master))
        dev = p[0].device
        self.step, self.lr, self.grads = 0, lr, g
        if bits == 8:
            zero = lambda t: torch.zeros(t.shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)  # noqa: E731
            ones = lambda: [torch.ones(-(-t.numel() // TILE), device=dev) for t in p]  # noqa: E731
            scales = {"m_scale": ones(), "v_scale": ones()}
        else:
            zero, scales = (lambda t: torch.zeros(t.shape, device=dev)), {}
        self.list = dc.chol_adamw_list(p, g, [zero(t) for t in p], [zero(t) for t in p], master=master, **scales)

    def update(self):
        self.step += 1
        size = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(t.float()) for t in self.grads]))
        clip = (1.0 / size).clamp(max=1.0)
        dc.chol_adamw(self.list, step=self.step, lr=self.lr, weight_decay=0.01, grad_scale=clip, seed=self.step)


def sequences(batch, length, vocab, gen, device="cuda"):
    """Counting sequences: each starts and strides at random, modulo the vocabulary."""
    start = torch.randint(0, vocab, (batch, 1), generator=gen)
    stride = torch.randint(1, 4, (batch, 1), generator=gen)
    return ((start + stride * torch.arange(length)) % vocab).to(device)


def train(model, steps, bits=8, batch=16, length=64, vocab=32, lr=3e-3, seed=0):
    """Returns the loss of every step."""
    opt, gen, losses = Optimizer(model, bits, lr), torch.Generator().manual_seed(seed), []
    for _ in range(steps):
        t = sequences(batch, length + 1, vocab, gen)
        logits, kept = model.forward(t[:, :-1])
        log_p = torch.log_softmax(logits.float(), -1)
        want = t[:, 1:, None]
        losses.append(-log_p.gather(2, want).mean())
        adj = log_p.exp()
        adj.scatter_add_(2, want, torch.full_like(adj[..., :1], -1.0))
        model.backward(adj / want.numel(), kept)
        opt.update()
    return torch.stack(losses).tolist()


def generate(model, prompt, count):
    """Greedy continuation of [batch, len] prompts."""
    states = model.states(prompt.shape[0])
    logits, _ = model.forward(prompt, states)
    token, out = logits[:, -1].argmax(-1), []
    for _ in range(count):
        out.append(token)
        token = model.next_logits(token, states).argmax(-1)
    return torch.stack(out, 1)


if __name__ == "__main__":
    args = argparse.ArgumentParser()
    args.add_argument("--steps", type=int, default=200)
    args.add_argument("--bits", type=int, choices=(8, 32), default=8)
    args = args.parse_args()
    lm = RecurrentLM(vocab=32, dim=256, layers=2)
    losses = train(lm, args.steps, args.bits)
    for k in range(0, args.steps, max(1, args.steps // 10)):
        print(f"step {k:4d}  loss {losses[k]:.4f}")
    print(f"step {args.steps - 1:4d}  loss {losses[-1]:.4f}")
    prompt = sequences(4, 12, 32, torch.Generator().manual_seed(1))
    more = generate(lm, prompt, 12)
    for a, b in zip(prompt.tolist(), more.tolist()):
        print(*a, "->", *b)
