"""The measured cases of the operators of a selective state space language model:
the short causal convolution and the selective scan, with their adjoints and
their form for single tokens, and the log probabilities of given tokens with
entropy, top alternatives and the gradient that reaches the logits.

``run`` computes a case either in plain torch operations (``own`` false) or
with the library's calls (``own`` true).  ``exact`` evaluates the definitions in
64 bits, apart from both.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

LARGEST_CONV = 8 * 4096 * 4096            # elements of the largest convolution
LARGEST_SCAN = 16384 * 4096 * 16          # steps of one state number in the largest scan
LARGEST_SCAN_ADJOINT = 4 * 2048 * 4096 * 16
LARGEST_LOGITS = 4096 * 128000            # elements of the largest array of logits


def library():
    import differentiable_cholesky_amd as dc
    return dc


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one generated token for a batch of 64 sequences, whose last three inputs are kept and shifted in place
        {"name": "conv_token", "op": "conv", "batch": 64, "len": 1, "dim": 4096, "width": 4, "type": "bf16",
         "bias": True, "state": True},
        # a training batch of ordinary length
        {"name": "conv_batch", "op": "conv", "batch": 8, "len": 4096, "dim": 4096, "width": 4, "type": "bf16",
         "bias": True, "state": False},
        # its backward pass
        {"name": "conv_adjoint_batch", "op": "conv_adjoint", "batch": 8, "len": 4096, "dim": 4096, "width": 4,
         "type": "bf16", "bias": True, "state": False},
        # one generated token for a batch of 64 sequences, state kept in fp32 and updated in place
        {"name": "scan_token", "op": "scan", "batch": 64, "len": 1, "dim": 4096, "groups": 1, "states": 16,
         "type": "bf16", "state": True, "save": False},
        # the forward pass of a training batch, which keeps what its adjoint needs
        {"name": "scan_batch", "op": "scan", "batch": 4, "len": 2048, "dim": 4096, "groups": 1, "states": 16,
         "type": "bf16", "state": False, "save": True},
        # one long prompt, carried on from the state of what was read before it
        {"name": "scan_prompt", "op": "scan", "batch": 1, "len": 16384, "dim": 4096, "groups": 1, "states": 16,
         "type": "bf16", "state": True, "save": False},
        # odd sizes in full precision, for a gradient check or a small model, with two groups of B and C
        {"name": "scan_adjoint_odd", "op": "scan_adjoint", "batch": 2, "len": 1023, "dim": 2 * 257, "groups": 2,
         "states": 11, "type": "f32", "state": True, "save": True},
        # the backward pass of the training batch
        {"name": "scan_adjoint_batch", "op": "scan_adjoint", "batch": 4, "len": 2048, "dim": 4096, "groups": 1,
         "states": 16, "type": "bf16", "state": False, "save": True},
        # one generated token for a batch of 16 sequences: what it was and what else was likely
        {"name": "logprob_token", "op": "logprob", "rows": 16, "vocab": 128000, "type": "bf16", "top": 8,
         "masked": False, "scale": 0.8},
        # the evaluation of a text in full precision, odd rows, a part of the vocabulary forbidden
        {"name": "logprob_odd", "op": "logprob", "rows": 513, "vocab": 50257, "type": "f32", "top": 5,
         "masked": True, "scale": 1.0},
        # the loss of a training batch
        {"name": "logprob_batch", "op": "logprob", "rows": 4096, "vocab": 128000, "type": "bf16", "top": 0,
         "masked": False, "scale": 1.0},
        # its gradient, with that of the entropy
        {"name": "logprob_adjoint", "op": "logprob_adjoint", "rows": 4096, "vocab": 128000, "type": "bf16", "top": 0,
         "masked": False, "scale": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_adjoint", "scan", "scan", "scan_adjoint", "scan_adjoint", "logprob", "logprob",
                     "logprob_adjoint"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    # the largest listed cases are 16-bit: a 32-bit one has half their elements
    part = 2 if kind == "f32" else 1
    if op.startswith("conv"):
        batch, dim = _log(rng, 1, 64), _log(rng, 16, 8192)
        most = max(1, min(65536, LARGEST_CONV // (batch * dim * part)))
        return {"op": op, "batch": batch, "len": _log(rng, 1, most), "dim": dim, "width": rng.choice([2, 3, 4, 4]),
                "type": kind, "bias": rng.random() < 0.7, "state": rng.random() < 0.5}
    if op.startswith("scan"):
        batch, groups = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4])
        dim = groups * max(1, _log(rng, 16, 8192) // groups)
        states = rng.choice([4, 8, 11, 16, 16, 16, 32, 64])
        largest = LARGEST_SCAN if op == "scan" else LARGEST_SCAN_ADJOINT
        most = max(1, min(16384, largest // (batch * dim * max(states, 16) * part)))
        return {"op": op, "batch": batch, "len": _log(rng, 1, most), "dim": dim, "groups": groups, "states": states,
                "type": kind, "state": rng.random() < 0.5, "save": op == "scan_adjoint" or rng.random() < 0.5}
    vocab = _log(rng, 100, 256000)
    rows = _log(rng, 1, max(1, min(32768, LARGEST_LOGITS // (vocab * part))))
    return {"op": op, "rows": rows, "vocab": vocab, "type": kind,
            "top": rng.choice([0, 0, 1, 5, 8, 20]) if op == "logprob" else 0,
            "masked": rng.random() < 0.4, "scale": rng.choice([1.0, 0.7, 1.5])}


def _bytes(kind):
    return 4 if kind == "f32" else 2


def work(case):
    e = _bytes(case["type"])
    if case["op"].startswith("conv"):
        n, c, k = case["batch"] * case["len"] * case["dim"], case["dim"], case["width"]
        kept = case["batch"] * (k - 1) * c * e
        params = c * (k + (1 if case["bias"] else 0))
        if case["op"] == "conv":
            return {"bytes": 2 * e * n + e * params + kept * (2 if case["state"] else 1), "flops": (2 * k + 5) * n}
        return {"bytes": 3 * e * n + (e + 4) * params + (2 * kept if case["state"] else 0), "flops": (6 * k + 10) * n}
    if case["op"].startswith("scan"):
        n, c, s = case["batch"] * case["len"] * case["dim"], case["dim"], case["states"]
        bc = 2 * case["batch"] * case["len"] * case["groups"] * s
        ends = 4 * case["batch"] * c * s
        if case["op"] == "scan":
            return {"bytes": 4 * e * n + e * bc + 4 * c * (s + 2) + ends * (2 if case["state"] else 1),
                    "flops": n * (6 * s + 15)}
        return {"bytes": 7 * e * n + 2 * e * bc + 8 * c * (s + 2) + ends * (2 if case["state"] else 1),
                "flops": n * (20 * s + 40)}
    n = case["rows"] * case["vocab"]
    if case["op"] == "logprob":
        return {"bytes": e * n + case["rows"] * (20 + 12 * case["top"]), "flops": 6 * n}
    return {"bytes": 2 * e * n + 24 * case["rows"], "flops": 7 * n}


# ----------------------------------------------------------------- inputs ----

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=gen).to(dtype)

    kind = TYPES[case["type"]]
    s = {"case": case}
    if case["op"].startswith("conv"):
        batch, length, dim, width = case["batch"], case["len"], case["dim"], case["width"]
        s["x"] = normal(batch, length, dim, dtype=kind)
        s["w"] = normal(dim, width, std=width ** -0.5, dtype=kind)
        s["bias"] = normal(dim, std=0.3, dtype=kind) if case["bias"] else None
        s["state"] = normal(batch, width - 1, dim, dtype=kind) if case["state"] else None
        if case["op"] == "conv_adjoint":
            s["adj"] = normal(batch, length, dim, dtype=kind)
            s["adj_last"] = normal(batch, width - 1, dim, dtype=kind) if case["state"] else None
        return s
    if case["op"].startswith("scan"):
        batch, length, dim, states = case["batch"], case["len"], case["dim"], case["states"]
        # what follows a convolution with SiLU; steps between about 0.001 and 0.1, as a layer starts with
        s["u"] = torch.nn.functional.silu(normal(batch, length, dim)).to(kind)
        s["delta"] = normal(batch, length, dim, std=0.5, dtype=kind)
        rate = torch.empty(dim, device=DEV).uniform_(math.log(1e-3), math.log(0.1), generator=gen).exp()
        s["bias"] = torch.log(torch.expm1(rate))
        s["A"] = -torch.arange(1, states + 1, device=DEV) * torch.exp(normal(dim, states, std=0.1))
        for name in ("B", "C"):
            s[name] = normal(batch, length, case["groups"], states, dtype=kind)
        s["D"] = 1 + normal(dim, std=0.1)
        s["z"] = normal(batch, length, dim, dtype=kind)
        s["h0"] = normal(batch, dim, states, std=0.3) if case["state"] else None
        if case["op"] == "scan":
            # a decoding program keeps the state
            s["keep"] = s["h0"].clone() if length == 1 and case["state"] else None
            return s
        s["adj"] = normal(batch, length, dim, dtype=kind)
        s["adj_last"] = normal(batch, dim, states) if case["state"] else None
        if own:
            s["starts"] = library().chol_selective_scan(s["u"], s["delta"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
                                                        bias=s["bias"], h0=s["h0"], save=True)[2]
        return s
    rows, vocab = case["rows"], case["vocab"]
    x = normal(rows, vocab, std=2.5)
    tokens = torch.randint(0, vocab, (rows,), device=DEV, generator=gen)
    # most of the given tokens are likely ones
    x.scatter_add_(1, tokens[:, None], normal(rows, 1, std=2.0) + 8.0)
    if case["masked"]:
        closed = torch.rand(vocab, device=DEV, generator=gen) < 0.3
        closed[tokens] = False
        x.masked_fill_(closed[None], -math.inf)
        # padding at the end of the text has no token
        tokens[rows - rows // 8:] = -1
    s["x"], s["tokens"] = x.to(kind), tokens
    if case["op"] == "logprob_adjoint":
        s["adj_logp"], s["adj_entropy"] = normal(rows, std=1.0 / rows), normal(rows, std=0.1 / rows)
        y = s["x"].double() if vocab * rows < 1 << 24 else s["x"].float()
        y = y * case["scale"]
        m = y.amax(1, keepdim=True)
        lse = (m + torch.log(torch.exp(y - m).sum(1, keepdim=True)))
        log_p = y - lse
        s["lse"] = lse[:, 0].float()
        s["entropy"] = -torch.where(log_p == -math.inf, 0.0, torch.exp(log_p) * log_p).sum(1).float()
    return s


# ------------------------------------------------------------ plain forms ----

def _silu_slope(p):
    s = torch.sigmoid(p)
    return s * (1 + p * (1 - s))


def _conv_rows(s):
    """The inputs in 32 bits with the rows before the first."""
    x, k = s["x"].float(), s["case"]["width"]
    before = s["state"].float() if s["state"] is not None else x.new_zeros(x.shape[0], k - 1, x.shape[2])
    return torch.cat([before, x], 1)


def _conv_sum(s, rows):
    k, w, length = s["case"]["width"], s["w"].float(), s["case"]["len"]
    p = sum(rows[:, i:i + length] * w[:, i] for i in range(k))
    return p if s["bias"] is None else p + s["bias"].float()


def _conv(s):
    rows = _conv_rows(s)
    p = _conv_sum(s, rows)
    last = rows[:, rows.shape[1] - s["case"]["width"] + 1:].to(s["x"].dtype)
    return (p * torch.sigmoid(p)).to(s["x"].dtype), last


def _conv_adjoint(s):
    rows = _conv_rows(s)
    k, w, length = s["case"]["width"], s["w"].float(), s["case"]["len"]
    q = s["adj"].float() * _silu_slope(_conv_sum(s, rows))
    d = torch.zeros_like(rows)
    for i in range(k):
        d[:, i:i + length] += q * w[:, i]
    if s["adj_last"] is not None:
        d[:, length:] += s["adj_last"].float()
    out = {"adj_x": d[:, k - 1:].to(s["x"].dtype),
           "adj_w": torch.stack([(q * rows[:, i:i + length]).sum((0, 1)) for i in range(k)], 1)}
    if s["bias"] is not None:
        out["adj_bias"] = q.sum((0, 1))
    if s["state"] is not None:
        out["adj_state"] = d[:, :k - 1].to(s["x"].dtype)
    return out


BLOCK = 64      # steps that the plain scan composes at once


def _compose(a, b):
    """Inclusive composition of x -> a x + b along axis 1, by doubling."""
    shift = 1
    while shift < a.shape[1]:
        b = torch.cat([b[:, :shift], a[:, shift:] * b[:, :-shift] + b[:, shift:]], 1)
        a = torch.cat([a[:, :shift], a[:, shift:] * a[:, :-shift]], 1)
        shift *= 2
    return a, b


def _wide(x, dim):
    """[batch, len, groups, states] as [batch, len, dim, states], in 32 bits."""
    return x.float().repeat_interleave(dim // x.shape[2], 2)


def _scan_block(s, t, state):
    """Steps t .. t + BLOCK - 1 from a state: (steps, gates, states)."""
    part = slice(t, t + BLOCK)
    dt = torch.nn.functional.softplus(s["delta"][:, part].float() + s["bias"])
    gate = torch.exp(dt[..., None] * s["A"])
    more = (dt * s["u"][:, part].float())[..., None] * _wide(s["B"][:, part], dt.shape[2])
    a, h = _compose(gate, more)
    return dt, gate, a * state[:, None] + h


def _start(s):
    case = s["case"]
    first = s["keep"] if s.get("keep") is not None else s["h0"]
    return torch.zeros(case["batch"], case["dim"], case["states"], device=DEV) if first is None else first


def _scan(s):
    case, state, y = s["case"], _start(s), torch.empty_like(s["u"])
    for t in range(0, case["len"], BLOCK):
        part = slice(t, t + BLOCK)
        _, _, h = _scan_block(s, t, state)
        state = h[:, -1]
        z = s["z"][:, part].float()
        v = (h * _wide(s["C"][:, part], case["dim"])).sum(3) + s["D"] * s["u"][:, part].float()
        y[:, part] = (v * z * torch.sigmoid(z)).to(y.dtype)
    return y, state.clone()


def _scan_adjoint(s):
    case, state, starts = s["case"], _start(s), []
    dim, groups, batch = case["dim"], case["groups"], case["batch"]
    for t in range(0, case["len"], BLOCK):
        starts.append(state)
        state = _scan_block(s, t, state)[2][:, -1].clone()
    out = {k: torch.empty_like(s[n]) for k, n in (("adj_u", "u"), ("adj_delta", "delta"), ("adj_B", "B"), ("adj_C", "C"),
                                                   ("adj_z", "z"))}
    adj_a, adj_d, adj_bias = torch.zeros_like(s["A"]), torch.zeros(dim, device=DEV), torch.zeros(dim, device=DEV)
    mu = torch.zeros_like(state) if s["adj_last"] is None else s["adj_last"]
    for t in reversed(range(0, case["len"], BLOCK)):
        part, state = slice(t, t + BLOCK), starts[t // BLOCK]
        dt, gate, h = _scan_block(s, t, state)
        u, z, adj = (s[k][:, part].float() for k in ("u", "z", "adj"))
        b, c = _wide(s["B"][:, part], dim), _wide(s["C"][:, part], dim)
        v = (h * c).sum(3) + s["D"] * u
        out["adj_z"][:, part] = (adj * v * _silu_slope(z)).to(s["z"].dtype)
        adj = adj * z * torch.sigmoid(z)
        g = adj[..., None] * c
        g[:, -1] += mu
        following = torch.cat([gate[:, 1:], torch.zeros_like(gate[:, :1])], 1)
        g = _compose(following.flip(1), g.flip(1))[1].flip(1)
        mu = gate[:, 0] * g[:, 0]
        sums = lambda x: x.view(batch, -1, groups, dim // groups, case["states"]).sum(3)  # noqa: E731
        out["adj_C"][:, part] = sums(adj[..., None] * h).to(s["C"].dtype)
        out["adj_B"][:, part] = sums(g * (dt * u)[..., None]).to(s["B"].dtype)
        back = g * gate * torch.cat([state[:, None], h[:, :-1]], 1)
        along = (g * b).sum(3)
        adj_dt = u * along + (back * s["A"]).sum(3)
        adj_dt = adj_dt * torch.sigmoid(s["delta"][:, part].float() + s["bias"])
        out["adj_u"][:, part] = (dt * along + s["D"] * adj).to(s["u"].dtype)
        out["adj_delta"][:, part] = adj_dt.to(s["u"].dtype)
        adj_a += (back * dt[..., None]).sum((0, 1))
        adj_d += (adj * u).sum((0, 1))
        adj_bias += adj_dt.sum((0, 1))
    return {**out, "adj_A": adj_a, "adj_D": adj_d, "adj_bias": adj_bias, "adj_h0": mu}


def _top(x, count):
    """Indices of the largest values of each row, the lowest index first among equal ones."""
    bits = (x.float() + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    order = (order << 32) - torch.arange(x.shape[1], device=DEV)
    return torch.topk(order, count, dim=1).indices


def _logprob(s):
    x, tokens, case = s["x"].float() * s["case"]["scale"], s["tokens"], s["case"]
    m = x.amax(1, keepdim=True)
    shifted = x - m
    e = torch.exp(shifted)
    total = e.sum(1)
    log_total = torch.log(total)
    inner = torch.where(e > 0, shifted * e, 0.0).sum(1) / total
    lse = m[:, 0] + log_total
    given = x.gather(1, tokens.clamp(min=0)[:, None])[:, 0] - lse
    out = {"logp": torch.where(tokens >= 0, given, 0.0), "lse": lse, "entropy": log_total - inner}
    if case["top"]:
        ids = _top(s["x"], min(case["top"], case["vocab"]))
        out["top_ids"], out["top_logp"] = ids, x.gather(1, ids) - lse[:, None]
    return out


def _logprob_adjoint(s):
    scale, tokens = s["case"]["scale"], s["tokens"]
    log_p = s["x"].float() * scale - s["lse"][:, None]
    p = torch.exp(log_p)
    some = torch.where(tokens >= 0, s["adj_logp"], 0.0)
    d = torch.where(p > 0, -p * (some[:, None] + s["adj_entropy"][:, None] * (log_p + s["entropy"][:, None])), 0.0)
    d.scatter_add_(1, tokens.clamp(min=0)[:, None], some[:, None])
    return (d * scale).to(s["x"].dtype)


# -------------------------------------------------------------- one pass ----

def run(s):
    case = s["case"]
    op = case["op"]
    if op == "conv":
        # a decoding program's kept rows are replaced; others get new ones
        keep = s["state"] if case["len"] == 1 else None
        if own:
            y, last = library().chol_causal_conv(s["x"], s["w"], bias=s["bias"], state=s["state"], last=keep)
        else:
            y, last = _conv(s)
            if keep is not None:
                last = keep.copy_(last)
        return {"y": y, "last": last}
    if op == "conv_adjoint":
        if not own:
            return _conv_adjoint(s)
        adj_x, adj_w, adj_bias, adj_state = library().chol_causal_conv_adjoint(
            s["x"], s["w"], s["adj"], bias=s["bias"], state=s["state"], adjLast=s["adj_last"])
        out = {"adj_x": adj_x, "adj_w": adj_w, "adj_bias": adj_bias, "adj_state": adj_state}
        return {k: t for k, t in out.items() if t is not None}
    if op == "scan":
        keep = s["keep"]
        if own:
            y, last, _ = library().chol_selective_scan(
                s["u"], s["delta"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], bias=s["bias"],
                h0=s["h0"] if keep is None else keep, hlast=keep, save=case["save"])
        else:
            y, last = _scan(s)
            if keep is not None:
                last = keep.copy_(last)
        return {"y": y, "last": last}
    if op == "scan_adjoint":
        if not own:
            return _scan_adjoint(s)
        names = ("adj_u", "adj_delta", "adj_A", "adj_B", "adj_C", "adj_D", "adj_z", "adj_bias", "adj_h0")
        return dict(zip(names, library().chol_selective_scan_adjoint(
            s["u"], s["delta"], s["A"], s["B"], s["C"], s["starts"], s["adj"], D=s["D"], z=s["z"], bias=s["bias"],
            adjHlast=s["adj_last"])))
    if op == "logprob":
        if not own:
            return _logprob(s)
        r = library().chol_token_logprob(s["x"], s["tokens"], scale=case["scale"], top=min(case["top"], case["vocab"]))
        out = {"logp": r.logp, "lse": r.lse, "entropy": r.entropy}
        return {**out, "top_ids": r.top_ids, "top_logp": r.top_logp} if case["top"] else out
    if own:
        d = library().chol_token_logprob_adjoint(s["x"], s["tokens"], s["lse"], adjLogp=s["adj_logp"],
                                                 entropy=s["entropy"], adjEntropy=s["adj_entropy"], scale=case["scale"])
    else:
        d = _logprob_adjoint(s)
    return {"adj_logits": d}


# ---------------------------------------------------------------- exact ----

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("conv"):
        k, length = case["width"], case["len"]
        x, w = s["x"].double(), s["w"].double()
        offset = 0.0 if s["bias"] is None else s["bias"].double()
        state = None if s["state"] is None else s["state"].double()
        past = torch.zeros_like(x[:, :1]).expand(-1, k - 1, -1) if state is None else state
        whole = torch.cat([past, x], 1)
        p = (whole.unfold(1, k, 1) * w).sum(-1) + offset
        slope = 1 / (1 + torch.exp(-p))
        if op == "conv":
            return {"y": p * slope, "last": whole[:, length:]}
        q = s["adj"].double() * (slope + p * slope * (1 - slope))
        after = torch.nn.functional.pad(q, (0, 0, k - 1, k - 1))
        d = (after.unfold(1, k, 1) * w.flip(1)).sum(-1)
        if s["adj_last"] is not None:
            d[:, length:] += s["adj_last"].double()
        out = {"adj_x": d[:, k - 1:], "adj_w": torch.stack([(whole[:, i:i + length] * q).sum(1).sum(0)
                                                            for i in range(k)], 1)}
        if case["bias"]:
            out["adj_bias"] = q.sum(1).sum(0)
        if case["state"]:
            out["adj_state"] = d[:, :k - 1]
        return out
    if op.startswith("scan"):
        batch, length, dim, groups, states = (case[k] for k in ("batch", "len", "dim", "groups", "states"))
        wide = (batch, groups, dim // groups, states)
        raw = s["delta"].double() + s["bias"].double()
        dt = torch.logaddexp(raw, torch.zeros_like(raw))
        a, u = s["A"].double(), s["u"].double()
        h = torch.zeros(batch, dim, states, dtype=torch.float64, device=DEV) if s["h0"] is None else s["h0"].double()
        d = s["D"].double()
        gated = s["z"].double()
        sigma = 1 / (1 + torch.exp(-gated))
        train = op == "scan_adjoint"
        kept = torch.empty(length + 1, batch, dim, states, dtype=torch.float64, device=DEV) if train else None
        if train:
            kept[0] = h
        v = torch.empty_like(u)
        for t in range(length):
            b, c = (s[k][:, t].double()[:, :, None].expand(wide).reshape(batch, dim, states) for k in ("B", "C"))
            step = dt[:, t, :, None]
            h = torch.exp(step * a) * h + step * u[:, t, :, None] * b
            v[:, t] = (h * c).sum(-1) + d * u[:, t]
            if train:
                kept[t + 1] = h
        if not train:
            return {"y": v * gated * sigma, "last": h}
        adj = s["adj"].double()
        out = {"adj_z": adj * v * (sigma + gated * sigma * (1 - sigma))}
        adj = adj * gated * sigma
        lam = torch.zeros_like(h) if s["adj_last"] is None else s["adj_last"].double()
        for name in ("adj_u", "adj_delta"):
            out[name] = torch.empty_like(u)
        for name in ("adj_B", "adj_C"):
            out[name] = torch.empty(batch, length, groups, states, dtype=torch.float64, device=DEV)
        adj_a = torch.zeros_like(a)
        for t in reversed(range(length)):
            b, c = (s[k][:, t].double()[:, :, None].expand(wide).reshape(batch, dim, states) for k in ("B", "C"))
            step, x, o = dt[:, t, :, None], u[:, t, :, None], adj[:, t, :, None]
            lam = lam + o * c
            out["adj_C"][:, t] = (o * kept[t + 1]).view(wide).sum(2)
            out["adj_B"][:, t] = (lam * step * x).view(wide).sum(2)
            out["adj_u"][:, t] = (lam * step * b).sum(-1) + d * adj[:, t]
            gate = torch.exp(step * a)
            turn = lam * kept[t] * gate
            out["adj_delta"][:, t] = (lam * x * b + turn * a).sum(-1)
            adj_a += (turn * step).sum(0)
            lam = lam * gate
        out["adj_delta"] *= 1 / (1 + torch.exp(-raw))
        return {**{k: out[k] for k in ("adj_u", "adj_delta", "adj_B", "adj_C", "adj_z")}, "adj_A": adj_a,
                "adj_D": (adj * u).sum((0, 1)), "adj_bias": out["adj_delta"].sum((0, 1)), "adj_h0": lam}
    rows, scale = case["rows"], case["scale"]
    logp, lse, entropy, ids, top_logp, grads = [], [], [], [], [], []
    step = max(1, (1 << 26) // case["vocab"])
    for r in range(0, rows, step):
        part = slice(r, r + step)
        x, tokens = s["x"][part].double() * scale, s["tokens"][part]
        some = tokens >= 0
        size = torch.logsumexp(x, 1, keepdim=True)
        log_p = x - size
        chance = torch.exp(log_p)
        surprise = torch.where(chance > 0, log_p, 0.0)
        if op == "logprob_adjoint":
            # the row's statistics are inputs of this call
            log_p = x - s["lse"][part].double()[:, None]
            chance = torch.exp(log_p)
            surprise = torch.where(chance > 0, log_p + s["entropy"][part].double()[:, None], 0.0)
            weight = torch.where(some, s["adj_logp"][part], 0.0).double()
            d = -chance * (weight[:, None] + s["adj_entropy"][part].double()[:, None] * surprise)
            d[torch.arange(len(tokens), device=DEV)[some], tokens[some]] += weight[some]
            grads.append(d * scale)
            continue
        given = torch.zeros_like(size[:, 0])
        given[some] = log_p[torch.arange(len(tokens), device=DEV)[some], tokens[some]]
        logp.append(given), lse.append(size[:, 0]), entropy.append(-(chance * surprise).sum(1))
        if case["top"]:
            place = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :case["top"]]
            ids.append(place), top_logp.append(log_p.gather(1, place))
    if op == "logprob_adjoint":
        return {"adj_logits": torch.cat(grads)}
    out = {"logp": torch.cat(logp), "lse": torch.cat(lse), "entropy": torch.cat(entropy)}
    return {**out, "top_ids": torch.cat(ids), "top_logp": torch.cat(top_logp)} if case["top"] else out
