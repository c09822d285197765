"""The measured cases of the training-step operators next to the factor: the
gated linear recurrence and its adjoint, the RMS norm with the residual's
addition (16-bit or 8-bit output) and its adjoint, and the AdamW step over many
tensors with 32-bit or 8-bit states.

``run`` computes a case either in plain torch operations (``own`` false) or
with the library's calls (``own`` true).  ``exact`` evaluates the definitions in
64 bits, apart from both.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
BLOCK = 256          # elements that share one scale of an 8-bit optimiser state
MASK32 = 0xFFFFFFFF

LARGEST_SEQUENCE = 65536 * 2048       # elements of the largest recurrence
LARGEST_ROWS = 16384 * 4096           # elements of the largest norm
LAYERS, WIDTH = 6, 2048               # the largest parameter list (302 M elements)


def library():
    import differentiable_cholesky_amd as dc
    return dc


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one generated token for a batch of 64 sequences, state kept in fp32 and updated in place
        {"name": "recurrence_token", "op": "recurrence", "batch": 64, "len": 1, "dim": 2048, "type": "bf16",
         "gate": "log", "state": True},
        # a training batch of ordinary length
        {"name": "recurrence_batch", "op": "recurrence", "batch": 8, "len": 4096, "dim": 2048, "type": "bf16",
         "gate": "log", "state": False},
        # one long document: little work across channels, all of it along the sequence
        {"name": "recurrence_long", "op": "recurrence", "batch": 1, "len": 65536, "dim": 2048, "type": "bf16",
         "gate": "linear", "state": True},
        # odd length and width in full precision, for a gradient check or a small model
        {"name": "recurrence_adjoint_odd", "op": "recurrence_adjoint", "batch": 3, "len": 2047, "dim": 1001,
         "type": "f32", "gate": "linear", "state": True},
        # the backward pass of the long document
        {"name": "recurrence_adjoint_long", "op": "recurrence_adjoint", "batch": 1, "len": 65536, "dim": 2048,
         "type": "bf16", "gate": "log", "state": False},
        # the norm of a decoding step
        {"name": "rmsnorm_token", "op": "rmsnorm", "rows": 8, "cols": 4096, "type": "bf16", "out": "same",
         "group": 0, "residual": True},
        # a prefill whose next product takes 8-bit operands with a scale for every 128 columns
        {"name": "rmsnorm_8bit", "op": "rmsnorm", "rows": 8192, "cols": 4096, "type": "bf16", "out": "e4m3",
         "group": 128, "residual": True},
        # odd rows, one scale a row
        {"name": "rmsnorm_8bit_odd", "op": "rmsnorm", "rows": 4099, "cols": 1003, "type": "f32", "out": "e4m3",
         "group": 0, "residual": False},
        # the backward pass of a training batch
        {"name": "rmsnorm_adjoint", "op": "rmsnorm_adjoint", "rows": 16384, "cols": 4096, "type": "bf16",
         "residual": True},
        # a small model: many small tensors in fp32
        {"name": "adamw_small", "op": "adamw", "layers": 4, "width": 96, "type": "f32", "master": False, "bits": 32},
        # a large model: bf16 weights and gradients, fp32 master weights and states
        {"name": "adamw_large", "op": "adamw", "layers": LAYERS, "width": WIDTH, "type": "bf16", "master": True,
         "bits": 32},
        # the same with 8-bit states
        {"name": "adamw_8bit", "op": "adamw", "layers": LAYERS, "width": WIDTH, "type": "bf16", "master": True,
         "bits": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["recurrence", "recurrence_adjoint", "rmsnorm", "rmsnorm_adjoint", "adamw"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    # the largest listed cases are 16-bit: a 32-bit one has half their elements
    part = 2 if kind == "f32" else 1
    if op.startswith("recurrence"):
        batch, dim = _log(rng, 1, 16), _log(rng, 16, 4096)
        most = max(1, min(65536, LARGEST_SEQUENCE // (batch * dim * part)))
        return {"op": op, "batch": batch, "len": _log(rng, 1, most), "dim": dim, "type": kind,
                "gate": rng.choice(["linear", "log"]), "state": rng.random() < 0.5}
    if op.startswith("rmsnorm"):
        cols = _log(rng, 64, 16384)
        most = max(1, min(16384, LARGEST_ROWS // (cols * part)))
        case = {"op": op, "rows": _log(rng, 1, most), "cols": cols, "type": kind, "residual": rng.random() < 0.7}
        if op == "rmsnorm":
            case["out"] = rng.choice(["same", "e4m3"])
            case["group"] = rng.choice([0, 64, 128]) if case["out"] == "e4m3" else 0
        return case
    return {"op": op, "layers": rng.randint(1, LAYERS), "width": _log(rng, 16, WIDTH), "type": kind,
            "master": kind != "f32" and rng.random() < 0.7, "bits": rng.choice([32, 8])}


def _bytes(kind):
    return 4 if kind == "f32" else 2


def _sizes(case):
    """Element counts of a model's tensors: per layer the matrices of the recurrence's and the mixer's
    projections, and the vectors between them."""
    w = case["width"]
    return [s for _ in range(case["layers"]) for s in (3 * w * w, w, w * w, w, 4 * w * w, 4 * w, 4 * w * w, w)]


def work(case):
    e = _bytes(case["type"])
    if case["op"].startswith("recurrence"):
        n = case["batch"] * case["len"] * case["dim"]
        ends = 8 * case["batch"] * case["dim"] if case["state"] else 0
        if case["op"] == "recurrence":
            return {"bytes": 3 * e * n + ends, "flops": 2 * n}
        return {"bytes": 5 * e * n + ends, "flops": 3 * n}
    if case["op"].startswith("rmsnorm"):
        n, c = case["rows"] * case["cols"], case["cols"]
        if case["op"] == "rmsnorm_adjoint":
            return {"bytes": (4 if case["residual"] else 3) * e * n + e * c + 4 * c, "flops": 10 * n}
        moved = e * n * (3 if case["residual"] else 1)
        if case["out"] == "same":
            return {"bytes": moved + e * n + e * c, "flops": 5 * n}
        groups = case["rows"] * (-(-c // case["group"]) if case["group"] else 1)
        return {"bytes": moved + n + 4 * groups + e * c, "flops": 8 * n}
    n = sum(_sizes(case))
    weights = 2 * e + (8 if case["master"] else 0) - (e if case["master"] else 0)   # with a master the copy is only written
    states = 16 if case["bits"] == 32 else 4 + 16.0 / BLOCK
    return {"bytes": (weights + e + states) * n, "flops": 15 * n}


# ----------------------------------------------------------------- inputs ----

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=gen).to(dtype)

    kind = TYPES[case["type"]]
    if case["op"].startswith("recurrence"):
        shape = (case["batch"], case["len"], case["dim"])
        # gates between about 0.8 and 0.999, as a trained layer has them; the input is scaled by sqrt(1 - a^2)
        # so that the state keeps unit size
        rate = torch.exp(normal(*shape) * 0.7 - 4.0)
        a = torch.exp(-rate)
        s = {"case": case, "a": (-rate if case["gate"] == "log" else a).to(kind)}
        b = (normal(*shape) * torch.sqrt(1 - a * a)).to(kind)
        s["h0"] = normal(case["batch"], case["dim"]) if case["state"] else None
        if case["op"] == "recurrence":
            s["b"] = b
            # a decoding program keeps the state and the token's output
            s["state"] = s["h0"].clone() if case["len"] == 1 and case["state"] else None
        else:
            s["h"] = _recurrence(s["a"], b, s["h0"], case["gate"])[0]
            s["adj"] = normal(*shape, dtype=kind)
            s["adj_last"] = normal(case["batch"], case["dim"]) if case["state"] else None
        return s
    if case["op"].startswith("rmsnorm"):
        shape = (case["rows"], case["cols"])
        s = {"case": case, "w": (1 + normal(case["cols"], std=0.1)).to(kind)}
        if case["op"] == "rmsnorm":
            s["x"] = normal(*shape, dtype=kind)
            s["r"] = normal(*shape, std=3.0, dtype=kind) if case["residual"] else None
        else:
            s["h"] = normal(*shape, std=3.0, dtype=kind)
            s["adj"] = normal(*shape, dtype=kind)
            s["adj_h"] = normal(*shape, dtype=kind) if case["residual"] else None
        return s
    # parameters as views into flat storage, each starting at a multiple of BLOCK elements
    sizes, starts, at = _sizes(case), [], 0
    for n in sizes:
        starts.append(at)
        at += -(-n // BLOCK) * BLOCK
    pad = torch.ones(at, dtype=torch.bool, device=DEV)
    for n, o in zip(sizes, starts):
        pad[o:o + n] = False
    weights = normal(at, std=0.02).masked_fill_(pad, 0.0)
    grads = normal(at, std=1e-3).masked_fill_(pad, 0.0)
    s = {"case": case, "p": weights.to(kind), "master": weights if case["master"] else None, "g": grads.to(kind),
         "hyper": {"step": 100, "lr": 1e-4, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.1},
         "clip": torch.tensor([0.5], device=DEV), "seed": seed & MASK32}
    m = normal(at, std=3e-4).masked_fill_(pad, 0.0)
    root = (normal(at, std=2e-4).abs_() + 1e-5).masked_fill_(pad, 0.0)
    if case["bits"] == 32:
        s["m"], s["v"] = m, root * root
        s["m_scale"] = s["v_scale"] = None
    else:
        noise = _noise(at, s["seed"] ^ 0x5A5A5A5A)
        s["m"], s["m_scale"] = _to_8bit(m, noise & 0xFFFF, False)
        s["v"], s["v_scale"] = _to_8bit(root, noise >> 16, True)
    if own:
        cut = lambda t: [t[o:o + n] for o, n in zip(starts, sizes)] if t is not None else None  # noqa: E731
        tiles = lambda t: ([t[o // BLOCK:(o + n + BLOCK - 1) // BLOCK] for o, n in zip(starts, sizes)]  # noqa: E731
                           if t is not None else None)
        s["list"] = library().chol_adamw_list(cut(s["p"]), cut(s["g"]), cut(s["m"]), cut(s["v"]),
                                              master=cut(s["master"]), m_scale=tiles(s["m_scale"]),
                                              v_scale=tiles(s["v_scale"]), first=starts)
    return s


# ------------------------------------------------------------ plain forms ----

def _scan(a, b):
    """Inclusive composition of x -> a x + b along axis 1, by doubling."""
    shift = 1
    while shift < a.shape[1]:
        b = torch.cat([b[:, :shift], a[:, shift:] * b[:, :-shift] + b[:, shift:]], 1)
        a = torch.cat([a[:, :shift], a[:, shift:] * a[:, :-shift]], 1)
        shift *= 2
    return a, b


def _gates(x, gate):
    return torch.exp(x.float()) if gate == "log" else x.float()


def _recurrence(x, b, h0, gate):
    a, h = _scan(_gates(x, gate), b.float())
    if h0 is not None:
        h = a * h0[:, None] + h
    return h.to(x.dtype), h[:, -1].clone()


def _recurrence_adjoint(x, h, adj, h0, adj_last, gate):
    a = _gates(x, gate)
    lam = adj.to(torch.float32, copy=True)
    if adj_last is not None:
        lam[:, -1] += adj_last
    nxt = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    lam = _scan(nxt.flip(1), lam.flip(1))[1].flip(1)
    first = torch.zeros_like(lam[:, 0]) if h0 is None else h0
    before = torch.cat([first[:, None], h[:, :-1].float()], 1)
    adj_a = lam * before * a if gate == "log" else lam * before
    return adj_a.to(x.dtype), lam.to(x.dtype), a[:, 0] * lam[:, 0]


EPS = 1e-6


def _rmsnorm(x, r, w, group, quantise):
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    f = h.float()
    y = f * torch.rsqrt((f * f).mean(1, keepdim=True) + EPS) * w.float()
    if not quantise:
        return h, y.to(x.dtype)
    rows, cols = y.shape
    size = group or cols
    count = -(-cols // size)
    full = torch.nn.functional.pad(y, (0, count * size - cols)).view(rows, count, size)
    most = full.abs().amax(2, keepdim=True)
    some = most > 0
    q = (full * torch.where(some, E4M3_MAX / most, 1.0)).to(E4M3).view(rows, -1)[:, :cols].contiguous()
    return h, q, torch.where(some, most / E4M3_MAX, 1.0).view(rows, count)


def _rmsnorm_adjoint(h, w, adj, adj_h):
    f, g = h.float(), adj.float() * w.float()
    s = torch.rsqrt((f * f).mean(1, keepdim=True) + EPS)
    d = s * (g - f * (s * s) * (g * f).mean(1, keepdim=True))
    if adj_h is not None:
        d = d + adj_h.float()
    return d.to(h.dtype), (adj.float() * f * s).sum(0)


def _mix(x):
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B1) & MASK32
    x = x ^ (x >> 15)
    x = (x * 0x85EBCA77) & MASK32
    return x ^ (x >> 16)


def _noise(count, seed):
    """32 random bits for every element of a parameter list, from the seed and the element's position."""
    key = torch.tensor(seed, dtype=torch.int64, device=DEV)
    return _mix((torch.arange(count, dtype=torch.int64, device=DEV) + _mix(key)) & MASK32)


def _to_8bit(x, noise, keep):
    """e4m3 codes of x and a power-of-two scale for every BLOCK elements, rounded up where the 16 random bits
    of `noise` and what is dropped carry; keep: a nonzero value is not stored as zero."""
    x = x.view(-1, BLOCK)
    most = (x.view(torch.int32) & 0x7FFFFFFF).amax(1, keepdim=True)
    field = torch.clamp((most >> 23) - 7, min=1)
    scale = (field << 23).view(torch.float32)
    y = (x * ((254 - field) << 23).view(torch.float32)).view(-1)
    bits = y.view(torch.int32).long()
    mag = bits & 0x7FFFFFFF
    small = torch.floor(y.abs() * 512.0 + noise.float() * 2.0 ** -16)
    code = torch.where(mag >= 0x3C800000, ((mag + (noise << 4)) >> 20) - (120 << 3),
                       torch.where(y.abs() < 0.015625, small, 0.0).long())
    if keep:
        code = torch.where(mag > 0, torch.clamp(code, min=1), code)
    code = torch.where(mag >= 0x7F800000, 0x7F, code)
    return (code | ((bits >> 24) & 0x80)).to(torch.uint8).view(E4M3), scale.view(-1)


def _from_8bit(code, scale):
    return (code.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def _adamw(s):
    k = s["hyper"]
    p = s["p"].float() if s["master"] is None else s["master"]
    g = s["g"].float() * s["clip"]
    if s["m_scale"] is None:
        m, v = s["m"], s["v"]
    else:
        m, r = _from_8bit(s["m"], s["m_scale"]), _from_8bit(s["v"], s["v_scale"])
        v = r * r
    m = m * k["beta1"] + g * (1 - k["beta1"])
    v = v * k["beta2"] + g * g * (1 - k["beta2"])
    root = torch.sqrt(v)
    p = p - p * (k["lr"] * k["weight_decay"])
    p = p - (k["lr"] / (1 - k["beta1"] ** k["step"])) * m / (root / math.sqrt(1 - k["beta2"] ** k["step"]) + k["eps"])
    if s["master"] is not None:
        s["master"].copy_(p)
    s["p"].copy_(p)
    if s["m_scale"] is None:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return
    noise = _noise(m.numel(), s["seed"])
    for name, value, bits, keep in (("m", m, noise & 0xFFFF, False), ("v", root, noise >> 16, True)):
        code, scale = _to_8bit(value, bits, keep)
        s[name].copy_(code)
        s[name + "_scale"].copy_(scale)


# -------------------------------------------------------------- one pass ----

def run(s):
    case = s["case"]
    op = case["op"]
    if op == "recurrence":
        keep = s["state"]
        if own:
            h, last = library().chol_recurrence(s["a"], s["b"], h0=s["h0"] if keep is None else keep, hlast=keep,
                                                gate=case["gate"])
        else:
            h, last = _recurrence(s["a"], s["b"], s["h0"] if keep is None else keep, case["gate"])
            if keep is not None:
                last = keep.copy_(last)
        return {"h": h, "last": last}
    if op == "recurrence_adjoint":
        if own:
            adj_a, adj_b, adj_h0 = library().chol_recurrence_adjoint(s["a"], s["h"], s["adj"], h0=s["h0"],
                                                                     adjHlast=s["adj_last"], gate=case["gate"])
        else:
            adj_a, adj_b, adj_h0 = _recurrence_adjoint(s["a"], s["h"], s["adj"], s["h0"], s["adj_last"],
                                                       case["gate"])
        return {"adj_a": adj_a, "adj_b": adj_b, "adj_h0": adj_h0}
    if op == "rmsnorm":
        if case["out"] == "same":
            if own:
                y, h = library().chol_rmsnorm(s["x"], s["w"], residual=s["r"], eps=EPS)
            else:
                h, y = _rmsnorm(s["x"], s["r"], s["w"], 0, False)
            return {"h": h, "y": y} if case["residual"] else {"y": y}
        if own:
            q, scale, h = library().chol_rmsnorm_quant(s["x"], s["w"], residual=s["r"], group=case["group"], eps=EPS)
        else:
            h, q, scale = _rmsnorm(s["x"], s["r"], s["w"], case["group"], True)
        out = {"q": q, "scale": scale}
        return {**out, "h": h} if case["residual"] else out
    if op == "rmsnorm_adjoint":
        if own:
            adj_x, adj_w = library().chol_rmsnorm_adjoint(s["h"], s["w"], s["adj"], adjH=s["adj_h"], eps=EPS)
        else:
            adj_x, adj_w = _rmsnorm_adjoint(s["h"], s["w"], s["adj"], s["adj_h"])
        return {"adj_x": adj_x, "adj_w": adj_w}
    if own:
        library().chol_adamw(s["list"], grad_scale=s["clip"], seed=s["seed"], **s["hyper"])
    else:
        _adamw(s)
    return {k: s[k] for k in ("p", "master", "m", "v", "m_scale", "v_scale") if s[k] is not None}


# ---------------------------------------------------------------- exact ----

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("recurrence"):
        x = s["a"].double()
        a = x.exp() if case["gate"] == "log" else x
        state = torch.zeros_like(a[:, 0]) if s["h0"] is None else s["h0"].double()
        if op == "recurrence":
            h = s["b"].double()
            for t in range(case["len"]):
                h[:, t].addcmul_(a[:, t], state)
                state = h[:, t]
            return {"h": h, "last": state}
        lam = s["adj"].double()
        if s["adj_last"] is not None:
            lam[:, -1] += s["adj_last"].double()
        for t in range(case["len"] - 1, 0, -1):
            lam[:, t - 1].addcmul_(a[:, t], lam[:, t])
        adj_a = lam.clone()
        adj_a[:, 0] *= state
        adj_a[:, 1:] *= s["h"][:, :-1].double()
        if case["gate"] == "log":
            adj_a *= a
        return {"adj_a": adj_a, "adj_b": lam, "adj_h0": a[:, 0] * lam[:, 0]}
    if op.startswith("rmsnorm"):
        w = s["w"].double()
        if op == "rmsnorm":
            h = s["x"] if s["r"] is None else (s["x"].double() + s["r"].double()).to(s["x"].dtype)
            d = h.double()
            y = d / torch.sqrt(d.square().mean(-1, keepdim=True) + EPS) * w
            if case["out"] == "same":
                return {"h": h, "y": y} if case["residual"] else {"y": y}
            parts = y.split(case["group"] or case["cols"], dim=1)
            scales = [p.abs().amax(1, keepdim=True) / E4M3_MAX for p in parts]
            out = {"q": torch.cat([(p / t).to(E4M3).double() for p, t in zip(parts, scales)], 1),
                   "scale": torch.cat(scales, 1)}
            return {**out, "h": h} if case["residual"] else out
        d, adj = s["h"].double(), s["adj"].double()
        size = torch.sqrt(d.square().mean(-1, keepdim=True) + EPS)
        unit = d / size
        along = (adj * w * unit).mean(-1, keepdim=True)
        adj_x = (adj * w - unit * along) / size
        if s["adj_h"] is not None:
            adj_x += s["adj_h"].double()
        return {"adj_x": adj_x, "adj_w": (adj * unit).sum(0)}
    k = s["hyper"]
    grad = s["g"].double() * s["clip"].double()
    old = (s["p"] if s["master"] is None else s["master"]).double()
    if case["bits"] == 32:
        m, v = s["m"].double(), s["v"].double()
    else:
        m = s["m"].double() * s["m_scale"].double().repeat_interleave(BLOCK)
        v = (s["v"].double() * s["v_scale"].double().repeat_interleave(BLOCK)).square()
    m.mul_(k["beta1"]).add_(grad, alpha=1 - k["beta1"])
    v.mul_(k["beta2"]).addcmul_(grad, grad, value=1 - k["beta2"])
    mean, var = m / (1 - k["beta1"] ** k["step"]), v / (1 - k["beta2"] ** k["step"])
    new = old * (1 - k["lr"] * k["weight_decay"]) - k["lr"] * mean / (var.sqrt() + k["eps"])
    out = {"p": new}
    if case["master"]:
        out["master"] = new
    if case["bits"] == 32:
        return {**out, "m": m, "v": v}
    # the stored states: one of the two neighbours in e4m3, by the random bits; scales are exact powers of two
    # chosen by comparison and have no value between
    place = torch.arange(m.numel(), dtype=torch.int64, device=DEV)
    bits = _mix((place + _mix(torch.tensor(s["seed"], dtype=torch.int64, device=DEV))) & MASK32)
    for name, value, part in (("m", m, bits % 65536), ("v", v.sqrt(), bits // 65536)):
        most = value.abs().view(-1, BLOCK).amax(1)
        low = torch.floor(torch.log2(torch.clamp(most, min=2.0 ** -119))) - 7
        y = value / torch.exp2(low).repeat_interleave(BLOCK)
        step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(y.abs(), min=2.0 ** -20))), min=-6) - 3)
        code = torch.floor(y.abs() / step + part.double() / 65536) * step
        if name == "v":
            code = torch.where((y != 0) & (code == 0), 2.0 ** -9, code)
        out[name] = code * torch.sign(y)
    return {**out, "m_scale": None, "v_scale": None}
