"""Plain 64-bit implementations of the convolution, the scan and the token log
probabilities, each with a bound on how far a kernel may be off that computes in fp32
and rounds its outputs once.

U is half a step of fp32.  Bounds count roundings: a sum of n products is off by at most
(n + 1) U of the sum of their magnitudes; an error that a later step multiplies is
carried on with the magnitudes, in the same recurrences as the values.
"""
import torch

import train_util
from train_util import U

# (differences are taken of 64-bit inputs, whose bounds nobody reads)
HALF = {**train_util.HALF, torch.float64: 0.0}
TINY = {**train_util.TINY, torch.float64: 0.0}
FLOOR = 1e-35   # results that pass through a reciprocal below 2^-126 are zero


def cuda(x):
    return None if x is None else x.cuda()


def rounded(ref, err, dtype):
    return HALF[dtype] * ref.abs() + (1 + HALF[dtype]) * err + TINY[dtype] + FLOOR


def sigmoid_err(p, dtype):
    """Relative error of 1 / (1 + exp(-p)): the exponential's (2 U of its own, and |p| 1.5 U
    where the exponent is one rounded product, at most 4 U where it is not), a sum and a
    reciprocal of one step."""
    return (8 + (1.5 if HALF[dtype] > U else 0.0) * p.abs()) * U


def slope_of(p):
    s = torch.sigmoid(p)
    return s * (1 + p * (1 - s))


def slope_err(p, dtype):
    """s (1 + p (1 - s)): the error of s enters twice, 1 - s is off by U more and multiplied by p."""
    s = torch.sigmoid(p)
    e = sigmoid_err(p, dtype) + 3 * U
    return e * slope_of(p).abs() + s * p.abs() * (e * s + 3 * U) + 2 * U


# ------------------------------------------------------------- convolution ----

def conv64(x, w, bias, state, silu):
    k, length = w.shape[1], x.shape[1]
    x, w = x.double(), w.double()
    before = x.new_zeros(x.shape[0], k - 1, x.shape[2]) if state is None else state.double()
    rows = torch.cat([before, x], 1)
    taps = [rows[:, i:i + length] * w[:, i] for i in range(k)]
    b = 0.0 if bias is None else bias.double()
    p, size = sum(taps) + b, sum(t.abs() for t in taps) + abs(b)
    return rows, p, (k + 1) * U * size, rows[:, length:]


def conv_forward(x, w, bias, state, silu):
    """(y, last) and y's bound."""
    _, p, err, last = conv64(x, w, bias, state, silu)
    if not silu:
        return p, last, rounded(p, err, x.dtype)
    y = p * torch.sigmoid(p)
    return y, last, rounded(y, 1.1 * err + y.abs() * (sigmoid_err(p, x.dtype) + U), x.dtype)


def conv_adjoint(x, w, adj, bias, state, adj_last, silu):
    """(adjX, adjW, adjBias, adjState) and their bounds."""
    rows, p, err, _ = conv64(x, w, bias, state, silu)
    k, length, t = w.shape[1], x.shape[1], x.dtype
    w, adj = w.double(), adj.double()
    if silu:
        q = adj * slope_of(p)
        qe = adj.abs() * (slope_err(p, t) + 0.5 * err) + U * q.abs()
    else:
        q, qe = adj, torch.zeros_like(adj)
    d, de = torch.zeros_like(rows), torch.zeros_like(rows)
    for i in range(k):
        d[:, i:i + length] += q * w[:, i]
        de[:, i:i + length] += (qe + (k + 2) * U * q.abs()) * w[:, i].abs()
    if adj_last is not None:
        d[:, length:] += adj_last.double()
        de[:, length:] += (k + 2) * U * adj_last.double().abs()
    # a run of at most 128 steps, the runs of a workgroup, every sixteenth workgroup, sixteen sums
    n = x.shape[0] * length
    depth = min(n, 128 + 256 + n // 128 + 16) + 1
    dw = torch.stack([(q * rows[:, i:i + length]).sum((0, 1)) for i in range(k)], 1)
    dwe = torch.stack([((qe + depth * U * q.abs()) * rows[:, i:i + length].abs()).sum((0, 1)) for i in range(k)], 1)
    db, dbe = q.sum((0, 1)), (qe + depth * U * q.abs()).sum((0, 1))
    values = (d[:, k - 1:], dw, db, d[:, :k - 1])
    bounds = (rounded(d[:, k - 1:], de[:, k - 1:], t), dwe + TINY[torch.float32], dbe + TINY[torch.float32],
              rounded(d[:, :k - 1], de[:, :k - 1], t))
    return values, bounds


# -------------------------------------------------------------------- scan ----

class Scan64:
    """The scan's values and bounds in 64 bits, step by step, and its adjoint's."""

    def __init__(self, u, delta, A, B, C, D, z, bias, h0, softplus=True):
        self.dtype, self.D = u.dtype, None if D is None else D.double()
        batch, length, dim = u.shape
        n = A.shape[1]
        wide = lambda x: (x if x.dim() == 4 else x[:, :, None]).double()  # noqa: E731
        B, C = wide(B), wide(C)
        self.groups = B.shape[2]
        self.B, self.C = (x.repeat_interleave(dim // self.groups, 2) for x in (B, C))
        self.u, self.A, self.z = u.double(), A.double(), None if z is None else z.double()
        raw = delta.double() + (0.0 if bias is None else bias.double())
        self.raw, self.softplus = raw, softplus
        self.dt = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
        # raw is rounded once (softplus changes by at most that of itself), the exponential, the
        # logarithm and the sums by a few more
        self.dt_err = (raw.abs() + 8) * U if softplus else torch.full_like(raw, U)
        state = u.new_zeros(batch, dim, n, dtype=torch.float64) if h0 is None else h0.double()
        size, err = state.abs(), torch.zeros_like(state)
        self.h, self.s, self.d = [state], [size], [err]
        self.e, self.E = [], []
        for t in range(length):
            x = self.dt[:, t, :, None] * self.A
            e = torch.exp(x)
            # dt's own error, the rounded exponent (3 U of it), the hardware's exponential; and where runs of
            # steps are composed, the rounding of the sum of their steps, in four parts
            E = x.abs() * (self.dt_err[:, t, :, None] + (4 + length / 4) * U) + 4 * U
            more = (self.dt * self.u)[:, t, :, None] * self.B[:, t]
            err = e * err + (E + 2 * U) * e * size + (self.dt_err[:, t, :, None] + 5 * U) * more.abs()
            state, size = e * state + more, e * size + more.abs()
            self.e.append(e), self.E.append(E), self.h.append(state), self.s.append(size), self.d.append(err)
        stack = lambda x: torch.stack(x[1:], 1) if length else u.new_zeros(batch, 0, dim, n, dtype=torch.float64)  # noqa: E731
        h, s, d = stack(self.h), stack(self.s), stack(self.d)
        self.v = (self.C * h).sum(3)
        self.v_err = (self.C.abs() * (d + (n + 4) * U * s)).sum(3)
        if D is not None:
            self.v = self.v + self.D * self.u
            self.v_err = self.v_err + 3 * U * (self.v.abs() + (self.D * self.u).abs())
        self.last, self.last_err = state, err + TINY[torch.float32]

    def forward(self):
        """(y, hlast) and their bounds."""
        y, err = self.v, self.v_err
        if self.z is not None:
            g = self.z * torch.sigmoid(self.z)
            err = err * g.abs() + (y * g).abs() * (sigmoid_err(self.z, self.dtype) + 3 * U)
            y = y * g
        return (y, self.last), (rounded(y, err, self.dtype), self.last_err)

    def adjoint(self, adj, adj_last):
        """(adjU, adjDelta, adjA, adjB, adjC, adjD, adjZ, adjBias, adjH0) and their bounds."""
        adj, t32 = adj.double(), TINY[torch.float32]
        batch, length, dim = adj.shape
        n, per = self.A.shape[1], dim // self.groups
        out, err = {}, {}
        a, rel = adj, torch.zeros_like(adj)
        if self.z is not None:
            slope = slope_of(self.z)
            out["z"] = adj * self.v * slope
            err["z"] = rounded(out["z"], adj.abs() * (self.v_err * slope.abs() +
                                                      self.v.abs() * (slope_err(self.z, self.dtype) + 3 * U)), self.dtype)
            a, rel = adj * self.z * torch.sigmoid(self.z), sigmoid_err(self.z, self.dtype) + 3 * U
        mu = torch.zeros_like(self.last) if adj_last is None else adj_last.double()
        ms, md = mu.abs(), torch.zeros_like(mu)
        # lanes of a row, waves, workgroups
        depth = (16 + 8 + per // 128 + 4) * U
        over = lambda x: x.view(batch, self.groups, per, n).sum(2)  # noqa: E731
        names = ("u", "dt", "B", "C")
        val, bnd = {k: [None] * length for k in names}, {k: [None] * length for k in names}
        dA, dAe, dAs = (torch.zeros_like(self.A) for _ in range(3))
        for t in range(length - 1, -1, -1):
            o, dt, x = a[:, t, :, None], self.dt[:, t, :, None], self.u[:, t, :, None]
            oe, te = rel[:, t, :, None], self.dt_err[:, t, :, None]
            B, C, e, E = self.B[:, t], self.C[:, t], self.e[t], self.E[t]
            h, s, d, h1, s1, d1 = self.h[t + 1], self.s[t + 1], self.d[t + 1], self.h[t], self.s[t], self.d[t]
            g, gs = C * o + mu, (C * o).abs() + ms
            gd = (C * o).abs() * (oe + 2 * U) + md + U * gs
            val["C"][t] = over(o * h)
            bnd["C"][t] = over(o.abs() * (d + (oe + 2 * U + depth) * s))
            val["B"][t] = over(g * dt * x)
            bnd["B"][t] = over((dt * x).abs() * (gd + (te + 3 * U + depth) * gs))
            along, ae = (g * B).sum(2), (B.abs() * (gd + (n + 4) * U * gs)).sum(2)
            big = (B.abs() * gs).sum(2)
            mu, ms, md = e * g, e * gs, e * gd + (E + 2 * U) * e * gs
            w, ws, wd = mu * h1, ms * s1, md * s1 + ms * d1 + 2 * U * ms * s1
            back, be = (self.A * w).sum(2), (self.A.abs() * (wd + (n + 6) * U * ws)).sum(2)
            bigger = (self.A.abs() * ws).sum(2)
            x, dt, te, o, oe = (q[..., 0] for q in (x, dt, te, o, oe))
            val["u"][t], bnd["u"][t] = dt * along, dt.abs() * (ae + (te + 3 * U) * big)
            if self.D is not None:
                val["u"][t] = val["u"][t] + self.D * o
                bnd["u"][t] = bnd["u"][t] + (self.D * o).abs() * (oe + 3 * U)
            val["dt"][t], bnd["dt"][t] = x * along + back, x.abs() * (ae + 3 * U * big) + be + 3 * U * bigger
            dA += (dt[..., None] * w).sum(0)
            dAe += (dt[..., None] * (wd + (te[..., None] + 2 * U) * ws)).abs().sum(0)
            dAs += (dt[..., None] * ws).abs().sum(0)
        whole = lambda x: torch.stack(x, 1)  # noqa: E731
        total = (length + batch + 32) * U      # a lane's sum over its steps, then over segments and batch
        out["u"], err["u"] = whole(val["u"]), rounded(whole(val["u"]), whole(bnd["u"]), self.dtype)
        dd, de = whole(val["dt"]), whole(bnd["dt"])
        if self.softplus:
            sg = torch.sigmoid(self.raw)
            de = sg * (de + dd.abs() * (self.raw.abs() + 12) * U)
            dd = dd * sg
        out["delta"], err["delta"] = dd, rounded(dd, de, self.dtype)
        for k in "BC":
            out[k], err[k] = whole(val[k]), rounded(whole(val[k]), whole(bnd[k]), self.dtype)
        out["A"], err["A"] = dA, dAe + total * dAs + t32
        out["D"] = (a * self.u).sum((0, 1))
        err["D"] = ((rel + total + 2 * U) * (a * self.u).abs()).sum((0, 1)) + t32
        out["bias"], err["bias"] = dd.sum((0, 1)), (de + total * dd.abs()).sum((0, 1)) + t32
        out["h0"], err["h0"] = mu, md + t32
        return out, err


# ------------------------------------------------------- log probabilities ----

def logprob64(x, tokens, scale, top):
    """(logp, lse, entropy, ids, top_logp) and the bounds of the first three and the last."""
    y = x.double() * scale
    m = y.amax(1, keepdim=True)
    lse = torch.logsumexp(y, 1, keepdim=True)
    lp = y - lse
    p = torch.exp(lp)
    some = p > 0
    entropy = -torch.where(some, p * lp, 0.0).sum(1)
    # every term is off by its exponent's size (1.5 U of it, and the difference before it), the sum by
    # its depth: 64 elements of a lane, then a tree over lanes, waves and chunks
    reach = torch.where(some, y - m, 0.0)
    depth = 64 + 6 + 4 + 6 + 8
    rel = (p * (3 * reach.abs() + depth)).sum(1) * U
    lse_err = rel + 4 * U * (m[:, 0].abs() + torch.log(torch.exp(reach).sum(1)).abs() + 1)
    width = x.shape[1]
    inner = (p * reach.abs() * (3 * reach.abs() + depth + 6)).sum(1) * U
    ent_err = rel + inner + (p * reach.abs()).sum(1) * rel + 4 * U * (entropy.abs() + (p * reach.abs()).sum(1) + 1) + width * 1e-36
    good = (tokens >= 0) & (tokens < width)
    at = torch.where(good, tokens, 0)[:, None]
    given = lp.gather(1, at)[:, 0]
    logp = torch.where(good, given, 0.0)
    logp_err = torch.where(good, lse_err + 2 * U * (y.gather(1, at)[:, 0].abs() + lse[:, 0].abs()), 0.0)
    ids = torch.sort(x.double(), dim=1, descending=True, stable=True).indices[:, :top]
    top_lp = lp.gather(1, ids)
    top_err = lse_err[:, None] + 2 * U * (y.gather(1, ids).abs() + lse.abs())
    return (logp, lse[:, 0], entropy, ids, top_lp), (logp_err, lse_err, ent_err, top_err)


def logprob_adjoint64(x, tokens, lse, entropy, gl, ge, scale):
    """The gradient at the given statistics, and its bound."""
    lp = x.double() * scale - lse.double()[:, None]
    p = torch.exp(lp)
    good = (tokens >= 0) & (tokens < x.shape[1])
    gl = torch.where(good, gl.double(), 0.0)[:, None] if gl is not None else torch.zeros_like(lp[:, :1])
    inner = gl.expand_as(lp)
    size = gl.abs().expand_as(lp)
    clean = torch.where(p > 0, lp, 0.0)
    # log p is one rounded sum, U of it; the exponential's argument has that error and its own product's
    rel = (U * clean.abs() * 4 + 4 * U)
    if ge is not None:
        ge, H = ge.double()[:, None], entropy.double()[:, None]
        inner = inner + ge * (clean + H)
        size = size + ge.abs() * (clean.abs() + H.abs())
    d = -p * inner
    err = p * size * (rel + 6 * U)
    hot = torch.zeros_like(d)
    hot[torch.arange(len(tokens), device=x.device)[good], tokens[good]] = 1.0
    d = (d + hot * gl) * scale
    err = (err + 2 * U * hot * gl.abs()) * scale + 2 * U * d.abs()
    return d, rounded(d, err, x.dtype)
