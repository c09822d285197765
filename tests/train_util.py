"""Plain 64-bit implementations of the training-step operators, and bounds on
how far a kernel that computes in fp32 and rounds its outputs once may be off.

A rounding to type t is off by at most HALF[t] relative to the value.
"""
import torch

HALF = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
# values below a type's normal range are off by up to half its smallest step
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
U = HALF[torch.float32]


def recurrence64(a, b, h0, gate):
    """(h, hlast, size): the recurrence in 64 bits and the same recurrence on
    absolute values, which bounds what roundings of the terms add up to."""
    a, b = a.double(), b.double()
    a = a.exp() if gate == "log" else a
    x = torch.zeros_like(a[:, 0] if a.shape[1] else b.sum(1)) if h0 is None else h0.double()
    s = x.abs()
    h, size = torch.empty_like(b), torch.empty_like(b)
    for t in range(a.shape[1]):
        x = a[:, t] * x + b[:, t]
        s = a[:, t].abs() * s + b[:, t].abs()
        h[:, t], size[:, t] = x, s
    return h, x, size, s


def recurrence_adjoint64(a, h, adj, h0, adj_last, gate):
    """(adjA, adjB, adjH0) and the same on absolute values."""
    a, h, adj = a.double(), h.double(), adj.double()
    a = a.exp() if gate == "log" else a
    first = torch.zeros(a.shape[0], a.shape[2], dtype=torch.float64, device=a.device)
    mu = first.clone() if adj_last is None else adj_last.double()
    ms = mu.abs()
    before0 = first if h0 is None else h0.double()
    adj_a, adj_b, sa, sb = (torch.empty_like(a) for _ in range(4))
    for t in range(a.shape[1] - 1, -1, -1):
        lam, ls = adj[:, t] + mu, adj[:, t].abs() + ms
        before = h[:, t - 1] if t else before0
        mu, ms = a[:, t] * lam, a[:, t].abs() * ls
        adj_b[:, t], sb[:, t] = lam, ls
        adj_a[:, t] = (mu if gate == "log" else lam) * before
        sa[:, t] = (ms if gate == "log" else ls) * before.abs()
    return (adj_a, adj_b, mu), (sa, sb, ms)


def steps_u(length, gate):
    """Relative error of a state per unit of the absolute-value recurrence: a
    value passes through at most `length` steps of one product and one sum, twice
    where a run is composed first and applied after (products of gates included),
    plus 2 roundings of each exponential (taken as 4)."""
    return (4 * length + 8 + (4 * length if gate == "log" else 0)) * U


def near(got, ref, bound, what):
    """|got - ref| <= bound elementwise; the first entry outside is named."""
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    err = (got - ref).abs()
    bad = err > bound
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds; first at {i}: got {got[i].item()!r} "
                             f"ref {ref[i].item()!r} bound {bound[i].item()!r}")
