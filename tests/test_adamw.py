"""chol_adamw against 64 bits, on the GPU."""
import math

import pytest

import train_util as tu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
E4M3 = torch.float8_e4m3fn
TILE = 256
HYPER = dict(step=7, lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)
SIZES = [1, 255, 256, 257, 4096, 4097, 3, 10000, 1024, 5]


def mix(x):
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B1) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0x85EBCA77) & 0xFFFFFFFF
    return x ^ (x >> 16)


def noise(first, n, seed):
    x = mix((torch.arange(n, dtype=torch.int64) + first + int(mix(torch.tensor(seed)))) & 0xFFFFFFFF)
    return x & 0xFFFF, x >> 16


def make(dtype, master, bits, seed=0, sizes=SIZES):
    g = torch.Generator().manual_seed(seed)
    rand = lambda n, s: s * torch.randn(n, generator=g)  # noqa: E731
    t = {"master": [rand(n, 0.1) for n in sizes], "g": [rand(n, 1e-2).to(dtype) for n in sizes]}
    t["p"] = [w.to(dtype) for w in t["master"]]
    if bits == 32:
        t["m"], t["v"] = [rand(n, 1e-2) for n in sizes], [rand(n, 1e-2).square() for n in sizes]
    else:
        code = lambda n: torch.randint(0, 0x78, (n,), generator=g, dtype=torch.uint8)  # noqa: E731  (up to 256)
        t["m"] = [(code(n) | (torch.randint(0, 2, (n,), generator=g, dtype=torch.uint8) << 7)).view(E4M3) for n in sizes]
        t["v"] = [code(n).view(E4M3) for n in sizes]
        for k, e in (("m_scale", -14), ("v_scale", -13)):
            t[k] = [torch.full((-(-n // TILE),), 2.0 ** e) for n in sizes]
    if not master:
        del t["master"]
    return t


def on_gpu(t):
    """Every tensor as a slice of a larger one whose other elements have to stay as they are."""
    out, walls = {}, []
    for k, tensors in t.items():
        out[k] = []
        for x in tensors:
            raw = torch.full((x.numel() + 7,), 0x55, dtype=torch.uint8).view(torch.uint8) if x.dtype == E4M3 else \
                torch.full((x.numel() + 7,), 5.0, dtype=x.dtype)
            raw = raw.cuda()
            mid = raw[3:3 + x.numel()]
            mid.copy_(x.view(torch.uint8) if x.dtype == E4M3 else x)
            walls.append((raw, x.numel(), raw[0].item()))
            out[k].append(mid.view(E4M3) if x.dtype == E4M3 else mid)
    return out, walls


def check(before, after, master, bits, clip, seed, firsts, hyper=HYPER):
    k = hyper
    for i, n in enumerate(x.numel() for x in before["p"]):
        w = (before["master"] if master else before["p"])[i].double()
        g = before["g"][i].double() * clip
        if bits == 32:
            m0, v0 = before["m"][i].double(), before["v"][i].double()
        else:
            wide = lambda s: s.double().repeat_interleave(TILE)[:n]  # noqa: E731
            m0 = before["m"][i].double() * wide(before["m_scale"][i])
            v0 = (before["v"][i].double() * wide(before["v_scale"][i])).square()
        m = k["beta1"] * m0 + (1 - k["beta1"]) * g
        v = k["beta2"] * v0 + (1 - k["beta2"]) * g * g
        m_size = k["beta1"] * m0.abs() + (1 - k["beta1"]) * g.abs()
        den = (v / (1 - k["beta2"] ** k["step"])).sqrt() + k["eps"]
        rate = k["lr"] / (1 - k["beta1"] ** k["step"])
        new = w * (1 - k["lr"] * k["weight_decay"]) - rate * m / den
        # m: two constants, three products and a sum; v: 6; the root halves v's; den, quotient and products: 8
        bound = 4 * tu.U * w.abs() + (8 + 6 + 8) * tu.U * rate * m_size / den + tu.U * new.abs()
        if master:
            tu.near(after["master"][i].cpu(), new, bound, f"master[{i}]")
            assert torch.equal(after["p"][i], after["master"][i].to(after["p"][i].dtype))
        half = tu.HALF[before["p"][i].dtype]
        tu.near(after["p"][i].cpu(), new, bound + half * (new.abs() + bound) + tu.TINY[before["p"][i].dtype], f"p[{i}]")
        if bits == 32:
            tu.near(after["m"][i].cpu(), m, 7 * tu.U * m_size + tu.TINY[torch.float32], f"m[{i}]")
            tu.near(after["v"][i].cpu(), v, 8 * tu.U * v + 2 * tu.TINY[torch.float32], f"v[{i}]")
            continue
        low, high = noise(firsts[i], n, seed)
        for name, x, size, r in (("m", m, m_size, low), ("v", v.sqrt(), v.sqrt(), high)):
            scale = after[name + "_scale"][i].cpu().double()
            most = torch.nn.functional.pad(x.abs(), (0, -n % TILE)).view(-1, TILE).amax(1)
            tiny = 2.0 ** -126
            low_s, high_s = (torch.exp2(torch.floor(torch.log2((most * f).clamp(min=tiny))) - 7).clamp(min=tiny)
                             for f in (1 - 8 * tu.U, 1 + 8 * tu.U))
            assert ((scale == low_s) | (scale == high_s)).all(), name
            y = x.abs() / wide(scale)
            step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
            place = y / step + r.double() / 65536
            # how far fp32 may put the value from x, in steps
            off = 8 * tu.U * size / wide(scale) / step + 2.0 ** -20
            got = after[name][i].cpu().double()
            assert torch.isfinite(got).all()
            steps = got.abs() / step
            fine = (steps >= torch.floor(place - off)) & (steps <= torch.floor(place + off))
            if name == "v":
                fine |= (steps == 1) & (torch.floor(place - off) <= 0) & (x > 0)
            assert fine.all(), (name, i, int((~fine).sum()))
            assert ((got == 0) | (torch.sign(got) == torch.sign(x)) | (x.abs() <= 8 * tu.U * size)).all()
            if name == "v":
                assert (got[x > 0] > 0).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_step(dtype, master, bits):
    import differentiable_cholesky_amd as dc
    before = make(dtype, master, bits)
    t, walls = on_gpu(before)
    handle = dc.chol_adamw_list(t["p"], t["g"], t["m"], t["v"], master=t.get("master"), m_scale=t.get("m_scale"),
                                v_scale=t.get("v_scale"))
    clip = torch.tensor([0.25], device="cuda")
    dc.chol_adamw(handle, grad_scale=clip, seed=123456789, **HYPER)
    firsts, at = [], 0
    for n in SIZES:
        firsts.append(at)
        at += -(-n // TILE) * TILE
    check(before, t, master, bits, 0.25, 123456789, firsts)
    for a, b in zip(before["g"], t["g"]):
        assert torch.equal(a, b.cpu())
    for raw, n, wall in walls:
        rest = torch.cat([raw[:3], raw[3 + n:]])
        assert (rest == wall).all()


def test_positions_wrap_and_no_grad_scale():
    import differentiable_cholesky_amd as dc
    sizes = [700, 300]
    before = make(torch.float32, False, 8, seed=1, sizes=sizes)
    t, _ = on_gpu(before)
    firsts = [2 ** 32 - 300, 5 * 2 ** 32 + 17]
    handle = dc.chol_adamw_list(t["p"], t["g"], t["m"], t["v"], m_scale=t["m_scale"], v_scale=t["v_scale"], first=firsts)
    dc.chol_adamw(handle, seed=0xFFFFFFFF, **HYPER)
    check(before, t, False, 8, 1.0, 0xFFFFFFFF, firsts)


@pytest.mark.parametrize("bits", [32, 8])
def test_states_of_zero_and_non_finite_gradients(bits):
    import differentiable_cholesky_amd as dc
    n = 1000
    before = make(torch.float32, False, bits, seed=2, sizes=[n])
    zero = torch.zeros(n, dtype=torch.uint8).view(E4M3) if bits == 8 else torch.zeros(n)
    before["m"], before["v"] = [zero], [zero.clone()]
    if bits == 8:
        for k in ("m_scale", "v_scale"):
            before[k] = [torch.ones(4)]
    before["g"][0][:512] = 0
    hyper = dict(HYPER, step=1)
    t, _ = on_gpu(before)
    handle = dc.chol_adamw_list(t["p"], t["g"], t["m"], t["v"], m_scale=t.get("m_scale"), v_scale=t.get("v_scale"))
    dc.chol_adamw(handle, seed=3, **hyper)
    check(before, t, False, bits, 1.0, 3, [0], hyper)
    assert not t["m"][0][:512].float().any() and not t["v"][0][:512].float().any()
    # an infinite gradient spoils its own element only
    t["g"][0][700] = float("inf")
    keep = [x.clone() for x in (t["p"][0],)]
    dc.chol_adamw(handle, seed=4, **hyper)
    p = t["p"][0]
    assert not torch.isfinite(p[700]) and torch.isfinite(torch.cat([p[:700], p[701:]])).all()
    assert not torch.equal(p[513:700], keep[0][513:700])


@pytest.mark.parametrize("bits", [32, 8])
def test_second_moments_of_every_size(bits):
    """Roots of values far from one, in tiles of their own and beside ordinary ones."""
    import differentiable_cholesky_amd as dc
    n = 4096
    before = make(torch.float32, False, bits, seed=7, sizes=[n])
    before["g"][0].zero_()
    g = torch.Generator().manual_seed(8)
    place = torch.rand(n // TILE, 1, generator=g) * 2 - 1 + torch.zeros(1, TILE)
    place[::3] = torch.rand(place[::3].shape, generator=g) * 2 - 1
    if bits == 32:
        before["v"] = [torch.pow(10.0, 36 * place.double()).float().view(-1)]
        before["m"] = [(before["v"][0].double().sqrt() * torch.randn(n, generator=g).double()).float()]
    else:
        for k in ("m_scale", "v_scale"):
            before[k] = [torch.exp2(torch.round(48 * place[:, 0]))]
    hyper = dict(HYPER, eps=0.0)
    if bits == 8:
        before["v"] = [torch.clamp(before["v"][0].view(torch.uint8), min=1).view(E4M3)]
    t, _ = on_gpu(before)
    handle = dc.chol_adamw_list(t["p"], t["g"], t["m"], t["v"], m_scale=t.get("m_scale"), v_scale=t.get("v_scale"))
    dc.chol_adamw(handle, seed=11, **hyper)
    check(before, t, False, bits, 1.0, 11, [0], hyper)


def test_eight_bit_states_are_unbiased():
    """The mean over seeds of a stored state is the state: no more than 6 standard deviations of a step's rounding off."""
    import differentiable_cholesky_amd as dc
    n, runs = 4096, 200
    g = torch.Generator().manual_seed(5)
    grad = torch.randn(n, generator=g)
    sums = torch.zeros(2, n, dtype=torch.float64)
    hyper = dict(HYPER, beta1=0.0, beta2=0.0)
    for seed in range(runs):
        z = lambda: torch.zeros(n, dtype=torch.uint8, device="cuda").view(E4M3)  # noqa: E731
        s = lambda: torch.ones(n // TILE, device="cuda")  # noqa: E731
        p, gr, m, v, ms, vs = torch.zeros(n, device="cuda"), grad.cuda(), z(), z(), s(), s()
        dc.chol_adamw(dc.chol_adamw_list([p], [gr], [m], [v], m_scale=[ms], v_scale=[vs]), seed=seed, **hyper)
        for k, (c, sc) in enumerate(((m, ms), (v, vs))):
            sums[k] += (c.float().view(-1, TILE) * sc[:, None]).view(-1).cpu().double()
    for k, want in enumerate((grad.double(), grad.double().abs())):
        step = want.abs() / 8 + grad.abs().view(-1, TILE).amax(1).repeat_interleave(TILE).double() * 2.0 ** -16
        # a root below the smallest code is stored as that code
        some = want.abs() > 4 * 2.0 ** -9 * 2.0 ** -7 * grad.abs().view(-1, TILE).amax(1).repeat_interleave(TILE).double()
        some |= torch.tensor(k == 0)
        assert ((sums[k] / runs - want).abs() <= 6 * step / 2 / math.sqrt(runs) + step * 2.0 ** -15)[some].all()


def test_captured_into_a_graph():
    import differentiable_cholesky_amd as dc
    before = make(torch.bfloat16, True, 8, seed=6)
    (a, _), (b, _) = on_gpu(before), on_gpu(before)
    lists = [dc.chol_adamw_list(t["p"], t["g"], t["m"], t["v"], master=t["master"], m_scale=t["m_scale"],
                                v_scale=t["v_scale"]) for t in (a, b)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dc.chol_adamw(lists[0], seed=9, **HYPER)
    for _ in range(4):
        for t in (a, b):
            for x in t["g"]:
                x.mul_(0.5)
        graph.replay()
        dc.chol_adamw(lists[1], seed=9, **HYPER)
        torch.cuda.synchronize()
        for k in a:
            for x, y in zip(a[k], b[k]):
                assert torch.equal(x.float(), y.float()), k


def test_a_list_longer_than_one_launch_takes():
    """2^21 chunks of 4096 weights and a few more: the last ones are stepped as a list of their own is."""
    import differentiable_cholesky_amd as dc
    big, tail = (1 << 21) * 4096, 5000
    dev = dict(device="cuda")
    p, g = (torch.zeros(big + tail, dtype=torch.bfloat16, **dev) for _ in range(2))
    m, v = (torch.zeros(big + tail, dtype=torch.uint8, **dev).view(E4M3) for _ in range(2))
    scales = [torch.ones(-(-(big + tail) // TILE), **dev) for _ in range(2)]
    p[big:].normal_()
    g[big:].normal_()
    own = [t[big:].clone() for t in (p, g)] + [torch.zeros(tail, dtype=torch.uint8, **dev).view(E4M3) for _ in range(2)]
    own_scales = [torch.ones(-(-tail // TILE), **dev) for _ in range(2)]
    dc.chol_adamw(dc.chol_adamw_list([p], [g], [m], [v], m_scale=[scales[0]], v_scale=[scales[1]]), seed=5, **HYPER)
    dc.chol_adamw(dc.chol_adamw_list([own[0]], [own[1]], [own[2]], [own[3]], m_scale=[own_scales[0]],
                                     v_scale=[own_scales[1]], first=[big]), seed=5, **HYPER)
    assert not torch.equal(own[0], torch.zeros_like(own[0])) and torch.equal(p[big:], own[0])
    for x, y in ((m, own[2]), (v, own[3])):
        assert torch.equal(x[big:].view(torch.uint8), y.view(torch.uint8))
    for x, y in zip(scales, own_scales):
        assert torch.equal(x[big // TILE:], y)
    assert not p[big - 100000:big].any()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_non_finite_gradient_stays_in_its_element(bad, bits):
    """Steps after it: every other weight and state is what it is where that element's gradient is zero, which adds
    nothing to its tile; a tile of non-finite elements only, and one at the ragged end, among them."""
    import differentiable_cholesky_amd as dc
    n, hit = 1000, torch.zeros(1000, dtype=torch.bool)
    hit[[3, 700, 999]] = True
    hit[256:512] = True
    before = make(torch.float32, False, bits, seed=9, sizes=[n])
    for k in ("m", "v"):
        raw = before[k][0].view(torch.uint8) if bits == 8 else before[k][0]
        raw[hit] = 0
    runs = []
    for value in (0.0, bad):
        t, _ = on_gpu(before)
        handle = dc.chol_adamw_list(t["p"], t["g"], t["m"], t["v"], m_scale=t.get("m_scale"), v_scale=t.get("v_scale"))
        g = torch.Generator().manual_seed(10)
        for step in range(1, 7):
            grad = 1e-2 * torch.randn(n, generator=g)
            grad[hit] = value if step == 2 else 0.0
            t["g"][0].copy_(grad)
            dc.chol_adamw(handle, seed=step, **dict(HYPER, step=step))
        runs.append(t)
    rest = ~hit.cuda()
    for k in ("p", "m", "v"):
        x, y = (t[k][0].float() for t in runs)
        assert torch.isfinite(x).all() and torch.equal(y[rest], x[rest]), k
        assert not torch.isfinite(y[~rest]).any(), k
    if bits == 8:
        for k in ("m_scale", "v_scale"):
            assert torch.equal(runs[0][k][0], runs[1][k][0]), k


def test_a_negative_second_moment_has_no_root():
    """A state that no step writes: its weight is NaN, not silently stepped; zeros of either sign are zero."""
    import differentiable_cholesky_amd as dc
    n = 600
    before = make(torch.float32, False, 32, seed=14, sizes=[n])
    before["g"][0].zero_()
    v = before["v"][0]
    bad = torch.zeros(n, dtype=torch.bool)
    bad[[0, 5, 300, 599]] = True
    v[bad] = -torch.tensor([1e-6, 1.0, 1e-30, float("inf")])
    v[[7, 8]] = torch.tensor([0.0, -0.0])
    t, _ = on_gpu(before)
    dc.chol_adamw(dc.chol_adamw_list(t["p"], t["g"], t["m"], t["v"]), **dict(HYPER, eps=1e-3))
    p = t["p"][0].cpu()
    assert torch.isnan(p[bad]).all() and torch.isfinite(p[~bad]).all()
