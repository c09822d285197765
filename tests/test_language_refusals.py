"""What the binding of the convolution, the scan and the token log probabilities refuses, each argument by itself and by
its name: on the CPU in place of the GPU, where a call that passes the checks ends at a stand-in for the library; on the
GPU with the library itself."""
import contextlib

import pytest

dc = pytest.importorskip("differentiable_cholesky_amd")
torch = pytest.importorskip("torch")
from differentiable_cholesky_amd import _language  # noqa: E402

F32, I64 = torch.float32, torch.int64
BATCH, LENGTH, DIM, WIDTH, GROUPS, STATES, ROWS, VOCAB, TOP = 2, 3, 4, 3, 2, 5, 6, 7, 2
SEQ, KEPT, STATE = (BATCH, LENGTH, DIM), (BATCH, WIDTH - 1, DIM), (BATCH, DIM, STATES)
MIXED, RATE, STARTS = (BATCH, LENGTH, GROUPS, STATES), (DIM, STATES), (BATCH, 1, DIM, STATES)

# (shape, type; None: the call's) of every tensor argument; the first one is what the others are measured by
CALLS = {
    "chol_causal_conv": dict(x=(SEQ, None), w=((DIM, WIDTH), None), bias=((DIM,), None), state=(KEPT, None), last=(KEPT, None),
                             y=(SEQ, None)),
    "chol_causal_conv_adjoint": dict(x=(SEQ, None), w=((DIM, WIDTH), None), adj=(SEQ, None), bias=((DIM,), None),
                                     state=(KEPT, None), adjLast=(KEPT, None), adjX=(SEQ, None), adjW=((DIM, WIDTH), F32),
                                     adjBias=((DIM,), F32), adjState=(KEPT, None)),
    "chol_selective_scan": dict(u=(SEQ, None), delta=(SEQ, None), A=(RATE, F32), B=(MIXED, None), C=(MIXED, None),
                                D=((DIM,), F32), z=(SEQ, None), bias=((DIM,), F32), h0=(STATE, F32), hlast=(STATE, F32),
                                y=(SEQ, None), starts=(STARTS, F32)),
    "chol_selective_scan_adjoint": dict(u=(SEQ, None), delta=(SEQ, None), A=(RATE, F32), B=(MIXED, None), C=(MIXED, None),
                                        starts=(STARTS, F32), adj=(SEQ, None), D=((DIM,), F32), z=(SEQ, None),
                                        bias=((DIM,), F32), adjHlast=(STATE, F32), adjU=(SEQ, None), adjDelta=(SEQ, None),
                                        adjA=(RATE, F32), adjB=(MIXED, None), adjC=(MIXED, None), adjD=((DIM,), F32),
                                        adjZ=(SEQ, None), adjBias=((DIM,), F32), adjH0=(STATE, F32)),
    "chol_token_logprob": dict(logits=((ROWS, VOCAB), None), tokens=((ROWS,), I64)),
    "chol_token_logprob_adjoint": dict(logits=((ROWS, VOCAB), None), tokens=((ROWS,), I64), lse=((ROWS,), F32),
                                       adjLogp=((ROWS,), F32), entropy=((ROWS,), F32), adjEntropy=((ROWS,), F32),
                                       adjLogits=((ROWS, VOCAB), None)),
}
WORKSPACES = ("chol_causal_conv_adjoint", "chol_selective_scan_adjoint")
# arguments that give the call a size: a change of theirs may make it another valid one, for which these are wrong
SIZED_BY = {"w": "state", "A": "B", "B": "C|.* groups do not divide"}
ARGUMENTS = [(call, name) for call, given in CALLS.items() for name in list(given)[1:]]


class Reached(Exception):
    pass


@pytest.fixture(params=["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def device(request, monkeypatch):
    if request.param == "cpu":
        def reached(*_):
            raise Reached
        monkeypatch.setattr(_language, "_on", lambda t, stream: contextlib.nullcontext())
        monkeypatch.setattr(_language, "_raw_stream", lambda t: 0)
        for call in CALLS:
            monkeypatch.setattr(_language.lib, call, reached)
    return request.param


def given(call, device, kind=torch.bfloat16):
    return {name: torch.zeros(shape, dtype=dtype or kind, device=device) for name, (shape, dtype) in CALLS[call].items()}


def run(call, args, **more):
    return getattr(dc, call)(**args, **more)


@pytest.mark.parametrize("call", CALLS)
def test_what_is_right_passes(call, device):
    args = given(call, device)
    if device == "cpu":
        with pytest.raises(Reached):
            run(call, args)
    else:
        run(call, args)


@pytest.mark.parametrize("call,name", ARGUMENTS)
def test_shapes(call, name, device):
    args = given(call, device)
    shape = args[name].shape
    # one more in any place, one less, and another number of axes
    wrong = [shape[:k] + (shape[k] + 1,) + shape[k + 1:] for k in range(len(shape))]
    wrong += [shape[:-1] + (shape[-1] - 1,), shape + (1,)]
    for other in wrong:
        with pytest.raises(ValueError, match=rf"^({name}|{SIZED_BY.get(name, name)})\b"):
            run(call, {**args, name: torch.zeros(other, dtype=args[name].dtype, device=device)})


@pytest.mark.parametrize("call,name", ARGUMENTS)
def test_types(call, name, device):
    args = given(call, device)
    for other in (torch.float16, torch.float64, torch.int32):
        with pytest.raises(TypeError, match=rf"^({name}|{SIZED_BY.get(name, name)})\b"):
            run(call, {**args, name: args[name].to(other)})


@pytest.mark.parametrize("call,name", ARGUMENTS)
def test_layouts(call, name, device):
    """Elements of the last axis two apart, or (one axis) every second."""
    args = given(call, device)
    t = args[name]
    wide = torch.zeros(t.shape[:-1] + (2 * t.shape[-1],), dtype=t.dtype, device=device)
    with pytest.raises(ValueError, match=rf"\b{name}\b"):
        run(call, {**args, name: wide[..., ::2]})


@pytest.mark.parametrize("call", CALLS)
def test_the_first_argument(call, device):
    args = given(call, device)
    name = next(iter(args))
    x = args[name]
    with pytest.raises(ValueError, match=rf"\b{name}\b"):
        run(call, {**args, name: x[0]})
    with pytest.raises(TypeError, match="expected float32"):
        run(call, {**args, name: x.double()})
    with pytest.raises(ValueError, match=rf"\b{name}\b"):
        run(call, {**args, name: torch.cat([x, x], -1)[..., ::2]})


@pytest.mark.gpu
@pytest.mark.parametrize("call,name", [(call, name) for call, of in CALLS.items() for name in of])
def test_other_devices(call, name):
    args = given(call, "cuda")
    with pytest.raises(ValueError, match=r"GPU|must live on"):
        run(call, {**args, name: args[name].cpu()})


@pytest.mark.parametrize("call", WORKSPACES)
def test_workspaces(call, device):
    args = given(call, device)
    whole = torch.zeros(1 << 16, dtype=torch.uint8, device=device)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        run(call, args, workspace=whole[::2])
    with pytest.raises(ValueError, match="workspace must live on"):
        run(call, args, workspace=torch.zeros(1 << 16, dtype=torch.uint8, device="meta"))
    if device == "cuda":
        with pytest.raises(dc.CholError):
            run(call, args, workspace=whole[:16])
        with pytest.raises(dc.CholError):
            run(call, args, workspace=whole[2:])


def test_values(device):
    args = given("chol_token_logprob", device)
    for top in (-1, VOCAB + 1, 33):
        with pytest.raises(ValueError, match="top must be"):
            run("chol_token_logprob", args, top=top)
    args = given("chol_token_logprob_adjoint", device)
    with pytest.raises(ValueError, match="adjEntropy needs entropy"):
        run("chol_token_logprob_adjoint", {**args, "entropy": None})
    args = given("chol_selective_scan_adjoint", device)
    with pytest.raises(ValueError, match="adjZ needs z"):
        run("chol_selective_scan_adjoint", {**args, "z": None})
    args = given("chol_causal_conv", device)
    for width in (1, 5):
        with pytest.raises(ValueError, match="w must be"):
            run("chol_causal_conv", {**args, "w": torch.zeros(DIM, width, dtype=torch.bfloat16, device=device)})
    args = given("chol_selective_scan", device)
    for states in (0, 65):
        with pytest.raises(ValueError, match="A must have"):
            run("chol_selective_scan", {**args, "A": torch.zeros(DIM, states, device=device)})
    with pytest.raises(ValueError, match="groups do not divide"):
        three = torch.zeros(BATCH, LENGTH, 3, STATES, dtype=torch.bfloat16, device=device)
        run("chol_selective_scan", {**args, "B": three, "C": three})
