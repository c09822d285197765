"""What orders the workgroups of a recurrence's chain: the protocol run on the host
(link_order.cpp), and calls that replace the state in place on the GPU."""
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")
HERE = os.path.dirname(os.path.abspath(__file__))


def test_the_start_is_read_before_the_end_is_written(tmp_path):
    from differentiable_cholesky_amd import build
    out = str(tmp_path / "link_order")
    subprocess.run([build.HIPCC, "-x", "hip", "--offload-host-only", "--offload-arch=gfx950", "-O1", "-std=c++17",
                    os.path.join(HERE, "link_order.cpp"), "-o", out], check=True)
    r = subprocess.run([out], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ordered\n", r.stdout


def make(batch, length, dim, dtype, gate, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = torch.exp(torch.randn(batch, length, dim, generator=g, device="cuda") - 4.0)
    a = (-r if gate == "log" else torch.exp(-r)).to(dtype)
    b, adj = (torch.randn(batch, length, dim, generator=g, device="cuda").to(dtype) for _ in range(2))
    return a, b, adj, *(torch.randn(batch, dim, generator=g, device="cuda") for _ in range(2))


# 256 steps a workgroup forward and 160 in the adjoint (8 waves of 32 and of 20): 2, 3, 8, 9 and 17 workgroups
# forward and more in the adjoint, then the adjoint's 8, 9 and 16; one chain, and many
@pytest.mark.gpu
@pytest.mark.parametrize("dtype,gate", [(torch.bfloat16, "log"), (torch.float32, "linear")])
@pytest.mark.parametrize("batch,dim", [(1, 64), (2, 2048), (8, 700)])
@pytest.mark.parametrize("length", [300, 700, 2048, 2100, 4300, 1280, 1300, 2560])
def test_a_state_replaced_in_place(length, batch, dim, dtype, gate):
    import differentiable_cholesky_amd as dc
    a, b, adj, h0, adj_last = make(batch, length, dim, dtype, gate, length + dim)
    h, last = dc.chol_recurrence(a, b, h0=h0, gate=gate)
    grads = dc.chol_recurrence_adjoint(a, h, adj, h0=h0, adjHlast=adj_last, gate=gate)
    for k in range(10):
        s = h0.clone()
        got, _ = dc.chol_recurrence(a, b, h0=s, hlast=s, gate=gate)
        assert torch.equal(got, h) and torch.equal(s, last), k
        d = adj_last.clone()
        da, db, _ = dc.chol_recurrence_adjoint(a, h, adj, h0=h0, adjHlast=d, adjH0=d, gate=gate)
        for x, y in zip((da, db, d), grads):
            assert torch.equal(x, y), k


@pytest.mark.gpu
@pytest.mark.parametrize("length", [1, 1500])
def test_a_kept_state_captured_into_a_graph(length):
    """Each replay carries the state on, one step or a longer piece at a time, as eager calls do."""
    import differentiable_cholesky_amd as dc
    a, b, _, h0, _ = make(4, length, 300, torch.bfloat16, "log", 21)
    s, t = h0.clone(), h0.clone()
    dc.chol_recurrence(a, b, h0=h0, gate="log")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, _ = dc.chol_recurrence(a, b, h0=s, hlast=s, gate="log")
    for k in range(5):
        graph.replay()
        want, _ = dc.chol_recurrence(a, b, h0=t, hlast=t, gate="log")
        torch.cuda.synchronize()
        assert torch.equal(h, want) and torch.equal(s, t), k
        b.mul_(-0.5)
