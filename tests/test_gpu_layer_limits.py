"""GPU: the operators around the experts where a call takes more than one launch,
in place, and where the squares of a row leave fp32.

A token's or row's values come from its own wave or workgroup alone, so a large
call's must have the bits of a small one of the same kernel."""
import numpy as np
import pytest
import torch

from fp4_quantized_moe_amd import _lib as Q

pytestmark = pytest.mark.gpu
bf = torch.bfloat16
U = 2.0 ** -24
GROUPS = 1 << 23  # workgroups of a launch


def seeded(n):
    return torch.Generator(device="cuda").manual_seed(n)


# rows of a workgroup, columns: 16 lanes, a wave and a workgroup a row
@pytest.mark.parametrize("per, cols", [(16, 16), (4, 144), (1, 1040)])
def test_norm_of_more_rows_than_a_launch(per, cols):
    edge = GROUPS * per
    x = torch.zeros(edge + 2501, cols, dtype=bf, device="cuda")
    x[edge - 2500:] = torch.randn(5001, cols, generator=seeded(1), device="cuda").to(bf)
    w = (1 + 0.2 * torch.randn(cols, generator=seeded(2), device="cuda")).to(bf)
    got = Q.rms_norm(x, w, keep=True)
    want = Q.rms_norm(x[edge - 2500:].clone(), w, keep=True)
    assert torch.equal(got.y[edge - 2500:], want.y) and torch.equal(got.rstd[edge - 2500:], want.rstd)
    assert (got.rstd[:edge - 2500] == got.rstd[0]).all() and not got.y[:edge - 2500].any()


def test_router_of_more_tokens_than_a_launch():
    edge, E = GROUPS * 16, 3
    T = edge + 77
    logits = torch.zeros(T, E, device="cuda")
    logits[edge - 500:] = torch.randn(577, E, generator=seeded(3), device="cuda")
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    ids[edge - 500:] = 2
    dw = torch.full((T, 1), 0.5, device="cuda")
    got = Q.moe_route_backward(logits, ids, dw=dw)
    tail = Q.moe_route_backward(*(t[edge - 500:].clone() for t in (logits, ids)), dw=dw[edge - 500:].clone())
    assert torch.equal(got[edge - 500:], tail) and (got[:edge - 500] == got[0]).all() and got[0, 0] > 0 > got[0, 1]
    b = Q.moe_balance_loss(logits, ids, 1.0)
    assert b.counts.tolist() == [edge - 500, 0, 577]
    p = torch.softmax(logits[edge - 500:].double(), 1).sum(0).cpu().numpy() + (edge - 500) / 3
    want = E * (np.array([edge - 500, 0, 577]) / T * p / T).sum()
    # a lane adds T / (128 * 64) terms, each off by 16 u (softmax); 64 lanes and 128 workgroups follow
    assert abs(b.loss.item() - want) <= (T / 8192 + 16 + 64 + 128 + 8) * U * want


def test_combine_of_more_tokens_than_a_launch():
    edge = GROUPS * 4
    T = edge + 33
    dout = torch.zeros(T, 16, dtype=bf, device="cuda")
    dout[edge - 100:] = torch.randn(133, 16, generator=seeded(4), device="cuda").to(bf)
    inverse = torch.arange(T, dtype=torch.int32, device="cuda").view(T, 1)
    w = torch.rand(T, 1, generator=seeded(5), device="cuda")
    dy, dw = Q.moe_combine_backward(dout, dout, inverse, w)  # y is dout: dw its square
    assert torch.equal(dy[edge - 100:], (w[edge - 100:] * dout[edge - 100:].float()).to(bf)) and not dy[:edge - 100].any()
    want = dout[edge - 100:].double().square().sum(1)
    assert ((dw[edge - 100:, 0].double() - want).abs() <= 18 * U * want).all() and not dw[:edge - 100].any()


@pytest.mark.parametrize("rows", [4, 3000])
def test_norm_of_rows_whose_squares_leave_fp32(rows):
    x = torch.ones(rows, 64, device="cuda")
    x[1], x[2] = 1e25, 1e-30
    x[3, 5] = float("inf")
    w = torch.ones(64, dtype=bf, device="cuda")
    r = Q.rms_norm(x, w, keep=True, eps=0.0)
    assert r.rstd[1] == 0 and (r.y[1] == 0).all()                                  # mean(s^2) = inf
    assert r.rstd[2] == float("inf") and (r.y[2] == float("inf")).all()            # mean(s^2) = 0
    assert r.rstd[3] == 0 and r.y[3, 5].isnan() and (r.y[3, 6:] == 0).all()
    assert (r.y[0] == 1).all() and (r.y[4:] == 1).all()
    assert (Q.rms_norm(x, w).y[2] == torch.tensor(1e-30 * 1e3, device="cuda").to(bf)).all()  # eps = 1e-6 alone


@pytest.mark.parametrize("batch, rows, cols", [(3, 144, 208), (2, 208, 144), (150, 1024, 2048), (3, 32, 96), (300, 96, 32), (3, 48, 2000), (400, 1296, 32)])
def test_orthogonalize_in_place(batch, rows, cols):
    """out may be g, also where the batch takes two passes."""
    g = torch.randn(batch, rows, cols, generator=seeded(6), device="cuda").to(bf)
    want = Q.orthogonalize(g, steps=2)
    assert Q.orthogonalize(g, steps=2, out=g) is g and torch.equal(g, want)


@pytest.mark.parametrize("batch, rows, cols", [(4, 272, 528), (1, 1024, 1040), (5, 64, 96), (300, 96, 64), (5, 32, 2048), (2, 1040, 128)])
def test_orthogonalize_in_graphs_that_share_a_workspace(batch, rows, cols):
    """Two captured calls with one workspace, replayed in turn, and again with other values in the captured inputs."""
    gs = [torch.randn(batch, rows, cols, generator=seeded(10 + i), device="cuda") for i in range(2)]
    outs = [torch.empty(batch, rows, cols, dtype=bf, device="cuda") for _ in gs]
    ws = torch.empty(max(Q.orthogonalize_workspace_bytes(batch, rows, cols), 16), dtype=torch.uint8, device="cuda")
    want = [Q.orthogonalize(g) for g in gs]
    torch.cuda.synchronize()
    graphs = []
    for g, out in zip(gs, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            Q.orthogonalize(g, out=out, ws=ws)
        graphs.append(graph)
    for _ in range(3):
        for out in outs:
            out.fill_(3)
        ws.random_(0, 256)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    gs[0].copy_(gs[1])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[1])


def test_small_and_long_matrices_on_two_streams():
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    gs = [torch.randn(*shape, generator=seeded(20 + i), device="cuda") for i, shape in enumerate(((700, 48, 160), (90, 64, 2048)))]
    want = [Q.orthogonalize(g) for g in gs]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for g, s in zip(gs, sides):
            with torch.cuda.stream(s):
                got.append(Q.orthogonalize(g))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_orthogonalize_in_slabs_and_passes():
    """A batch whose slabs take two passes of the workspace: zeros but for matrices on both sides of the passes' edge."""
    batch, rows, cols = 9000, 32, 2048
    g = torch.zeros(batch, rows, cols, dtype=bf, device="cuda")
    at = [0, 4499, 4500, 4501, batch - 1]
    g[at] = torch.randn(len(at), rows, cols, generator=seeded(30), device="cuda").to(bf)
    assert Q.orthogonalize_workspace_bytes(batch, rows, cols) < 2.7e9 < 2 * Q.orthogonalize_workspace_bytes(batch, rows, cols)
    got = Q.orthogonalize(g)
    assert torch.equal(got[at], Q.orthogonalize(g[at]))
    got[at] = 0
    assert not got.any()
