"""The trainer's gated block (bf16) and its backward on the GPU against the
64-bit oracle.

Tolerances.  bf16 products are exact in fp32, so a sum of K products is off by
at most K 2^-24 sum |w x| to first order; sigmoid and silu are a few fp32 ulp
(2^-21 here); every output is rounded once to bf16 (half a step: 2^-8 of the
value, 2^-134 among the subnormals)."""
import numpy as np
import pytest
import torch

from fp4_quantized_moe_amd import _lib as Q
from oracle import mxfp4_oracle as M
from gpu_util import host

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8
TINY = 2.0 ** -133


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).cuda()


def make(seed, counts, H, I, gather=True):
    rng = np.random.default_rng(seed)
    offsets = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    R, E = int(offsets[-1]), len(counts)
    A = max(1, R // 2) if gather else R
    d = {"x": bf16(rng.standard_normal((A, H))), "w_gu": bf16(rng.standard_normal((E, 2 * I, H)) * H ** -0.5 * 2),
         "w_down": bf16(rng.standard_normal((E, H, I)) * 0.05), "dy": bf16(rng.standard_normal((R, H))),
         "offs": torch.from_numpy(offsets).cuda(), "o": offsets,
         "token": torch.from_numpy(rng.integers(0, A, R).astype(np.int32)).cuda() if gather else None}
    d["t"] = host(d["token"]) if gather else None
    return d


# rows per expert; hidden; inter: single rows, empty experts, odd sizes, whole tiles
SHAPES = [
    ([1], 16, 16), ([0, 3, 1], 48, 80), ([64], 256, 128), ([33, 0, 31, 1], 656, 272), ([17] * 9, 512, 256),
    ([130, 5, 0, 257], 384, 192), ([512, 255, 1], 512, 384), ([1024], 1024, 128), ([40] * 3, 4096, 64),
    ([20, 300], 72 * 16, 16), ([260, 3], 64, 528),
]


@pytest.mark.parametrize("counts, H, I", SHAPES)
@pytest.mark.parametrize("gather", [True, False])
def test_forward(counts, H, I, gather):
    d = make(H + I, counts, H, I, gather)
    h, gu = Q.moe_gated_forward(d["x"], d["w_gu"], d["offs"], d["token"])
    x, w = host(d["x"].double()), host(d["w_gu"].double())
    want = M.grouped(x, w, d["o"], d["t"])
    tol = H * 2.0 ** -24 * M.grouped(x, w, d["o"], d["t"], magnitude=True)
    assert (np.abs(host(gu.double()) - want) <= tol + HALF * np.abs(want) + TINY).all()
    g, u = np.split(want, 2, 1)
    tg, tu = np.split(tol, 2, 1)
    hw = M.gated(want)
    err = 1.1 * tg * (np.abs(u) + tu) + np.abs(M.silu(g)) * tu + (2.0 ** -21 + HALF) * np.abs(hw) + TINY
    assert (np.abs(host(h.double()) - hw) <= err).all()
    alone, none = Q.moe_gated_forward(d["x"], d["w_gu"], d["offs"], d["token"], keep=False)
    assert none is None and torch.equal(alone, h)


@pytest.mark.parametrize("counts, H, I", SHAPES)
def test_backward(counts, H, I):
    d = make(H + I + 1, counts, H, I)
    R = int(d["o"][-1])
    gu = bf16(np.random.default_rng(I).standard_normal((R, 2 * I)) * 2)
    dgu = Q.moe_gated_backward(d["dy"], d["w_down"], gu, d["offs"])
    dy, w = host(d["dy"].double()), host(d["w_down"].double()).transpose(0, 2, 1)
    dh = M.grouped(dy, w, d["o"])
    tol = H * 2.0 ** -24 * M.grouped(dy, w, d["o"], magnitude=True)
    pre = host(gu.double())
    g, u = np.split(pre, 2, 1)
    s = M.sigmoid(g)
    # d gate = dh u s (1 + g (1 - s)): s and 1 - s are off by 2^-21 of s and of 1
    part = np.concatenate((np.abs(u) * s * (1 + np.abs(g)), np.abs(g) * s), 1)
    want = M.gated_grad(dh, pre)
    err = np.concatenate((tol, tol), 1) * part + 2.0 ** -20 * np.concatenate((np.abs(dh), np.abs(dh)), 1) * part
    assert (np.abs(host(dgu.double()) - want) <= err + HALF * np.abs(want) + TINY).all()
    Q.moe_gated_backward(d["dy"], d["w_down"], gu, d["offs"], dgu=gu)  # in place
    assert torch.equal(gu, dgu)


def test_backward_of_large_preactivations():
    """sigmoid at its limits: gradients stay finite, the closed gate gives 0."""
    d = make(4, [40], 64, 32, gather=False)
    gu = torch.zeros(40, 64, dtype=torch.bfloat16, device="cuda")
    gu[:, 32:] = 1.0
    gu[:, 0:8], gu[:, 8:16], gu[:, 16:24] = 200.0, -200.0, -3e38
    dgu = host(Q.moe_gated_backward(d["dy"], d["w_down"], gu, d["offs"]).double())
    want = M.gated_grad(M.grouped(host(d["dy"].double()), host(d["w_down"].double()).transpose(0, 2, 1), d["o"]),
                        host(gu.double()))
    assert np.isfinite(dgu).all()
    assert (dgu[:, 8:24] == 0).all() and (dgu[:, 40:56] == 0).all()
    assert (np.abs(dgu - want) <= HALF * np.abs(want) + 64 * 2.0 ** -24 * 60 + 1e-30)[:, :8].all()


def test_rows_behind_the_last_expert_stay():
    d = make(6, [20, 0, 13], 64, 48, gather=False)
    R = 33
    x = torch.cat((d["x"], d["x"][:9]))
    h, gu = Q.moe_gated_forward(x, d["w_gu"], d["offs"])
    h2, gu2 = Q.moe_gated_forward(d["x"], d["w_gu"], d["offs"])
    assert torch.equal(h[:R], h2) and torch.equal(gu[:R], gu2)
    dgu = torch.full((42, 96), 5.0, dtype=torch.bfloat16, device="cuda")
    dy = torch.cat((d["dy"], d["dy"][:9]))
    Q.moe_gated_backward(dy, d["w_down"], gu.fill_(1.0), d["offs"], dgu=dgu)
    assert bool((dgu[R:] == 5.0).all()) and not bool((dgu[:R] == 5.0).all())


def test_block_gradients():
    """The whole block as it is trained: MXFP4 QDQ of the masters, forward, backward with the existing
    weight-gradient and input-gradient calls, against the formulas in 64 bits.  The chain rounds h,
    gu and dgu to bf16: each gradient is a sum of products with relative errors of a few half steps, bounded by
    4 * 2^-8 of the sum of their magnitudes."""
    rng = np.random.default_rng(11)
    T, E, top, H, I = 200, 4, 2, 256, 128
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    _, _, offs, token, inv = Q.moe_route(logits, top)
    x = bf16(rng.standard_normal((T, H)))
    w_gu, _ = Q.weight_qdq_mxfp4(bf16(rng.standard_normal((E, 2 * I, H)) * 0.06))
    w_down, _ = Q.weight_qdq_mxfp4(bf16(rng.standard_normal((E, H, I)) * 0.06))
    dy = bf16(rng.standard_normal((T * top, H)))
    h, gu = Q.moe_gated_forward(x, w_gu, offs, token)
    dgu = Q.moe_gated_backward(dy, w_down, gu, offs)
    down = Q.QatBackward(w_down, dy, h, offs)
    up = Q.QatBackward(w_gu, dgu, x, offs, token, inv)
    _, _, dw_down = down()
    dx, _, dw_gu = up()

    X, G, D = (host(t.double()) for t in (x, w_gu, w_down))
    Y, o, t = host(dy.double()), host(offs), host(token)
    pre = M.grouped(X, G, o, t)
    hv = M.gated(pre)
    dh = M.grouped(Y, D.transpose(0, 2, 1), o)
    dpre = M.gated_grad(dh, pre)
    g, u = np.split(pre, 2, 1)
    s = M.sigmoid(g)
    # magnitudes that errors of g, u and dh can reach: |dh| |u| |silu''| <= |dh| |u| / 2 for a step of g
    ag, au = np.split(M.grouped(X, G, o, t, magnitude=True) * 0 + np.abs(pre), 2, 1)
    mag = np.concatenate((np.abs(dh) * (np.abs(u) * (1.1 + 0.5 * ag)), np.abs(dh) * (np.abs(g * s) + 1.1 * ag)), 1)
    hmag = np.abs(hv) + 1.1 * ag * np.abs(u)
    dXr, bound_x = M.grouped(dpre, G.transpose(0, 2, 1), o), M.grouped(mag, np.abs(G).transpose(0, 2, 1), o)
    want_dx, bdx = np.zeros((T, H)), np.zeros((T, H))
    np.add.at(want_dx, t, dXr)
    np.add.at(bdx, t, bound_x)
    assert (np.abs(host(dx) - want_dx) <= 4 * HALF * bdx).all()
    for e in range(E):
        a, b = o[e], o[e + 1]
        assert (np.abs(host(dw_gu[e]) - dpre[a:b].T @ X[t[a:b]]) <= 4 * HALF * (mag[a:b].T @ np.abs(X[t[a:b]]))).all()
        assert (np.abs(host(dw_down[e]) - Y[a:b].T @ hv[a:b]) <= 4 * HALF * (np.abs(Y[a:b]).T @ hmag[a:b])).all()


def test_gradient_against_differences():
    """dgu against differences of the forward's own formula: L = sum dy . W_down h(gu) in float64."""
    d = make(13, [7], 32, 16, gather=False)
    gu = bf16(np.random.default_rng(3).standard_normal((7, 32)))
    got = host(Q.moe_gated_backward(d["dy"], d["w_down"], gu, d["offs"]).double())
    dy, w, pre = host(d["dy"].double()), host(d["w_down"].double())[0], host(gu.double())
    loss = lambda p: (dy * (M.gated(p) @ w.T)).sum(1)  # noqa: E731
    eps = 1e-5
    for i in range(32):
        step = np.zeros_like(pre)
        step[:, i] = eps
        num = (loss(pre + step) - loss(pre - step)) / (2 * eps)
        dh = np.abs(dy) @ np.abs(w)
        part = (np.abs(pre[:, 16:]) * (1 + np.abs(pre[:, :16])) if i < 16 else np.abs(pre[:, :16]))[:, i % 16]
        tol = HALF * np.abs(num) + 32 * 2.0 ** -23 * dh[:, i % 16] * part + 1e-7
        assert (np.abs(got[:, i] - num) <= tol).all()


def test_capture():
    """Forward and backward captured once, replayed with the program's own work between the replays."""
    d = make(21, [70, 0, 30], 128, 64, gather=False)
    h, gu = Q.moe_gated_forward(d["x"], d["w_gu"], d["offs"])
    dgu = Q.moe_gated_backward(d["dy"], d["w_down"], gu, d["offs"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h1, gu1 = Q.moe_gated_forward(d["x"], d["w_gu"], d["offs"])
        dgu1 = Q.moe_gated_backward(d["dy"], d["w_down"], gu1, d["offs"])
    for _ in range(3):
        for t in (h1, gu1, dgu1):
            t.zero_()
        graph.replay()
        assert torch.equal(Q.moe_gated_forward(d["x"], d["w_gu"], d["offs"])[0], h)
        torch.cuda.synchronize()
        assert torch.equal(h1, h) and torch.equal(gu1, gu) and torch.equal(dgu1, dgu)


def test_empty_calls():
    d = make(2, [2, 1], 32, 16)
    offs = torch.zeros(3, dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    h, gu = Q.moe_gated_forward(d["x"], d["w_gu"], offs, none)
    assert h.shape == (0, 16) and gu.shape == (0, 32)
    assert Q.moe_gated_backward(d["dy"][:0], d["w_down"], gu, offs).shape == (0, 32)
