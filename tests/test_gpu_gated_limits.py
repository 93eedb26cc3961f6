"""The gated block at the ends of its documented range: inter up to 2^24, and
operands past 32-bit offsets, against float64 products on the GPU.

Tolerances: K products exact in fp32 are off by at most K 2^-24 sum |w x| in any
order, to first order; a bf16 output by half a step more, 2^-8 |y|; silu and the
gradient of (g, u) by 2^-18 of their terms for the |g| < 16 here (7 + 1.23 |g| and
16 + 2.5 |g| halves of an fp32 step, 2^-24)."""
import pytest
import torch

from fp4_quantized_moe_amd import _lib as Q

gpu = pytest.mark.gpu
P = 16  # an aligned address that is not touched
HALF = 2.0 ** -8


def test_accepted_and_refused():
    L = Q.load()
    for hidden, inter, status in ((16, 1 << 23, 0), (16, (1 << 24) - 16, 0), (16, 1 << 24, -2), ((1 << 24) - 16, 16, 0),
                                  (1 << 24, 16, -2)):
        assert L.quads_moe_gated_forward_bf16(None, P, None, P, 1, 0, 0, hidden, inter, None, None, None) == status
        assert L.quads_moe_gated_backward_bf16(None, P, None, P, 1, 0, hidden, inter, None, None) == status
    # 2 inter is an N of the MXFP4 product, whose limit is 2^24 as it stands
    wg, wd = Q._MXFP4(P, P, 1, 1 << 24, 32), Q._MXFP4(P, P, 1, 32, 1 << 23)
    assert L.quads_moe_mxfp4_ffn(None, wg, wd, None, P, 1, 0, 0, 32, 1 << 23, None, 0, None, 0, None) == -2


def seeded(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(gen, *shape):
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    for p in flat.split(1 << 28):
        p.copy_(torch.randn(p.shape, generator=gen, device="cuda"))
    return out


def check_forward(x, w, h, gu):
    """Rows x of one expert w [2 I, H], in column chunks."""
    I, H = w.shape[0] // 2, w.shape[1]
    xd = x.double()
    for a in range(0, I, 1 << 20):
        b = min(I, a + (1 << 20))
        part = {}
        for name, off in (("g", 0), ("u", I)):
            wd = w[off + a:off + b].double()
            y, tol = xd @ wd.T, H * 2.0 ** -24 * (xd.abs() @ wd.abs().T)
            assert bool(((gu[:, off + a:off + b].double() - y).abs() <= tol + HALF * y.abs()).all()), (name, a)
            part[name] = (y, tol)
        (g, tg), (u, tu) = part["g"], part["u"]
        s = g * torch.sigmoid(g)
        err = 1.1 * tg * (u.abs() + tu) + s.abs() * tu + (2.0 ** -18 + HALF) * (s * u).abs()
        assert bool(((h[:, a:b].double() - s * u).abs() <= err).all()), a


def check_backward(dy, w, gu, dgu):
    """Rows dy of one expert w [H, I], in column chunks."""
    H, I = w.shape
    d = dy.double()
    for a in range(0, I, 1 << 20):
        b = min(I, a + (1 << 20))
        wd = w[:, a:b].double()
        dh, tol = d @ wd, H * 2.0 ** -24 * (d.abs() @ wd.abs())
        g, u = gu[:, a:b].double(), gu[:, I + a:I + b].double()
        s = torch.sigmoid(g)
        for got, f, size in ((dgu[:, a:b], u * s * (1 + g * (1 - s)), u.abs() * s * (1 + g.abs())), (dgu[:, I + a:I + b], g * s, g.abs() * s)):
            want = dh * f
            assert bool(((got.double() - want).abs() <= (tol + 2.0 ** -18 * dh.abs()) * size + HALF * want.abs()).all()), a


@gpu
@pytest.mark.parametrize("inter", [1 << 23, (1 << 24) - 16])
def test_widest(inter):
    gen, H, R = seeded(1), 16, 3
    offs = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    x, w = randn(gen, R, H), randn(gen, 1, 2 * inter, H).mul_(0.25)
    h, gu = Q.moe_gated_forward(x, w, offs)
    check_forward(x, w[0], h, gu)
    wd = w.view(-1)[:H * inter].view(1, H, inter)
    dgu = Q.moe_gated_backward(x, wd, gu, offs)
    check_backward(x, wd[0], gu, dgu)


@gpu
@pytest.mark.parametrize("R", [40, 700])  # 8 and 92 MB of weights to read: the streaming and the staged kernel
def test_rows_past_32_bits(R):
    gen, H, I = seeded(R), 2048, 512
    rows = 2 ** 32 // (2 * H) + R + 3
    x = torch.zeros(rows, H, dtype=torch.bfloat16, device="cuda")
    x[-R:] = randn(gen, R, H)
    w = randn(gen, 2, 2 * I, H).mul_(H ** -0.5)
    token = torch.arange(rows - 1, rows - R - 1, -1, dtype=torch.int32, device="cuda")
    h, gu = Q.moe_gated_forward(x, w, torch.tensor([0, R // 3, R], dtype=torch.int32, device="cuda"), token)
    for e, (a, b) in enumerate(((0, R // 3), (R // 3, R))):
        check_forward(x[token[a:b].long()], w[e], h[a:b], gu[a:b])


@gpu
def test_rows_and_outputs_past_32_bits():
    """Backward: dy, gu and dgu past 2^32 bytes, of one expert's rows; slices at the start, the middle and the end."""
    gen, H, I = seeded(5), 2048, 1024
    R = 2 ** 32 // (2 * H) + 300
    dy = randn(gen, R, H)
    gu, w = randn(gen, R, 2 * I), randn(gen, 1, H, I).mul_(0.05)
    dgu = Q.moe_gated_backward(dy, w, gu, torch.tensor([0, R], dtype=torch.int32, device="cuda"))
    for a in (0, R // 2, R - 600):
        check_backward(dy[a:a + 600], w[0], gu[a:a + 600], dgu[a:a + 600])


@gpu
def test_weights_past_32_bits():
    gen, H, I, E, R = seeded(6), 1024, 2048, 520, 50
    w = torch.zeros(E, 2 * I, H, dtype=torch.bfloat16, device="cuda")
    w[-1] = randn(gen, 2 * I, H).mul_(H ** -0.5)
    assert (E - 1) * 4 * I * H >= 2 ** 32
    offs = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offs[-1] = R
    x = randn(gen, R, H)
    h, gu = Q.moe_gated_forward(x, w, offs)
    check_forward(x, w[-1], h, gu)
    w, H = w.view(E, 2048, 2048), 2048  # the same bytes as down projections of another hidden size
    dy, gu = randn(gen, R, H), randn(gen, R, 2 * 2048)
    check_backward(dy, w[-1], gu, Q.moe_gated_backward(dy, w, gu, offs))
