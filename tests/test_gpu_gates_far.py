"""SwiGLU and its gradient with gates far from 0, in every kernel that has the
epilogue: one product a sum, so that g, u and dh are exact and what is left is
the error of silu and sigmoid.

With U = 2^-24 (half an fp32 step): the argument of 2^(-z log2 e) is off by a
rounding of the product and by 0.224 U of the constant, which e^-z multiplies by
|z|: 1.23 |z| U.  exp2 and the reciprocal are off by an ulp (2 U) each, the sum
and each product by U.  So s = sigmoid(z) by (5 + 1.23 |z|) U of s and silu(z) u
by (7 + 1.23 |z|) U.  1 - s is off by the error of s and U, so d gate = dh u s
(1 + z (1 - s)) and d up = dh z s by (16 + 2.5 |z|) U of |dh u| s (1 + |z|) and
|dh z| s.  Below z = -87 the reciprocal's result is subnormal and may be 0: off
by s, below 2^-124 from z = -86 on.  A bf16 output adds half a step, 2^-8 of it, 2^-134 among the
subnormals."""
import numpy as np
import pytest
import torch

from fp4_quantized_moe_amd import _lib as Q
from oracle import mxfp4_oracle as M
from gpu_util import host

pytestmark = pytest.mark.gpu
U, HALF, TINY = 2.0 ** -24, 2.0 ** -8, 2.0 ** -134


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).cuda()


def lost(z):
    """Bound on a sigmoid that may have become 0."""
    return np.where(z < -86, 2.0 ** -124, 0.0)


def offsets(R):
    return torch.tensor([0, R], dtype=torch.int32, device="cuda")


def silu_error(g, u):
    h = M.silu(g) * u
    return (7 + 1.23 * np.abs(g)) * U * np.abs(h) + np.abs(g * u) * lost(g) + HALF * np.abs(h) + TINY


def gates(I):
    """bf16 values from -95 to 95, and factors from 2^-6 to 2^6 of both signs."""
    rng = np.random.default_rng(I)
    g, u = np.linspace(-95, 95, I), rng.standard_normal(I) * np.exp2(rng.integers(-6, 7, I))
    return [host(bf16(v).double()) for v in (g, u)]


@pytest.mark.parametrize("R", [5, 9000])  # the streaming and the staged kernel
def test_gated_forward(R):
    I, H = 1024, 16
    g, u = gates(I)
    x, w = torch.zeros(R, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 2 * I, H, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1.0
    w[0, :, 0] = bf16(np.concatenate((g, u)))
    h, gu = Q.moe_gated_forward(x, w, offsets(R))
    assert bool((gu == w[0, :, 0]).all())
    assert bool((h == h[0]).all())
    assert (np.abs(host(h[0].double()) - M.silu(g) * u) <= silu_error(g, u)).all()


@pytest.mark.parametrize("R", [5, 9000])
def test_gated_backward(R):
    I, H = 1024, 16
    g, u = gates(I)
    dy, w = torch.zeros(R, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, H, I, dtype=torch.bfloat16, device="cuda")
    c = host(bf16(np.random.default_rng(1).standard_normal(I)).double())
    dy[:, 0] = 2.0
    w[0, 0] = bf16(c)
    gu = bf16(np.concatenate((g, u))).expand(R, 2 * I).contiguous()
    dgu = Q.moe_gated_backward(dy, w, gu, offsets(R))
    assert bool((dgu == dgu[0]).all())
    dh, s = 2 * c, M.sigmoid(g)
    want = M.gated_grad(dh, np.concatenate((g, u)))
    part = np.concatenate((np.abs(dh * u) * (1 + np.abs(g)), np.abs(dh * g)))
    z, ss = np.concatenate((g, g)), np.concatenate((s, s))
    err = part * ((16 + 2.5 * np.abs(z)) * U * ss + lost(z)) + HALF * np.abs(want) + TINY
    assert (np.abs(host(dgu[0].double()) - want) <= err).all()


@pytest.mark.parametrize("kernel, R, E, I, K", [("direct", 5, 1, 1024, 32), ("stream", 5, 1, 16384, 128),
                                                ("staged_small", 200, 2, 8192, 2048), ("staged_large", 40000, 1, 1024, 128)])
def test_mxfp4_swiglu(kernel, R, E, I, K):
    """Gates from 2^-6 to 96 that MXFP4 holds exactly, each alone in its block."""
    assert Q.mxfp4_gemm_kernel(R, E, 2 * I, K, Q.EPI_SWIGLU, torch.bfloat16) == kernel
    rng = np.random.default_rng(K)
    levels = np.outer([1, 1.5, -1, -1.5], np.exp2(np.arange(-6, 7))).ravel()
    g, u = rng.choice(levels, I), rng.choice(levels, I) / 32
    x, w = torch.zeros(R, K, device="cuda"), torch.zeros(E, 2 * I, K, device="cuda")
    x[:, 0] = 1.0
    w[:, :, 0] = torch.from_numpy(np.concatenate((g, u))).float().cuda()
    xq, wq = Q.quantize_mxfp4(x), Q.quantize_mxfp4(w)
    assert torch.equal(Q.dequantize_mxfp4(wq, torch.float32).view(E, 2 * I, K), w)
    offs = torch.tensor([R * e // E for e in range(E + 1)], dtype=torch.int32, device="cuda")
    h = Q.moe_mxfp4_gemm(xq, wq, offs, epilogue=Q.EPI_SWIGLU, y_dtype=torch.bfloat16)
    assert bool((h == h[0]).all())
    assert (np.abs(host(h[0].double()) - M.silu(g) * u) <= silu_error(g, u)).all()
