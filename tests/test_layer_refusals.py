"""What the norm, router-gradient and combine-gradient entry points refuse,
before anything is enqueued: status codes of the C ABI on the CPU host, and the
binding's own checks."""
import ctypes
import os

import pytest
import torch

from fp4_quantized_moe_amd import _lib as Q

ARG, SHAPE, WORKSPACE = -1, -2, -3
P = 16  # an aligned non-null address: never dereferenced on the host


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(Q.LIB_PATH):
        pytest.fail("libquads.so is not built (python -m fp4_quantized_moe_amd.build)")
    return Q.load()


def norm_args(**kw):
    a = Q._RmsNormArgs()
    base = dict(struct_size=ctypes.sizeof(Q._RmsNormArgs), x_dtype=1, residual_dtype=1, weight_dtype=1, q_format=-1, rows=4,
                cols=64, x=P, residual=P, weight=P, sum=P, y_bf16=P, eps=1e-6)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw, status, word", [
    (dict(struct_size=8), ARG, b"struct_size"), (dict(q_format=0), ARG, b"q_format"), (dict(q_format=4), ARG, b"q_format"),
    (dict(flags=8), ARG, b"flags"), (dict(flags=8, q_format=3, q_codes=P, q_scales=P), ARG, b"flags"),
    (dict(flags=1, q_format=2, q_codes=P, q_scales=P), ARG, b"flags"), (dict(reserved=1), ARG, b"flags"),
    (dict(x_dtype=2), ARG, b"dtype"), (dict(residual_dtype=-1), ARG, b"dtype"), (dict(weight_dtype=3), ARG, b"dtype"),
    (dict(cols=0), SHAPE, b"multiple of 16"), (dict(cols=24), SHAPE, b"multiple of 16"),
    (dict(cols=16400), SHAPE, b"16384"), (dict(rows=-1), SHAPE, b"row count"), (dict(rows=1 << 31), SHAPE, b"row count"),
    (dict(cols=48, q_format=2, q_codes=P, q_scales=P), SHAPE, b"% 32"), (dict(eps=-1.0), ARG, b"eps"),
    (dict(eps=float("nan")), ARG, b"eps"), (dict(x=24), ARG, b"aligned"), (dict(rstd=4), ARG, b"aligned"),
    (dict(residual=None), ARG, b"sum without"), (dict(q_codes=P), ARG, b"without a q_format"), (dict(x=None), ARG, b"null"),
    (dict(weight=None), ARG, b"null"), (dict(sum=None), ARG, b"null"), (dict(q_format=2, q_codes=P), ARG, b"null"),
])
def test_rms_norm(L, kw, status, word):
    assert L.quads_rms_norm(ctypes.byref(norm_args(**kw)), None) == status
    assert word in L.quads_last_error()


def test_rms_norm_without_rows(L):
    assert L.quads_rms_norm(None, None) == ARG
    a = norm_args(rows=0, x=None, residual=None, sum=None, weight=None, y_bf16=None)
    assert L.quads_rms_norm(ctypes.byref(a), None) == 0


@pytest.mark.parametrize("kw, status, word", [
    (dict(dt=2), ARG, b"dtype"), (dict(st=5), ARG, b"dtype"), (dict(cols=8), SHAPE, b"multiple of 16"),
    (dict(rows=-1), SHAPE, b"row count"), (dict(s=None), ARG, b"null"), (dict(dx=None), ARG, b"null"),
    (dict(dsum=8), ARG, b"aligned"), (dict(rows=4000, ws=None), WORKSPACE, b"workspace"),
    (dict(rows=4000, nws=16), WORKSPACE, b"workspace"),
])
def test_rms_norm_backward(L, kw, status, word):
    d = dict(dy=P, dt=1, s=P, st=1, w=P, wt=0, rstd=P, dsum=None, rows=4, cols=64, dx=P, dw=P, ws=P, nws=1 << 20, stream=None)
    assert L.quads_rms_norm_backward(*{**d, **kw}.values()) == status
    assert word in L.quads_last_error()


def test_rms_norm_backward_workspace(L):
    f = L.quads_rms_norm_backward_workspace_bytes
    assert f(4000, 64) >= 256 and f(4, 64) == 0 and f(0, 64) == 0 and f(4, 24) == 0 and f(-1, 64) == 0 and f(4, 1 << 20) == 0
    assert L.quads_rms_norm_backward(None, 1, None, 1, None, 1, None, None, 0, 64, None, None, None, 0, None) == 0


def test_dequantize_mxfp8(L):
    f = L.quads_dequantize_mxfp8
    q = lambda rows, cols, batch=1, ptr=P: Q._MXFP4(ptr, ptr, batch, rows, cols)  # noqa: E731
    assert f(q(4, 48), P, 0, None) == SHAPE and f(q(4, 64, 0), P, 0, None) == SHAPE
    assert f(q(1 << 40, 1 << 20), P, 0, None) == SHAPE and f(q(4, 64), P, 2, None) == ARG
    assert f(q(4, 64, 1, None), P, 0, None) == ARG and f(q(4, 64), 8, 0, None) == ARG
    assert f(q(0, 64, 1, None), None, 0, None) == 0


@pytest.mark.parametrize("kw, status, word", [
    (dict(E=0), SHAPE, b"E must"), (dict(E=1025), SHAPE, b"E must"), (dict(top=0), SHAPE, b"top must"),
    (dict(top=5), SHAPE, b"top must"), (dict(E=64, top=17), SHAPE, b"top must"), (dict(T=-1), SHAPE, b"token count"),
    (dict(T=1 << 31), SHAPE, b"token count"), (dict(logits=None), ARG, b"null"), (dict(ids=None), ARG, b"null"),
    (dict(slope=None), ARG, b"null"), (dict(loss=4), ARG, b"aligned"), (dict(T=5000, ws=None), WORKSPACE, b"workspace"),
    (dict(T=5000, nws=64), WORKSPACE, b"workspace"),
])
def test_balance_loss(L, kw, status, word):
    d = dict(logits=P, ids=P, mask=None, T=8, E=4, top=2, coef=0.01, loss=P, counts=P, slope=P, ws=P, nws=1 << 20, stream=None)
    assert L.quads_moe_balance_loss(*{**d, **kw}.values()) == status
    assert word in L.quads_last_error()


def test_balance_loss_workspace(L):
    f = L.quads_moe_balance_loss_workspace_bytes
    assert f(8, 4) == 0 and f(1 << 20, 128) > 0 and f(-1, 4) == 0 and f(8, 0) == 0 and f(8, 2000) == 0


@pytest.mark.parametrize("kw, status, word", [
    (dict(E=0), SHAPE, b"E must"), (dict(top=17, E=32), SHAPE, b"top must"), (dict(T=-1), SHAPE, b"token count"),
    (dict(dlogits=None), ARG, b"null"), (dict(ids=None), ARG, b"null"), (dict(dw=20), ARG, b"aligned"),
])
def test_route_backward(L, kw, status, word):
    d = dict(logits=P, ids=P, mask=None, dw=P, slope=P, dloss=None, T=8, E=4, top=2, dlogits=P, stream=None)
    assert L.quads_moe_route_backward(*{**d, **kw}.values()) == status
    assert word in L.quads_last_error()


def test_route_backward_without_tokens(L):
    assert L.quads_moe_route_backward(None, None, None, None, None, None, 0, 4, 2, None, None) == 0


@pytest.mark.parametrize("kw, status, word", [
    (dict(dt=2), ARG, b"dtype"), (dict(yt=2), ARG, b"dtype"), (dict(top=0), SHAPE, b"top must"), (dict(top=17), SHAPE, b"top must"),
    (dict(T=-1), SHAPE, b"token count"), (dict(N=24), SHAPE, b"multiple of 16"), (dict(N=0), SHAPE, b"multiple of 16"),
    (dict(T=1 << 24, N=1 << 20), SHAPE, b"overflow"), (dict(y=None), ARG, b"null"), (dict(dy=None), ARG, b"null"),
    (dict(inv=8), ARG, b"aligned"),
])
def test_combine_backward(L, kw, status, word):
    d = dict(dout=P, dt=0, y=P, yt=0, inv=P, w=P, T=8, top=2, N=32, dy=P, dw=P, stream=None)
    assert L.quads_moe_combine_backward(*{**d, **kw}.values()) == status
    assert word in L.quads_last_error()


def test_combine_backward_without_tokens(L):
    assert L.quads_moe_combine_backward(None, 0, None, 0, None, None, 0, 2, 32, None, None, None) == 0


def test_binding_refuses_cpu_tensors():
    f, h, i = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: Q.rms_norm(h, h[0]), lambda: Q.rms_norm_backward(h, h, h[0], f[:, 0]),
                 lambda: Q.dequantize_mxfp8(Q.MXFP8Tensor(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8), 1, 4, 64)),
                 lambda: Q.moe_balance_loss(f, i, 0.01), lambda: Q.moe_route_backward(f, i),
                 lambda: Q.moe_combine_backward(h, f, i, f[:, :2])):
        with pytest.raises(Q.QuadsError, match="contiguous and on the GPU"):
            call()
    with pytest.raises(Q.QuadsError):
        Q.rms_norm(torch.zeros(4, 64, dtype=torch.float16), h[0])


@pytest.mark.parametrize("kw, status, word", [
    (dict(dt=2), ARG, b"dtype"), (dict(rows=0), SHAPE, b"multiples of 16"), (dict(cols=40), SHAPE, b"multiples of 16"),
    (dict(rows=1 << 20), SHAPE, b"below 2^20"), (dict(batch=-1), SHAPE, b"batch"), (dict(batch=65536), SHAPE, b"batch"),
    (dict(batch=60000, rows=16, cols=(1 << 20) - 16), SHAPE, b"overflow"), (dict(steps=0), ARG, b"steps"),
    (dict(steps=65), ARG, b"steps"), (dict(co=None), ARG, b"coefficients"), (dict(eps=-1e-9), ARG, b"eps"),
    (dict(g=8), ARG, b"aligned"), (dict(g=None), ARG, b"null"), (dict(out=None), ARG, b"null"),
    (dict(ws=None), WORKSPACE, b"workspace"), (dict(nws=1000), WORKSPACE, b"workspace"),
])
def test_orthogonalize(L, kw, status, word):
    d = dict(g=P, dt=0, batch=2, rows=160, cols=208, steps=5, co=(ctypes.c_float * 3)(3.4, -4.8, 2.0), eps=1e-7, out=P, ws=P,
             nws=1 << 20, stream=None)
    assert L.quads_orthogonalize(*{**d, **kw}.values()) == status
    assert word in L.quads_last_error()


def test_orthogonalize_without_matrices(L):
    f = L.quads_orthogonalize_workspace_bytes
    assert f(2, 160, 208) >= 2 * (3 * 160 * 208 + 2 * 160 * 160) * 2 and f(0, 160, 208) == 0 and f(2, 24, 48) == 0
    assert f(2, 32, 48) == 0  # a workgroup's LDS holds it
    assert L.quads_orthogonalize(None, 0, 0, 32, 48, 5, (ctypes.c_float * 3)(1, 1, 1), 0.0, None, None, 0, None) == 0
    with pytest.raises(Q.QuadsError, match="contiguous and on the GPU"):
        Q.orthogonalize(torch.zeros(32, 32))
