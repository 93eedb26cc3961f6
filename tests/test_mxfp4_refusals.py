"""What the MXFP4 and gated entry points refuse, before anything is enqueued:
status codes of the C ABI on the CPU host, and the binding's own checks."""
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


def mx(rows, cols, batch=1, ptr=P):
    return Q._MXFP4(ptr, ptr, batch, rows, cols)


@pytest.mark.parametrize("args, status, word", [
    ((P, 0, mx(4, 48), 0), SHAPE, b"multiple of 32"),
    ((P, 0, mx(4, 0), 0), SHAPE, b"multiple of 32"),
    ((P, 0, mx(-1, 32), 0), SHAPE, b"bad shape"),
    ((P, 0, mx(4, 32, batch=0), 0), SHAPE, b"bad shape"),
    ((P, 0, mx(1 << 40, 1 << 20), 0), SHAPE, b"overflow"),
    ((P, 2, mx(4, 32), 0), ARG, b"dtype"),
    ((P, 0, mx(4, 32), 1), ARG, b"flags"),
    ((None, 0, mx(4, 32), 0), ARG, b"null"),
    ((P, 0, mx(4, 32, ptr=None), 0), ARG, b"null"),
    ((P, 0, mx(4, 32, ptr=24), 0), ARG, b"aligned"),
    ((24, 1, mx(4, 32), 8), ARG, b"aligned"),
])
def test_quantize(L, args, status, word):
    assert L.quads_quantize_mxfp4(*args, None) == status
    assert word in L.quads_last_error()


def test_quantize_no_rows(L):
    assert L.quads_quantize_mxfp4(None, 0, mx(0, 32, ptr=None), 0, None) == 0
    assert L.quads_dequantize_mxfp4(mx(0, 32, ptr=None), None, 0, None) == 0
    assert L.quads_weight_qdq_mxfp4(None, 1, 0, 32, None, None, 0, None) == 0


def test_dequantize_and_qdq(L):
    assert L.quads_dequantize_mxfp4(mx(4, 16), P, 0, None) == SHAPE
    assert L.quads_dequantize_mxfp4(mx(4, 32), None, 0, None) == ARG
    assert L.quads_dequantize_mxfp4(mx(4, 32), P, 3, None) == ARG
    assert L.quads_dequantize_mxfp4(mx(4, 32), 8, 0, None) == ARG
    q = mx(4, 64)
    assert L.quads_weight_qdq_mxfp4(P, 1, 4, 32, P, ctypes.byref(q), 0, None) == SHAPE
    assert L.quads_weight_qdq_mxfp4(P, 1, 4, 40, P, None, 0, None) == SHAPE
    assert L.quads_weight_qdq_mxfp4(P, 1, 4, 32, None, None, 0, None) == ARG
    assert L.quads_weight_qdq_mxfp4(P, 1, 4, 32, P, None, 2, None) == ARG


def gemm_args(**kw):
    a = Q._MxGemmArgs()
    base = dict(struct_size=ctypes.sizeof(Q._MxGemmArgs), num_experts=2, num_rows=4, act_rows=4, N=64, K=64, x_codes=P,
                x_scales=P, w_codes=P, w_scales=P, expert_offsets=P, y=P)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw, status, word", [
    (dict(struct_size=8), ARG, b"struct_size"), (dict(flags=1), ARG, b"flags"), (dict(reserved=1), ARG, b"flags"),
    (dict(epilogue=2), ARG, b"epilogue"), (dict(y_dtype=2), ARG, b"y_dtype"),
    (dict(epilogue=1, y_dtype=0), ARG, b"y_dtype"), (dict(K=48), SHAPE, b"K must"), (dict(K=0), SHAPE, b"K must"),
    (dict(N=48), SHAPE, b"N must"), (dict(N=96, epilogue=1, y_dtype=1), SHAPE, b"multiple of 64"),
    (dict(num_experts=0), SHAPE, b"num_experts"), (dict(num_experts=1025), SHAPE, b"num_experts"),
    (dict(num_rows=-1), SHAPE, b"row counts"), (dict(num_rows=1 << 31), SHAPE, b"row counts"),
    (dict(act_rows=3), SHAPE, b"identity"), (dict(act_rows=0, row_token=P), SHAPE, b"no activation"),
    (dict(K=1 << 24), SHAPE, b"overflow"), (dict(expert_offsets=None), ARG, b"null"), (dict(w_scales=None), ARG, b"null"),
    (dict(x_codes=None), ARG, b"null"), (dict(y=None), ARG, b"null"), (dict(x_scales=20), ARG, b"aligned"),
    (dict(epilogue=1, y_dtype=2, y_scales=None), ARG, b"null"),
])
def test_gemm(L, kw, status, word):
    assert L.quads_moe_mxfp4_gemm(ctypes.byref(gemm_args(**kw)), None) == status
    assert word in L.quads_last_error()


def test_gemm_no_rows(L):
    assert L.quads_moe_mxfp4_gemm(ctypes.byref(gemm_args(num_rows=0, act_rows=0, x_codes=None, x_scales=None, y=None)), None) == 0
    assert L.quads_moe_mxfp4_gemm(None, None) == ARG


@pytest.mark.parametrize("kw, status, word", [
    (dict(H=48), SHAPE, b"multiples of 32"), (dict(I=0), SHAPE, b"multiples of 32"), (dict(dt=2), ARG, b"y_dtype"),
    (dict(wg=mx(64, 64, 2)), SHAPE, b"weights must"), (dict(wd=mx(64, 32, 3)), SHAPE, b"weights must"),
    (dict(wg=mx(128, 64, 2, None)), ARG, b"null"), (dict(offs=None), ARG, b"null"), (dict(x=None), ARG, b"null"),
    (dict(y=8), ARG, b"aligned"), (dict(ws=None), WORKSPACE, b"workspace"), (dict(nws=100), WORKSPACE, b"workspace"),
    (dict(E=0), SHAPE, b"num_experts"), (dict(A=2), SHAPE, b"identity"),
])
def test_ffn(L, kw, status, word):
    d = dict(x=P, wg=mx(128, 64, 2), wd=mx(64, 64, 2), rt=None, offs=P, E=2, R=4, A=4, H=64, I=64, y=P, dt=0, ws=P,
             nws=1 << 20, stream=None)
    d.update(kw)
    d["wg"], d["wd"] = ctypes.byref(d["wg"]), ctypes.byref(d["wd"])
    assert L.quads_moe_mxfp4_ffn(*d.values()) == status
    assert word in L.quads_last_error()


def test_ffn_workspace(L):
    f = L.quads_moe_mxfp4_ffn_workspace_bytes
    assert f(4, 8, 64, 64) >= (4 * 64 + 8 * 64) * 17 // 32
    assert f(-1, 8, 64, 64) == 0 and f(4, 8, 48, 64) == 0 and f(1 << 40, 8, 1 << 20, 64) == 0


def test_gated(L):
    fwd, bwd = L.quads_moe_gated_forward_bf16, L.quads_moe_gated_backward_bf16
    assert fwd(P, P, None, P, 2, 4, 4, 40, 32, P, P, None) == SHAPE and b"multiples of 16" in L.quads_last_error()
    assert fwd(P, P, None, P, 2, 4, 4, 32, 24, P, P, None) == SHAPE
    assert fwd(P, P, None, P, 0, 4, 4, 32, 32, P, P, None) == SHAPE
    assert fwd(P, P, None, P, 2, 4, 3, 32, 32, P, P, None) == SHAPE
    assert fwd(P, None, None, P, 2, 4, 4, 32, 32, P, P, None) == ARG
    assert fwd(P, P, None, None, 2, 4, 4, 32, 32, P, P, None) == ARG
    assert fwd(P, P, None, P, 2, 4, 4, 32, 32, None, P, None) == ARG
    assert fwd(P, P, None, P, 2, 4, 4, 32, 32, 8, P, None) == ARG and b"aligned" in L.quads_last_error()
    assert fwd(None, P, None, P, 2, 0, 0, 32, 32, None, None, None) == 0
    assert bwd(P, P, P, P, 2, 4, 32, 40, P, None) == SHAPE
    assert bwd(P, P, P, P, 1025, 4, 32, 32, P, None) == SHAPE
    assert bwd(P, P, None, P, 2, 4, 32, 32, P, None) == ARG
    assert bwd(P, P, P, P, 2, 4, 32, 32, None, None) == ARG
    assert bwd(P, P, P, P, 2, 4, 32, 32, 24, None) == ARG
    assert bwd(None, P, None, P, 2, 0, 32, 32, None, None) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: Q.quantize_mxfp4(x), lambda: Q.weight_qdq_mxfp4(x),
                 lambda: Q.mxfp4_tensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)),
                 lambda: Q.moe_gated_forward(x, x[None], torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(Q.QuadsError, match="on the GPU"):
            call()


@pytest.mark.gpu
def test_binding_refuses_shapes_and_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    q = Q.quantize_mxfp4(x)
    w = Q.quantize_mxfp4(torch.zeros(2, 64, 64, dtype=torch.bfloat16, device="cuda"))
    offs = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    up, down = torch.zeros(2, 64, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 64, 32, dtype=torch.bfloat16, device="cuda")
    gu = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    for word, call in (
        ("multiple of 32", lambda: Q.quantize_mxfp4(x[:, :48].contiguous())),
        ("contiguous", lambda: Q.quantize_mxfp4(x.t())),
        ("must be torch", lambda: Q.quantize_mxfp4(x.half())),
        ("rule", lambda: Q.quantize_mxfp4(x, rule="ceil")),
        ("expected", lambda: Q.quantize_mxfp4(x[0])),
        ("out is", lambda: Q.quantize_mxfp4(x, out=Q.empty_mxfp4(1, 3, 64, "cuda"))),
        ("dtype", lambda: Q.dequantize_mxfp4(q, torch.float16)),
        ("do not match", lambda: Q.mxfp4_tensor(q.codes, q.scales[:, :1].contiguous())),
        ("expert_offsets holds", lambda: Q.moe_mxfp4_gemm(q, w, offs[:2])),
        ("must be torch.int32", lambda: Q.moe_mxfp4_gemm(q, w, offs.long())),
        ("must be torch.int32", lambda: Q.moe_mxfp4_gemm(q, w, offs, offs.float())),
        ("y_dtype", lambda: Q.moe_mxfp4_gemm(q, w, offs, y_dtype=torch.float16)),
        ("y_dtype", lambda: Q.moe_mxfp4_gemm(q, w, offs, y_dtype=Q.MXFP4)),
        ("y_dtype", lambda: Q.moe_mxfp4_gemm(q, w, offs, epilogue=Q.EPI_SWIGLU)),
        ("y must be", lambda: Q.moe_mxfp4_gemm(q, w, offs, y=torch.zeros(4, 32, device="cuda"))),
        ("needs w_gate_up", lambda: Q.moe_mxfp4_ffn(x, w, w, offs)),
        ("do not match", lambda: Q.moe_gated_forward(x, up[..., :32].contiguous(), offs)),
        ("do not match", lambda: Q.moe_gated_backward(x, down, gu[:3], offs)),
        ("expert_offsets holds", lambda: Q.moe_gated_backward(x, down, gu, offs[:2])),
        ("must be torch.bfloat16", lambda: Q.moe_gated_backward(x.float(), down, gu, offs)),
    ):
        with pytest.raises(Q.QuadsError, match=word):
            call()
