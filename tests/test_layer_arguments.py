"""What the operators around the experts take and refuse at the edges of their
documented arguments, before anything is enqueued: the C ABI on the CPU host.
Addresses are never dereferenced there; calls that would launch are not made."""
import ctypes
import os

import pytest

from fp4_quantized_moe_amd import _lib as Q

ARG, SHAPE, WORKSPACE = -1, -2, -3
P = 1 << 20  # an address


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(Q.LIB_PATH):
        pytest.fail("libquads.so is not built (python -m fp4_quantized_moe_amd.build)")
    return Q.load()


# up to 2^39 elements, however long their longer side
@pytest.mark.parametrize("batch, rows, cols", [(2, 16, 1048560), (300, 65536, 32), (17, 262144, 64), (65535, 16, 32768), (1, 1 << 19, 1 << 19),
                                               (32768, 4096, 4096)])
def test_orthogonalize_takes_the_documented_sizes(L, batch, rows, cols):
    assert batch * rows * cols <= 2 ** 39
    for r, c in ((rows, cols), (cols, rows)):
        assert L.quads_orthogonalize_workspace_bytes(batch, r, c) > 0
        d = (P, 1, batch, r, c, 5, (ctypes.c_float * 3)(3.4, -4.8, 2.0), 1e-7, P, None, 0, None)
        assert L.quads_orthogonalize(*d) == WORKSPACE  # the last check


@pytest.mark.parametrize("batch, rows, cols", [(32769, 4096, 4096), (2, 1 << 19, (1 << 19) + 16), (65535, 32, (1 << 18) + 16)])
def test_orthogonalize_refuses_more(L, batch, rows, cols):
    for r, c in ((rows, cols), (cols, rows)):
        assert L.quads_orthogonalize_workspace_bytes(batch, r, c) == 0 and b"overflow" in L.quads_last_error()


N8 = 8 * 64  # elements of the small calls below; every array has a place of its own, from which a case moves one
AT = {name: P + (1 << 20) * i for i, name in enumerate("x residual weight sum y_bf16 q_codes q_scales rstd dy s w dsum dx dw ws".split())}


@pytest.mark.parametrize("kw", [
    dict(sum=AT["x"], x_dtype=0), dict(sum=AT["x"] + 16), dict(sum=AT["residual"] + 2 * N8 - 16), dict(sum=AT["weight"] - 2 * N8 + 16),
    dict(y_bf16=AT["sum"]), dict(y_bf16=AT["x"], x_dtype=0), dict(y_bf16=AT["x"] - 16), dict(y_bf16=AT["residual"], residual_dtype=0),
    dict(y_bf16=AT["weight"]), dict(q_codes=AT["x"]), dict(q_codes=AT["y_bf16"]), dict(q_scales=AT["q_codes"]), dict(rstd=AT["q_scales"]),
    dict(rstd=AT["x"] + 64), dict(q_codes=AT["sum"] + 2 * N8 - 16), dict(q_scales=AT["residual"] + 16)])
def test_rms_norm_refuses_overlaps(L, kw):
    a = Q._RmsNormArgs()
    base = dict(struct_size=ctypes.sizeof(a), x_dtype=1, residual_dtype=1, weight_dtype=1, q_format=3, rows=8, cols=64, eps=1e-6)
    base.update({k: AT[k] for k in ("x", "residual", "weight", "sum", "y_bf16", "q_codes", "q_scales", "rstd")})
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    assert L.quads_rms_norm(ctypes.byref(a), None) == ARG and b"overlap" in L.quads_last_error()


@pytest.mark.parametrize("kw", [
    dict(dx=AT["dy"], dt=0), dict(dx=AT["dy"], st=0), dict(dx=AT["dy"] + 16), dict(dx=AT["s"] + 16), dict(dx=AT["s"] - 16),
    dict(dx=AT["dsum"] + 32), dict(dx=AT["w"]), dict(dx=AT["rstd"]), dict(dw=AT["dx"]), dict(dw=AT["s"]), dict(dw=AT["dy"]), dict(dw=AT["w"]),
    dict(ws=AT["dy"], rows=2000), dict(ws=AT["dx"] + 2 * 2000 * 64 - 16, rows=2000), dict(ws=AT["dw"] - 64, rows=2000)])
def test_rms_norm_backward_refuses_overlaps(L, kw):
    d = dict(dy=AT["dy"], dt=1, s=AT["s"], st=1, w=AT["w"], wt=0, rstd=AT["rstd"], dsum=AT["dsum"], rows=8, cols=64, dx=AT["dx"], dw=AT["dw"],
             ws=AT["ws"], nws=1 << 20, stream=None)
    assert L.quads_rms_norm_backward(*{**d, **kw}.values()) == ARG and b"overlap" in L.quads_last_error()


@pytest.mark.parametrize("kw", [dict(out=P), dict(out=P + 4 * 2 * 160 * 208 - 16), dict(out=P + 16, dt=1), dict(out=P - 16, dt=1), dict(ws=P),
                                dict(ws=P, out=P, dt=1), dict(ws=P + (4 << 20) + 16), dict(ws=P + (4 << 20) - 4096), dict(ws=P - 4096)])
@pytest.mark.parametrize("tall", [False, True])
def test_orthogonalize_refuses_overlaps(L, kw, tall):
    """g of fp32 under a bf16 out half its size: later passes and other matrices would read results."""
    d = dict(g=P, dt=0, batch=2, rows=160, cols=208, steps=5, co=(ctypes.c_float * 3)(3.4, -4.8, 2.0), eps=1e-7, out=P + (4 << 20),
             ws=P + (8 << 20), nws=1 << 20, stream=None)
    d.update(kw)
    if tall:
        d["rows"], d["cols"] = d["cols"], d["rows"]
    assert L.quads_orthogonalize(*d.values()) == ARG and b"overlap" in L.quads_last_error()


def test_orthogonalize_of_small_matrices_refuses_overlaps(L):
    for kw in (dict(out=P), dict(out=P + 32)):
        d = dict(g=P, dt=0, batch=2, rows=32, cols=48, steps=5, co=(ctypes.c_float * 3)(3.4, -4.8, 2.0), eps=1e-7, out=P, ws=None, nws=0, stream=None)
        assert L.quads_orthogonalize(*{**d, **kw}.values()) == ARG and b"overlap" in L.quads_last_error()


# places for the router's and the combine's arrays
PLACE = {name: P + (1 << 20) * i for i, name in enumerate("logits ids mask loss counts slope ws dw dloss dlogits dout y inv w dy".split())}


@pytest.mark.parametrize("kw", [dict(loss="logits"), dict(counts="ids"), dict(slope="mask"), dict(ws="logits"), dict(ws="counts"), dict(loss="slope"),
                                dict(counts="loss"), dict(slope="counts"), dict(loss=PLACE["logits"] + 4 * 5000 * 8 - 16), dict(ws=PLACE["ids"] - 1024)])
def test_balance_loss_refuses_overlaps(L, kw):
    d = dict(logits="logits", ids="ids", mask="mask", T=5000, E=8, top=2, coef=0.01, loss="loss", counts="counts", slope="slope", ws="ws",
             nws=1 << 20, stream=None)
    assert L.quads_moe_balance_loss(*[PLACE.get(v, v) for v in {**d, **kw}.values()]) == ARG and b"overlap" in L.quads_last_error()


@pytest.mark.parametrize("kw", [dict(dlogits=PLACE["logits"] + 16), dict(dlogits=PLACE["logits"] - 16), dict(dlogits="ids"), dict(dlogits="mask"), dict(dlogits="dw"),
                                dict(dlogits=PLACE["slope"] - 4 * 500 * 8 + 16), dict(dlogits="dloss")])
def test_route_backward_refuses_overlaps(L, kw):
    d = dict(logits="logits", ids="ids", mask="mask", dw="dw", slope="slope", dloss="dloss", T=500, E=8, top=2, dlogits="dlogits", stream=None)
    assert L.quads_moe_route_backward(*[PLACE.get(v, v) for v in {**d, **kw}.values()]) == ARG and b"overlap" in L.quads_last_error()


@pytest.mark.parametrize("kw", [dict(dy="dout"), dict(dy="y"), dict(dy=PLACE["y"] + 16, yt=1), dict(dy=PLACE["y"] - 32, yt=1), dict(dy="inv"), dict(dy="w"),
                                dict(dw="w"), dict(dw="inv"), dict(dw="dy"), dict(dw="y"), dict(dw=PLACE["dout"] + 4 * 50 * 32 - 16),
                                dict(dy=PLACE["dout"] + 16, y=None, dw=None)])
def test_combine_backward_refuses_overlaps(L, kw):
    d = dict(dout="dout", dt=0, y="y", yt=0, inv="inv", w="w", T=50, top=2, N=32, dy="dy", dw="dw", stream=None)
    assert L.quads_moe_combine_backward(*[PLACE.get(v, v) for v in {**d, **kw}.values()]) == ARG and b"overlap" in L.quads_last_error()


def test_dloss_is_a_float(L):
    for at in (1, 2, 3, 18):
        assert L.quads_moe_route_backward(P, P, None, P, P, P + at, 8, 4, 2, P, None) == ARG and b"4-byte aligned" in L.quads_last_error()


@pytest.mark.parametrize("out", [P, P + 496, P - 1008, P + (1 << 20), P + (1 << 20) - 16])
def test_dequantize_mxfp8_refuses_overlaps(L, out):
    """Values are two or four bytes, codes one: later codes would be read from values."""
    for dtype in (0, 1):
        assert L.quads_dequantize_mxfp8(Q._MXFP4(P, P + (1 << 20), 2, 4, 64), out, dtype, None) == ARG and b"overlap" in L.quads_last_error()
