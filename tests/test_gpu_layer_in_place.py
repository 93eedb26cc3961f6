"""GPU: outputs in the place of inputs, where quads.h allows it: what the call
with arrays of its own gives, bit for bit."""
import ctypes

import pytest
import torch

from fp4_quantized_moe_amd import _lib as Q

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def stream():
    return torch.cuda.current_stream().cuda_stream


def seeded(n):
    return torch.Generator(device="cuda").manual_seed(n)


@pytest.mark.parametrize("rows, cols", [(1, 16), (5, 112), (333, 656), (2100, 496), (2100, 1008), (3, 4112), (700, 16384)])
@pytest.mark.parametrize("over", ["x", "residual"])
def test_norm_over_its_inputs(rows, cols, over):
    x, res = (torch.randn(rows, cols, generator=seeded(rows + i), device="cuda").to(bf) for i in range(2))
    w = (1 + 0.2 * torch.randn(cols, generator=seeded(3), device="cuda")).to(bf)
    want = Q.rms_norm(x, w, residual=res, keep=True)
    # y over one of the two, the stream over the other
    y, s = (x, res) if over == "x" else (res, x)
    rstd = torch.empty(rows, device="cuda")
    a = Q._RmsNormArgs(ctypes.sizeof(Q._RmsNormArgs), 0, Q.BF16, Q.BF16, Q.BF16, -1, rows, cols, x.data_ptr(), res.data_ptr(), w.data_ptr(),
                       s.data_ptr(), y.data_ptr(), None, None, rstd.data_ptr(), 1e-6, 0)
    assert Q.load().quads_rms_norm(ctypes.byref(a), stream()) == 0
    assert torch.equal(y, want.y) and torch.equal(s, want.sum) and torch.equal(rstd, want.rstd)


@pytest.mark.parametrize("rows", [1, 127, 129, 511, 1023, 1024, 1025, 3000])
@pytest.mark.parametrize("cols", [16, 64, 1072, 4112])
@pytest.mark.parametrize("dy_type, s_type", [(bf, bf), (f32, bf), (bf, f32)])
def test_norm_gradient_over_the_stream(rows, cols, dy_type, s_type):
    """dx in the place of s, whose rows dweight's sums need too."""
    s, dsum = (torch.randn(rows, cols, generator=seeded(rows + cols + i), device="cuda").to(s_type) for i in range(2))
    dy = torch.randn(rows, cols, generator=seeded(7), device="cuda").to(dy_type)
    w = torch.rand(cols, generator=seeded(8), device="cuda") + 0.5
    rstd = torch.rsqrt(s.float().square().mean(1) + 1e-6)
    dx, dweight = Q.rms_norm_backward(dy, s, w, rstd, dsum=dsum)
    L, code = Q.load(), lambda t: Q.F32 if t == f32 else Q.BF16
    nbytes = L.quads_rms_norm_backward_workspace_bytes(rows, cols)
    ws, dw = torch.empty(nbytes + 16, dtype=torch.uint8, device="cuda"), torch.empty(cols, device="cuda")
    st = L.quads_rms_norm_backward(dy.data_ptr(), code(dy_type), s.data_ptr(), code(s_type), w.data_ptr(), Q.F32, rstd.data_ptr(),
                                   dsum.data_ptr(), rows, cols, s.data_ptr(), dw.data_ptr(), ws.data_ptr(), nbytes, stream())
    assert st == 0 and torch.equal(s, dx) and torch.equal(dw, dweight)


@pytest.mark.parametrize("T, E, top", [(1, 3, 1), (777, 12, 3), (3000, 100, 8), (70, 1000, 16)])
def test_router_gradient_over_the_logits(T, E, top):
    logits = 2 * torch.randn(T, E, generator=seeded(T + E), device="cuda")
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :top].int().contiguous()
    dw, b = torch.randn(T, top, generator=seeded(1), device="cuda"), Q.moe_balance_loss(logits, ids, 0.01)
    want = Q.moe_route_backward(logits, ids, dw=dw, slope=b.slope)
    assert Q.load().quads_moe_route_backward(logits.data_ptr(), ids.data_ptr(), None, dw.data_ptr(), b.slope.data_ptr(), None, T, E, top,
                                             logits.data_ptr(), stream()) == 0
    assert torch.equal(logits, want)


@pytest.mark.parametrize("T, top, N", [(1, 3, 16), (333, 3, 656), (1100, 16, 528), (1100, 5, 2064), (40, 8, 2048)])
@pytest.mark.parametrize("drop", [False, True])
def test_combine_gradient_over_the_rows(T, top, N, drop):
    """dy in the place of y, also with slots that have no row (their rows keep y)."""
    inverse = torch.randperm(T * top, generator=seeded(2), device="cuda").int().view(T, top)
    dout, y = torch.randn(T, N, generator=seeded(3), device="cuda"), torch.randn(T * top, N, generator=seeded(4), device="cuda").to(bf)
    w = torch.rand(T, top, generator=seeded(5), device="cuda")
    if drop:
        inverse[torch.rand(T, top, generator=seeded(6), device="cuda") < 0.3] = -1
    dy, dw = Q.moe_combine_backward(dout, y, inverse, w, out=y.clone())
    got, dw_got = Q.moe_combine_backward(dout, y, inverse, w, out=y)
    assert got is y and torch.equal(got, dy) and torch.equal(dw_got, dw)
