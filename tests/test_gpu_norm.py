"""GPU: the norm with its residual addition and quantized outputs, its gradient
and the MXFP8 codec against the 64-bit oracle.

Tolerances, with u = 2^-24.  The kernel's sum of squares is off by at most H u
of itself in any order, so rstd by (H / 2 + 4) u (mean, eps, root and quotient
u each) and y = s r w by two more: e_y = (H / 2 + 6) u relative.  A bf16 output
rounds once more, 2^-8 |y|.  A quantized output must be what the oracle makes
of some value within e_y of y: the scale byte lies between those of the block's
largest magnitude times (1 -+ e_y), a code between those of y times (1 -+ e_y)
under that byte.
Gradient, on the oracle's s and rstd as given (rounded to fp32, u): n = s r is
off by 2 u, d = dy w by u; mean(d n) by (H + 4) u mean|d n|; so dx = r (d - n
mean) + dsum by 8 u (|r d| + |r n mean|) + (H + 4) u |r n| mean|d n| + 2 u |dsum|,
and 2^-8 |dx| more in bf16; dweight, a sum of T products, by (T + 4) u sum |dy n|."""
import numpy as np
import pytest
import torch

from fp4_quantized_moe_amd import _lib as Q
from oracle import layer_oracle as O
from oracle import mxfp4_oracle as MX

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16 = 2.0 ** -8
EPS = 1e-6


def host(t):
    return t.detach().double().cpu().numpy()


def make(seed, rows, cols, x_dtype, r_dtype, w_dtype):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    r = randn(rows, cols)
    r[:, ::37] *= 30.0
    x = (0.3 * randn(rows, cols)).to(x_dtype)
    return x, None if r_dtype is None else r.to(r_dtype), (1 + 0.2 * randn(cols)).to(w_dtype)


def check_quantized(q, y, e, rule):
    """q's codes and scales against values y that may be off by e, relative."""
    mx4 = isinstance(q, Q.MXFP4Tensor)
    codes, scales = q.codes.cpu().numpy(), q.scales.cpu().numpy()
    amax = np.abs(y.reshape(*y.shape[:-1], -1, 32)).max(-1)
    byte = (lambda a: MX.block_bytes(a, rule)) if mx4 else O.mxfp8_bytes
    assert (scales >= byte(amax * (1 - e))).all() and (scales <= byte(amax * (1 + e))).all()
    if mx4:
        codes = MX.unpack(codes)
    quantize = (lambda v: MX.quantize(v, rule, scales=scales)[0]) if mx4 else (lambda v: O.quantize_mxfp8(v, scales=scales)[0])
    assert (codes >= quantize(y * (1 - e))).all() and (codes <= quantize(y * (1 + e))).all()  # the sign is the top bit of both
    values = Q.dequantize_mxfp4(q) if mx4 else Q.dequantize_mxfp8(q)
    assert np.array_equal(host(values), MX.dequantize(codes, scales) if mx4 else O.dequantize_mxfp8(codes, scales))


bf, f32 = torch.bfloat16, torch.float32
# rows, cols: a wave a row (from 2048 rows on) and a workgroup a row, each with 1, 2, 4 and 8 units a lane, whole and partial
SIZES = [(1, 32), (1, 2048), (3, 16384), (5, 4128), (7, 8160), (333, 656), (2, 15008), (2048, 64), (2049, 544), (2050, 1056),
         (2051, 2048), (2048, 4096), (4099, 2080), (2048, 4128), (4, 16), (2500, 1072)]


@pytest.mark.parametrize("rows, cols", SIZES)
@pytest.mark.parametrize("types", [(bf, bf, bf), (f32, bf, f32), (bf, f32, bf), (f32, None, bf), (bf, None, f32)])
def test_norm(rows, cols, types):
    x, res, w = make(rows + cols, rows, cols, *types)
    quantize = Q.MXFP4 if (rows + (types[0] == f32)) % 2 else Q.MXFP8
    if cols % 32:
        quantize = None
    rule = "even" if quantize == Q.MXFP4 and rows % 3 else "floor"
    r = Q.rms_norm(x, w, res, eps=EPS, quantize=quantize, bf16=True, rule=rule, keep=True)
    if res is None:
        assert r.sum is x
    else:
        assert torch.equal(r.sum, (x.float() + res.float()).to(res.dtype))
    y, rstd = O.rms_norm(host(r.sum), host(w), EPS)
    e = (cols / 2 + 6) * U
    assert (np.abs(host(r.rstd) - rstd) <= e * rstd).all()
    assert (np.abs(host(r.y) - y) <= (BF16 + e) * np.abs(y)).all()
    if quantize is not None:
        check_quantized(r.q, y, e, rule)
    again = Q.rms_norm(x, w, res, eps=EPS, quantize=quantize, bf16=False, rule=rule)
    assert again.y is None and torch.equal(again.sum, r.sum)
    if quantize is not None:
        assert torch.equal(again.q.codes, r.q.codes) and torch.equal(again.q.scales, r.q.scales)


@pytest.mark.parametrize("quantize", [Q.MXFP4, Q.MXFP8])
@pytest.mark.parametrize("rows", [9, 2500])
def test_quantized_blocks_without_values(rows, quantize):
    """Rows of zeros, NaN and infinities, and weights of zero; the rows beside them are as alone."""
    x, res, w = make(5, rows, 512, bf, bf, bf)
    w[32:64] = 0
    plain = Q.rms_norm(x, w, res, quantize=quantize, bf16=True)
    x[1], res[1] = 0, 0
    x[3, 7] = float("nan")
    res[5, 200] = float("inf")
    r = Q.rms_norm(x, w, res, quantize=quantize, bf16=True)
    values = (Q.dequantize_mxfp4 if quantize == Q.MXFP4 else Q.dequantize_mxfp8)(r.q)
    assert (values[1] == 0).all() and (r.q.scales[1] == 0).all() and (r.y[1] == 0).all()
    assert r.y[3].isnan().all() and values[3].isnan().all() and (r.q.codes[3] == 0).all() and (r.q.scales[3] == 255).all()
    # an infinite sum of squares: r = 0, so the row is 0 but for the infinite element (inf * 0)
    assert r.y[5, 200].isnan() and (r.y[5, :200] == 0).all() and values[5, 192:224].isnan().all() and (values[5, :192] == 0).all()
    others = [i for i in range(rows) if i not in (1, 3, 5)]
    assert torch.equal(r.q.codes[others], plain.q.codes[others]) and torch.equal(r.y[others], plain.y[others])


@pytest.mark.parametrize("rows", [4, 3000])
def test_norm_in_place_and_eps(rows):
    x, res, w = make(6, rows, 1056, f32, bf, bf)
    want = Q.rms_norm(x, w, res, eps=0.5, keep=True)
    kept = res.clone()
    got = Q.rms_norm(x, w, res, eps=0.5, keep=True, out_sum=res)
    assert got.sum is res and torch.equal(res, want.sum) and torch.equal(got.y, want.y) and not torch.equal(res, kept)
    z = Q.rms_norm(torch.zeros_like(x), w, eps=0.0)  # 0 * inf
    assert z.y.isnan().all()


def test_norm_without_rows():
    x, res, w = make(7, 0, 64, bf, bf, bf)
    r = Q.rms_norm(x, w, res, quantize=Q.MXFP8, keep=True)
    assert r.q.codes.shape == (0, 64) and r.rstd.shape == (0,)
    dx, dw = Q.rms_norm_backward(x, r.sum, w, r.rstd)
    assert dx.shape == (0, 64) and (dw == 0).all()
    assert Q.dequantize_mxfp8(r.q).shape == (0, 64)


def test_mxfp8_every_code():
    """All 256 codes under all 256 scale bytes, in both types."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(256, 1).contiguous()
    scales = torch.arange(256, dtype=torch.uint8, device="cuda")[:, None].repeat(1, 8).contiguous()
    want = O.dequantize_mxfp8(codes.cpu().numpy(), scales.cpu().numpy())
    for dtype in (f32, bf):
        with np.errstate(over="ignore"):
            w = torch.from_numpy(want).to(dtype).double().numpy()  # infinities past the type's range
        got = host(Q.dequantize_mxfp8(Q.mxfp8_tensor(codes, scales), dtype))
        assert np.array_equal(got, w, equal_nan=True)
    batched = Q.mxfp8_tensor(codes.view(2, 128, 256), scales.view(2, 128, 8))
    assert batched.batch == 2 and Q.dequantize_mxfp8(batched).shape == (2, 128, 256)


@pytest.mark.parametrize("rows, cols", [(1, 16), (1, 2048), (3, 16384), (9, 4112), (333, 656), (17, 8176), (2048, 48), (2300, 528),
                                        (2051, 1040), (6000, 2048), (2048, 4096), (2049, 4112)])
@pytest.mark.parametrize("types", [(bf, bf, bf), (f32, bf, f32), (f32, f32, bf), (bf, f32, f32)])
def test_norm_backward(rows, cols, types):
    dy_type, s_type, w_type = types
    gen = torch.Generator(device="cuda").manual_seed(rows * 7 + cols)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    s, dy, dsum = randn(rows, cols).to(s_type), (0.1 * randn(rows, cols)).to(dy_type), (0.1 * randn(rows, cols)).to(s_type)
    w = (1 + 0.2 * randn(cols)).to(w_type)
    r64 = 1 / np.sqrt((host(s) ** 2).mean(1) + EPS)
    rstd = torch.from_numpy(r64).float().cuda()
    for extra in (dsum, None):
        dx, dweight = Q.rms_norm_backward(dy, s, w, rstd, dsum=extra)
        e = host(extra) if extra is not None else np.zeros((rows, cols))
        want, want_w = O.rms_norm_grad(host(dy), host(s), host(w), EPS, e)
        n, d, r = host(s) * r64[:, None], host(dy) * host(w), r64[:, None]
        mean, mean_abs = (d * n).mean(1, keepdims=True), np.abs(d * n).mean(1, keepdims=True)
        tol = 8 * U * (np.abs(r * d) + np.abs(r * n * mean)) + (cols + 4) * U * np.abs(r * n) * mean_abs + 2 * U * np.abs(e)
        if s_type == bf:
            tol += BF16 * (np.abs(want) + tol)
        assert (np.abs(host(dx) - want) <= tol).all()
        assert (np.abs(host(dweight) - want_w) <= (rows + 4) * U * np.abs(host(dy) * n).sum(0)).all()
    alone, none = Q.rms_norm_backward(dy, s, w, rstd, dsum=None, want_dweight=False)
    assert none is None and torch.equal(alone, dx)


@pytest.mark.parametrize("rows", [1, 127, 128, 129, 511, 513, 1023, 1024, 1025, 3000])
@pytest.mark.parametrize("cols", [16, 48, 64, 1072])
@pytest.mark.parametrize("dtype", [bf, f32])
def test_norm_backward_in_place(rows, cols, dtype):
    """dx written over dy, and over dsum: what the call with a dx of its own gives, and dweight of the dy that was there;
    rows around the number from which dweight's sums take a launch of their own.  Rows of NaN stay in their row."""
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    s, dy, dsum = (torch.randn(rows, cols, generator=gen, device="cuda").to(dtype) for _ in range(3))
    w = torch.rand(cols, generator=gen, device="cuda") + 0.5
    rstd = torch.rsqrt(s.float().square().mean(1) + EPS)
    dx, dweight = Q.rms_norm_backward(dy, s, w, rstd, dsum=dsum)
    n = host(s) * host(rstd)[:, None]
    assert (np.abs(host(dweight) - (host(dy) * n).sum(0)) <= (rows + 4) * U * np.abs(host(dy) * n).sum(0)).all()
    L, code = Q.load(), Q.F32 if dtype == f32 else Q.BF16
    nbytes = L.quads_rms_norm_backward_workspace_bytes(rows, cols)
    for target in (dy.clone(), dsum.clone()):
        over_dy = torch.equal(target, dy)
        ws, dw = torch.empty(nbytes + 16, dtype=torch.uint8, device="cuda"), torch.full((cols + 4,), 7.0, device="cuda")
        st = L.quads_rms_norm_backward(target.data_ptr() if over_dy else dy.data_ptr(), code, s.data_ptr(), code, w.data_ptr(), Q.F32,
                                       rstd.data_ptr(), dsum.data_ptr() if over_dy else target.data_ptr(), rows, cols,
                                       target.data_ptr(), dw.data_ptr(), ws.data_ptr(), nbytes, torch.cuda.current_stream().cuda_stream)
        assert st == 0 and torch.equal(target, dx) and torch.equal(dw[:cols], dweight) and (dw[cols:] == 7).all()
    if rows > 1:
        dy[rows // 2] = float("nan")
        bad, bad_w = Q.rms_norm_backward(dy, s, w, rstd, dsum=dsum)
        keep = torch.arange(rows, device="cuda") != rows // 2
        assert bad[rows // 2].isnan().all() and bad_w.isnan().all() and torch.equal(bad[keep], dx[keep])


def test_norm_gradient_is_the_forwards():
    """<dx, v> against a difference of the kernel's own fp32 forward, in a direction v: h = 2^-6 |s| leaves the cubic
    term; both sides of the 64-bit difference come from the oracle, so the kernel's sum is compared with O(h^2) alone."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    s, v = (torch.randn(4, 256, generator=gen, device="cuda") for _ in range(2))
    dy, w = torch.randn(4, 256, generator=gen, device="cuda"), torch.rand(256, generator=gen, device="cuda") + 0.5
    rstd = torch.rsqrt(s.double().square().mean(1) + EPS).float()
    dx, _ = Q.rms_norm_backward(dy, s, w, rstd)
    h = 1e-5
    f = lambda a: (O.rms_norm(a, host(w), EPS)[0] * host(dy)).sum()  # noqa: E731
    slope = (f(host(s) + h * host(v)) - f(host(s) - h * host(v))) / (2 * h)
    assert abs((host(dx) * host(v)).sum() - slope) <= 1e-5 * np.abs(host(dx) * host(v)).sum()


def test_norm_past_32_bit_offsets():
    """The last rows of a stream of more than 2^32 bytes."""
    rows, cols = 140000, 16384
    x = torch.zeros(rows, cols, dtype=bf, device="cuda")
    tail = make(8, 5, cols, bf, None, bf)
    x[-5:] = tail[0]
    got = Q.rms_norm(x, tail[2], quantize=Q.MXFP8, keep=True, bf16=True)
    want = Q.rms_norm(tail[0], tail[2], quantize=Q.MXFP8, keep=True, bf16=True)
    assert torch.equal(got.y[-5:], want.y) and torch.equal(got.q.codes[-5:], want.q.codes)
    assert torch.equal(got.q.scales[-5:], want.q.scales) and (got.y[:-5] == 0).all()
    dx, dw = Q.rms_norm_backward(got.y, x, tail[2], got.rstd)
    dx5, dw5 = Q.rms_norm_backward(want.y, tail[0], tail[2], want.rstd)
    assert torch.equal(dx[-5:], dx5)
    scale = (want.y.float() * tail[0].float() * want.rstd[:, None]).abs().sum(0)
    assert ((dw - dw5).abs() <= 16 * U * scale).all()  # sums of the same five terms in another order


def test_norm_checks_its_tensors():
    x, res, w = make(9, 4, 64, bf, bf, bf)
    for call, word in ((lambda: Q.rms_norm(x, w[:32]), "weight"), (lambda: Q.rms_norm(x, w, res[:2]), "residual must"),
                       (lambda: Q.rms_norm(x, w, quantize=7), "quantize must"), (lambda: Q.rms_norm(x, w, rule="even"), "for MXFP4"),
                       (lambda: Q.rms_norm(x, w, out_sum=res), "without a residual"),
                       (lambda: Q.rms_norm(x, w, res, out_sum=res.float()), "out_sum"),
                       (lambda: Q.rms_norm(x.t(), w), "contiguous"), (lambda: Q.rms_norm(x[:, :40].contiguous(), w[:40], quantize=Q.MXFP4), "multiple of 32"),
                       (lambda: Q.rms_norm(x, w, eps=-1.0), "eps"),
                       (lambda: Q.rms_norm_backward(x, x, w, torch.ones(3, device="cuda")), "do not match"),
                       (lambda: Q.rms_norm_backward(x, x, w, torch.ones(4, device="cuda"), dsum=x.float()), "dsum"),
                       (lambda: Q.mxfp8_tensor(torch.zeros(4, 64, dtype=torch.uint8, device="cuda"), torch.zeros(4, 3, dtype=torch.uint8, device="cuda")), "do not match")):
        with pytest.raises(Q.QuadsError, match=word):
            call()
