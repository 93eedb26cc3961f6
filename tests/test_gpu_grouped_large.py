"""The MXFP4 and gated products at sizes where a workgroup runs many tiles, many
experts are empty or offsets pass 32 bits, against float64 products on the GPU
of the operands' values (whose codec test_gpu_mxfp4.py pins).

Tolerances: K products exact in fp32 are off by at most K 2^-24 sum |w x| in
any order, to first order; a bf16 output by half a step more, 2^-8 |y|."""
import pytest
import torch

from fp4_quantized_moe_amd import _lib as Q

pytestmark = pytest.mark.gpu


def counts_of(kind, E, R, gen):
    """Rows per expert: even, a few loud experts, or all in the last."""
    if kind == "even":
        n = torch.full((E,), R // E)
    elif kind == "skewed":
        p = 1.0 / torch.arange(1, E + 1).double() ** 1.5
        n = (p / p.sum() * R).long()[torch.randperm(E, generator=gen)]
    else:
        n = torch.zeros(E, dtype=torch.long)
        n[-1] = R
    return n


def grouping(kind, E, R, A, seed=0):
    gen = torch.Generator().manual_seed(seed)
    n = counts_of(kind, E, R, gen)
    offs = torch.cat((torch.zeros(1, dtype=torch.long), n.cumsum(0)))
    token = torch.randint(0, A, (int(offs[-1]),), generator=gen)
    return offs.tolist(), offs.to(torch.int32).cuda(), token.to(torch.int32).cuda()


def check(y, x, w, ends, token, K):
    """y against x[token] w^T per expert (w, x float64 values; w(e) on demand)."""
    half = 2.0 ** -8 if y.dtype == torch.bfloat16 else 0.0
    for e, (a, b) in enumerate(zip(ends[:-1], ends[1:])):
        for i in range(a, b, 4096):
            j = min(b, i + 4096)
            xe, we = x[token[i:j].long()], w(e)
            want = xe @ we.T
            tol = K * 2.0 ** -24 * (xe.abs() @ we.abs().T) + half * want.abs()
            assert bool(((y[i:j].double() - want).abs() <= tol).all()), (e, i)


# 256-row tiles many to a workgroup, with stages 1 (padded to 2), 2, 3, 8; odd column counts; one 128-row case
CASES = [
    ("skewed", 8, 30000, 1536, 256), ("even", 64, 64 * 520, 768, 512), ("last", 3, 20000, 2080, 768),
    ("skewed", 16, 40000, 1024, 2048), ("skewed", 300, 30000, 544, 384), ("even", 128, 128 * 70, 576, 640),
    # scale rows that no dword fits: 5, 9, 27 and 33 blocks a row
    ("skewed", 8, 30000, 1536, 160), ("last", 3, 20000, 2080, 288), ("even", 64, 64 * 520, 768, 864), ("even", 40, 40 * 70, 448, 1056),
]


@pytest.mark.parametrize("kind, E, R, N, K", CASES)
def test_mxfp4(kind, E, R, N, K):
    ends, offs, token = grouping(kind, E, R, 5000)
    gen = torch.Generator(device="cuda").manual_seed(N)
    x = Q.quantize_mxfp4(torch.randn(5000, K, generator=gen, device="cuda"))
    w = Q.quantize_mxfp4(torch.randn(E, N, K, generator=gen, device="cuda") * 0.02)
    xv, wv = Q.dequantize_mxfp4(x, torch.float32).double(), Q.dequantize_mxfp4(w, torch.float32).view(E, N, K)
    y = Q.moe_mxfp4_gemm(x, w, offs, token)
    check(y, xv, lambda e: wv[e].double(), ends, token, K)
    assert torch.equal(Q.moe_mxfp4_gemm(x, w, offs, token, y_dtype=torch.bfloat16), y.to(torch.bfloat16))
    assert torch.equal(Q.moe_mxfp4_gemm(x, w, offs, token), y)
    if N % 64:
        return
    # the SwiGLU epilogue sees the same accumulators: h is silu(g) u of y's columns, to a few fp32 ulp
    g, u = y.double().chunk(2, 1)
    want = g * torch.sigmoid(g) * u
    h = Q.moe_mxfp4_gemm(x, w, offs, token, epilogue=Q.EPI_SWIGLU, y_dtype=torch.bfloat16).double()
    assert bool(((h - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want.abs() + 1e-37).all())
    # and requantized, each value is off by at most half a step of the block's grid (a quarter where it saturates)
    q = Q.moe_mxfp4_gemm(x, w, offs, token, epilogue=Q.EPI_SWIGLU, y_dtype=Q.MXFP4)
    v = Q.dequantize_mxfp4(q, torch.float32).double()
    unit = torch.exp2(q.scales.double() - 127).repeat_interleave(32, 1)
    assert bool(((v - want).abs() <= (2.0 + 2.0 ** -18) * unit).all())
    block = want.abs().view(want.shape[0], -1, 32).amax(-1)
    assert bool((block < 8 * (1 + 2.0 ** -18) * torch.exp2(q.scales.double() - 127) + 1e-37).all())
    again = Q.quantize_mxfp4(want.float().contiguous())  # equal but where fp32 silu crosses a rounding point
    assert float((again.codes != q.codes).float().mean()) < 1e-3


@pytest.mark.parametrize("kind, E, R, H, I", [
    ("even", 32, 32 * 520, 512, 512), ("skewed", 8, 30000, 64, 272), ("last", 5, 10000, 192, 1040),
    ("skewed", 200, 20000, 128, 128), ("even", 64, 64 * 60, 320, 192),
    # 256-row tiles in the forward too, of 1, 3, 17 and 2 stages, with last tiles above and below 128 rows
    ("skewed", 16, 4900, 64, 880), ("even", 16, 16 * 310, 192, 896), ("skewed", 16, 4900, 1088, 864), ("last", 3, 6000, 128, 1040)])
def test_gated(kind, E, R, H, I):
    ends, offs, token = grouping(kind, E, R, 4000)
    gen = torch.Generator(device="cuda").manual_seed(H)
    x = torch.randn(4000, H, generator=gen, device="cuda").to(torch.bfloat16)
    w = (torch.randn(E, 2 * I, H, generator=gen, device="cuda") * H ** -0.5).to(torch.bfloat16)
    h, gu = Q.moe_gated_forward(x, w, offs, token)
    check(gu, x.double(), lambda e: w[e].double(), ends, token, H)
    R = ends[-1]
    dy = torch.randn(R, H, generator=gen, device="cuda").to(torch.bfloat16)
    wd = (torch.randn(E, H, I, generator=gen, device="cuda") * 0.05).to(torch.bfloat16)
    dgu = Q.moe_gated_backward(dy, wd, gu, offs).double()
    g, u = gu.double().chunk(2, 1)
    s = torch.sigmoid(g)
    for e, (a, b) in enumerate(zip(ends[:-1], ends[1:])):
        if a == b:
            continue
        d, m = dy[a:b].double() @ wd[e].double(), dy[a:b].double().abs() @ wd[e].double().abs()
        for got, f, size in ((dgu[a:b, :I], u[a:b] * s[a:b] * (1 + g[a:b] * (1 - s[a:b])), u[a:b].abs() * s[a:b] * (1 + g[a:b].abs())),
                             (dgu[a:b, I:], g[a:b] * s[a:b], g[a:b].abs() * s[a:b])):
            want = d * f
            tol = H * 2.0 ** -24 * m * size + 2.0 ** -20 * d.abs() * size + 2.0 ** -8 * want.abs() + 1e-37
            assert bool(((got - want).abs() <= tol).all()), e


@pytest.mark.parametrize("rows, R", [(4_300_000, 40), (4_300_000, 700)])
def test_offsets_past_32_bits(rows, R):
    """Activation rows whose bytes and outputs whose elements lie past 2^32: few rows (the streaming kernels)
    and many (the staged one) of the far end of a long table."""
    K, N, E = 2048, 256, 2
    x = Q.empty_mxfp4(1, rows, K, "cuda")  # 4.4 GB of codes
    x.codes.zero_()
    x.scales.fill_(127)
    part = Q.quantize_mxfp4(torch.randn(R, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)))
    x.codes[-R:], x.scales[-R:] = part.codes, part.scales
    w = Q.quantize_mxfp4(torch.randn(E, N, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)))
    token = torch.arange(rows - R, rows, dtype=torch.int32, device="cuda")
    offs = torch.tensor([0, R // 2, R], dtype=torch.int32, device="cuda")
    near = Q.moe_mxfp4_gemm(part, w, offs)
    assert torch.equal(Q.moe_mxfp4_gemm(x, w, offs, token), near)
    assert float(near.abs().max()) > 0


def test_outputs_past_32_bits():
    """More than 2^32 output elements: the last rows equal the same rows computed alone."""
    R, K, N = 2_200_000, 128, 2048
    x = Q.quantize_mxfp4(torch.randn(1000, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)))
    w = Q.quantize_mxfp4(torch.randn(1, N, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)))
    token = (torch.arange(R, device="cuda") % 1000).to(torch.int32)
    offs = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    y = Q.moe_mxfp4_gemm(x, w, offs, token, y_dtype=torch.bfloat16)
    alone = Q.moe_mxfp4_gemm(x, w, torch.tensor([0, 1000], dtype=torch.int32, device="cuda"), y_dtype=torch.bfloat16)
    for a in (0, R // 2 // 1000 * 1000, R - 1000):
        assert torch.equal(y[a:a + 1000], alone)


def test_most_experts():
    """1024 experts, most without rows; single rows in the first and the last."""
    E, N, K = 1024, 64, 128
    gen = torch.Generator(device="cuda").manual_seed(5)
    w = Q.quantize_mxfp4(torch.randn(E, N, K, generator=gen, device="cuda"))
    wv = Q.dequantize_mxfp4(w, torch.float32).view(E, N, K)
    for counts in ({0: 1, 1023: 1}, {64: 40, 65: 3, 700: 129}, {i: 1 + i % 3 for i in range(0, 1024, 5)}):
        n = torch.zeros(E, dtype=torch.long)
        for e, c in counts.items():
            n[e] = c
        offs = torch.cat((torch.zeros(1, dtype=torch.long), n.cumsum(0)))
        R = int(offs[-1])
        x = Q.quantize_mxfp4(torch.randn(R, K, generator=gen, device="cuda"))
        y = Q.moe_mxfp4_gemm(x, w, offs.to(torch.int32).cuda())
        check(y, Q.dequantize_mxfp4(x, torch.float32).double(), lambda e: wv[e].double(), offs.tolist(),
              torch.arange(R, device="cuda"), K)


def test_two_streams_at_once():
    """Two blocks in flight on two streams, each with its own output and workspace."""
    ends, offs, token = grouping("skewed", 16, 6000, 1500)
    gen = torch.Generator(device="cuda").manual_seed(6)
    xs = [torch.randn(1500, 512, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2)]
    wg = Q.quantize_mxfp4(torch.randn(16, 512, 512, generator=gen, device="cuda") * 0.05)
    wd = Q.quantize_mxfp4(torch.randn(16, 512, 256, generator=gen, device="cuda") * 0.05)
    want = [Q.moe_mxfp4_ffn(x, wg, wd, offs, token) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k] = Q.moe_mxfp4_ffn(xs[k], wg, wd, offs, token)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("K", [448, 512, 1088])
def test_nan_and_rows_behind_the_last_expert_staged(K):
    """At sizes that go through the staged kernel: a NaN block stays in its row or column, rows behind the last
    expert are left as they were."""
    R, N, behind = 40000, 256, 77
    gen = torch.Generator(device="cuda").manual_seed(K)
    x = Q.quantize_mxfp4(torch.randn(R + behind, K, generator=gen, device="cuda"))
    w = Q.quantize_mxfp4(torch.randn(1, N, K, generator=gen, device="cuda"))
    offs = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    clean = Q.moe_mxfp4_gemm(x, w, offs)
    bad_rows, bad_col = [0, 255, 256, 39999], 200
    for r in bad_rows:
        x.scales[r, K // 32 - 1] = 255
    w.scales.view(N, K // 32)[bad_col, 0] = 255
    y = torch.full((R + behind, N), 3.0, device="cuda")
    Q.moe_mxfp4_gemm(x, w, offs, y=y)
    nan = torch.zeros(R + behind, N, dtype=torch.bool, device="cuda")
    nan[bad_rows] = True
    nan[:R, bad_col] = True
    assert torch.equal(torch.isnan(y), nan)
    assert bool((y[R:] == 3.0).all())
    assert torch.equal(y[:R][~nan[:R]], clean[:R][~nan[:R]])
    q = Q.empty_mxfp4(1, R + behind, N // 2, "cuda")
    q.codes.fill_(0x5A)
    q.scales.fill_(0x77)
    Q.moe_mxfp4_gemm(x, w, offs, epilogue=Q.EPI_SWIGLU, y_dtype=Q.MXFP4, y=q)
    assert bool((q.codes[R:] == 0x5A).all()) and bool((q.scales[R:] == 0x77).all())
    hit = torch.zeros(R, N // 64, dtype=torch.bool, device="cuda")
    hit[bad_rows] = True
    hit[:, (bad_col - N // 2) // 32] = True  # the up column's block of h
    assert torch.equal(q.scales[:R] == 255, hit)


def test_gated_rows_behind_the_last_expert_staged():
    R, H, I, behind = 20000, 128, 144, 50
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(R + behind, H, generator=gen, device="cuda").to(torch.bfloat16)
    w = torch.randn(2, 2 * I, H, generator=gen, device="cuda").to(torch.bfloat16)
    offs = torch.tensor([0, 137, R], dtype=torch.int32, device="cuda")
    h, gu = Q.moe_gated_forward(x, w, offs)
    h2, gu2 = Q.moe_gated_forward(x[:R].contiguous(), w, offs)
    assert torch.equal(h[:R], h2) and torch.equal(gu[:R], gu2)
    gu[R:] = 1.0
    dgu = torch.full_like(gu, 5.0)
    Q.moe_gated_backward(x, torch.randn(2, H, I, generator=gen, device="cuda").to(torch.bfloat16), gu, offs, dgu=dgu)
    assert bool((dgu[R:] == 5.0).all()) and not bool((dgu[:R] == 5.0).any(1).all())


def test_quantize_past_32_bits_of_lanes():
    """2^34 elements are 2^31 lanes of 8: a launch's most.  Slices around the
    seam and at both ends against the same slices quantized alone."""
    n = 2 ** 34 + 4096
    x = torch.zeros(n // 32, 32, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    seam = 2 ** 34 // 32
    parts = [slice(0, 64), slice(2 ** 31 // 32 - 32, 2 ** 31 // 32 + 32), slice(seam - 64, seam + 64), slice(n // 32 - 40, n // 32)]
    for p in parts:
        x[p] = torch.randn(x[p].shape, generator=gen, device="cuda").bfloat16()
    q = Q.quantize_mxfp4(x)
    back = Q.dequantize_mxfp4(q)
    for p in parts:
        alone = Q.quantize_mxfp4(x[p].contiguous())
        assert torch.equal(q.codes[p], alone.codes) and torch.equal(q.scales[p], alone.scales), p
        assert torch.equal(back[p], Q.dequantize_mxfp4(alone)), p
    assert int(q.scales.count_nonzero()) <= sum(p.stop - p.start for p in parts)
    del back
    out, _ = Q.weight_qdq_mxfp4(x)
    for p in parts:
        assert torch.equal(out[p], Q.weight_qdq_mxfp4(x[p].contiguous())[0]), p
