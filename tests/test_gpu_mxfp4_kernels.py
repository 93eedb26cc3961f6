"""Each kernel of the grouped MXFP4 product at sizes that the library says it
takes there (quads_moe_mxfp4_gemm_kernel, asserted for every case on the CPU):
the streaming kernel with several items a wave.

References are float64 products on the GPU of the operands' values (whose codec
test_gpu_mxfp4.py pins).  Tolerances, with u = 2^-24: K products exact in fp32
are off by at most K u sum |w x| in any order, to first order; a bf16 output by
half a step more, 2^-8 |y|.  h = silu(g) up from fp32 g: the argument of
2^(-g log2 e) is off by 1.23 |g| u (the constant and its product), exp2 and the
reciprocal by one ulp (2 u) each, the sum and two products by u each, so h by
(7 + 1.23 |g|) u |h|."""
import pytest
import torch

from fp4_quantized_moe_amd import _lib as Q

gpu = pytest.mark.gpu
U = 2.0 ** -24


def uneven(E, most, seed):
    """Rows per expert between 0 and `most`, none in every seventh."""
    n = torch.randint(0, most + 1, (E,), generator=torch.Generator().manual_seed(seed)).tolist()
    return [0 if e % 7 == 3 else c for e, c in enumerate(n)]


# rows per expert; N; K, all on the streaming kernel with several items a wave and experts of several row tiles.
# "once": at most 32 rows an expert on average (the weights are read once if routing is even); "again": more.
# K = 128, 256 are one stage (half of it zeros, and whole), 384 and 512 two, 640 three (the last half zeros), 1024 four;
# N = 2080 has an odd number of 32-column tiles.
STREAM = {
    "once, 1 half stage": (uneven(64, 70, 1), 4160, 128),
    "once, 1 stage": (uneven(60, 70, 2), 2048, 256),
    "once, 2 stages": (uneven(64, 70, 3), 2048, 384),
    "once, 3 stages": (uneven(40, 70, 4), 2080, 640),
    "once, 4 stages": (uneven(36, 64, 5), 2112, 1024),
    "once, all in one expert": ([0] * 70 + [1900] + [0] * 3, 2048, 256),
    "again, 1 half stage": (uneven(32, 120, 6), 8192, 128),
    "again, 2 stages": (uneven(32, 130, 7), 2048, 512),
    "again, 3 stages": (uneven(32, 130, 8), 2080, 640),
    "again, 4 stages": (uneven(32, 130, 9), 1024, 1024),
}
EPILOGUES = {"f32": (Q.EPI_NONE, torch.float32), "bf16": (Q.EPI_NONE, torch.bfloat16),
             "swiglu bf16": (Q.EPI_SWIGLU, torch.bfloat16), "swiglu mxfp4": (Q.EPI_SWIGLU, Q.MXFP4)}


def test_cases_reach_their_kernels():
    for name, (counts, N, K) in STREAM.items():
        R, E = sum(counts), len(counts)
        assert (R <= 32 * E) == name.startswith("once"), (name, R, E)
        for epi, (epilogue, dtype) in EPILOGUES.items():
            if epilogue == Q.EPI_NONE or N % 64 == 0:
                assert Q.mxfp4_gemm_kernel(R, E, N, K, epilogue, dtype) == "stream", (name, epi)
        assert sum(-(-c // 32) for c in counts) * -(-N // 64) > 1024, name  # more items than waves
        assert max(counts) > 32


def test_kernel_query():
    assert Q.mxfp4_gemm_kernel(0, 4, 64, 64) == "none"
    with pytest.raises(Q.QuadsError, match="K must"):
        Q.mxfp4_gemm_kernel(4, 4, 64, 48)
    with pytest.raises(Q.QuadsError, match="y_dtype"):
        Q.mxfp4_gemm_kernel(4, 4, 64, 64, Q.EPI_SWIGLU, torch.float32)


def offsets(counts):
    ends = [0]
    for c in counts:
        ends.append(ends[-1] + c)
    return ends, torch.tensor(ends, dtype=torch.int32, device="cuda")


def seeded(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def operands(seed, A, E, N, K):
    gen = seeded(seed)
    x = Q.quantize_mxfp4(torch.randn(A, K, generator=gen, device="cuda"))
    w = Q.quantize_mxfp4(torch.randn(E, N, K, generator=gen, device="cuda") * 0.05)
    return x, w


def values(q):
    return Q.dequantize_mxfp4(q, torch.float32)


def product(xv, wv, ends, token):
    """Rows xv[token] times their expert's wv^T in float64, and K u sum |w x|."""
    y = torch.zeros(ends[-1], wv.shape[1], dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(y)
    for e, (a, b) in enumerate(zip(ends[:-1], ends[1:])):
        if a < b:
            xe, we = xv[token[a:b].long()].double(), wv[e].double()
            y[a:b], tol[a:b] = xe @ we.T, xv.shape[1] * U * (xe.abs() @ we.abs().T)
    return y, tol


def check_block(q, h, err):
    """q must be a quantization of values within err of h: each scale byte between those of the largest magnitude
    -+ err, each value off by half a step of its place in the grid at most (by 2 units where 6 saturates)."""
    unit = torch.exp2(q.scales.double() - 127)
    top = h.abs().unflatten(1, (-1, 32))
    e = err.unflatten(1, (-1, 32))
    high, low = (top + e).amax(-1), (top - e).amax(-1)
    assert bool((high >= 4 * unit).logical_or(q.scales == 0).all()) and bool((low < 8 * unit).all())
    v = values(q).double()
    step = unit.repeat_interleave(32, 1)
    mag = h.abs() / step
    half = torch.where(mag <= 2, 0.25, torch.where(mag <= 4, 0.5, torch.where(mag <= 6, 1.0, 2.0))) * step
    assert bool(((v - h).abs() <= half + err).all())


@gpu
@pytest.mark.parametrize("name", STREAM)
def test_stream(name):
    counts, N, K = STREAM[name]
    ends, offs = offsets(counts)
    R, E = ends[-1], len(counts)
    x, w = operands(N + K, R // 2, E, N, K)
    token = torch.randint(0, R // 2, (R,), generator=seeded(K), device="cuda").to(torch.int32)
    want, tol = product(values(x), values(w).view(E, N, K), ends, token)
    y = Q.moe_mxfp4_gemm(x, w, offs, token)
    assert bool(((y.double() - want).abs() <= tol).all())
    assert torch.equal(Q.moe_mxfp4_gemm(x, w, offs, token, y_dtype=torch.bfloat16), y.to(torch.bfloat16))
    assert torch.equal(Q.moe_mxfp4_gemm(x, w, offs, token), y)
    if N % 64:
        return
    g, u = y.double().chunk(2, 1)  # the epilogue sees the same accumulators
    h = g * torch.sigmoid(g) * u
    err = (7 + 1.23 * g.abs()) * U * h.abs() + 2.0 ** -125
    got = Q.moe_mxfp4_gemm(x, w, offs, token, epilogue=Q.EPI_SWIGLU, y_dtype=torch.bfloat16).double()
    assert bool(((got - h).abs() <= err + 2.0 ** -8 * h.abs()).all())
    check_block(Q.moe_mxfp4_gemm(x, w, offs, token, epilogue=Q.EPI_SWIGLU, y_dtype=Q.MXFP4), h, err)


@gpu
@pytest.mark.parametrize("name", ["once, 1 stage", "once, 4 stages", "again, 1 half stage", "again, 4 stages"])
def test_stream_nan_and_rows_behind(name):
    """A NaN block stays in its row or column; rows behind the last expert are left as they were."""
    counts, N, K = STREAM[name]
    ends, offs = offsets(counts)
    R, E, behind = ends[-1], len(counts), 37
    assert Q.mxfp4_gemm_kernel(R + behind, E, N, K) == "stream"
    x, w = operands(N - K, R + behind, E, N, K)
    clean = Q.moe_mxfp4_gemm(x, w, offs, y=torch.zeros(R + behind, N, device="cuda"))
    last = max(e for e, c in enumerate(counts) if c)
    bad_rows, bad_col = [0, 31, 32, R - 1], N - 40
    for r in bad_rows:
        x.scales[r, K // 32 - 1] = 255
    w.scales.view(E, N, K // 32)[last, bad_col, 0] = 255
    y = torch.full((R + behind, N), 3.0, device="cuda")
    Q.moe_mxfp4_gemm(x, w, offs, y=y)
    nan = torch.zeros(R + behind, N, dtype=torch.bool, device="cuda")
    nan[bad_rows] = True
    nan[ends[last]:R, bad_col] = True
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
    hit[ends[last]:, (bad_col - N // 2) // 32] = True
    assert torch.equal(q.scales[:R] == 255, hit)
