"""Each kernel of the grouped MXFP4 product at sizes that the library says it
takes there (quads_moe_mxfp4_gemm_kernel, asserted for every case on the CPU):
the streaming kernel with several items a wave, and every kernel past 32-bit
offsets, on two streams at once and in a replayed graph.

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

# num_rows, experts, N, K of far operands by the kernel that takes them
FAR_ROWS = {"direct": (40, 2, 256, 2048), "stream": (200, 8, 4096, 2048), "staged_small": (200, 2, 8192, 2048),
            "staged_large": (700, 2, 16384, 2048)}
FAR_ROWS_ODD = {"direct": (40, 2, 256, 2080), "staged_small": (200, 2, 8192, 2080), "staged_large": (700, 2, 16384, 2080)}
FAR_WEIGHTS = {"stream": (40, 130, 32768, 2048), "staged_small": (5200, 130, 32768, 2048),
               "staged_large": (5200, 18, 131072, 4096)}
BLOCKS = {"stream": (2000, 64, 1024, 1024), "staged_small": (4000, 32, 2048, 1024), "staged_large": (6000, 16, 2048, 2048)}


def test_cases_reach_their_kernels():
    for name, (counts, N, K) in STREAM.items():
        R, E = sum(counts), len(counts)
        assert (R <= 32 * E) == name.startswith("once"), (name, R, E)
        for epi, (epilogue, dtype) in EPILOGUES.items():
            if epilogue == Q.EPI_NONE or N % 64 == 0:
                assert Q.mxfp4_gemm_kernel(R, E, N, K, epilogue, dtype) == "stream", (name, epi)
        assert sum(-(-c // 32) for c in counts) * -(-N // 64) > 1024, name  # more items than waves
        assert max(counts) > 32
    for table in (FAR_ROWS, FAR_ROWS_ODD, FAR_WEIGHTS):
        for kernel, sizes in table.items():
            assert Q.mxfp4_gemm_kernel(*sizes) == kernel, sizes
    for kernel, (R, E, H, I) in BLOCKS.items():
        assert Q.mxfp4_gemm_kernel(R, E, 2 * I, H, Q.EPI_SWIGLU, Q.MXFP4) == kernel
        assert Q.mxfp4_gemm_kernel(R, E, H, I, Q.EPI_NONE, torch.float32) == kernel


def test_kernel_query():
    assert Q.mxfp4_gemm_kernel(0, 4, 64, 64) == "none"
    with pytest.raises(Q.QuadsError, match="K must"):
        Q.mxfp4_gemm_kernel(4, 4, 64, 48)
    with pytest.raises(Q.QuadsError, match="y_dtype"):
        Q.mxfp4_gemm_kernel(4, 4, 64, 64, Q.EPI_SWIGLU, torch.float32)
    with pytest.raises(Q.QuadsError, match="y_dtype"):
        Q.mxfp4_gemm_kernel(4, 4, 64, 64, y_dtype=torch.float16)
    assert Q.load().quads_moe_mxfp4_gemm_kernel(None) == -1


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


def far_rows(R, E, N, K):
    """R rows at the end of a table whose codes pass 2^32 bytes, against 64-bit products."""
    rows = 2 ** 32 // (K // 2) + R + 5
    part, w = operands(R + K, R, E, N, K)
    x = Q.empty_mxfp4(1, rows, K, "cuda")
    x.codes.zero_()
    x.scales.fill_(127)
    x.codes[-R:], x.scales[-R:] = part.codes, part.scales
    assert (rows - R) * (K // 2) >= 2 ** 32
    # the last row first: the far end of the ids too
    token = torch.arange(rows - 1, rows - R - 1, -1, dtype=torch.int32, device="cuda")
    ends, offs = offsets([R // E] * (E - 1) + [R - R // E * (E - 1)])
    want, tol = product(values(part), values(w).view(E, N, K), ends, (token - (rows - R)))
    y = Q.moe_mxfp4_gemm(x, w, offs, token)
    assert bool(((y.double() - want).abs() <= tol).all())


@gpu
@pytest.mark.parametrize("kernel", FAR_ROWS)
def test_rows_past_32_bits(kernel):
    far_rows(*FAR_ROWS[kernel])


@gpu
@pytest.mark.parametrize("kernel", FAR_ROWS_ODD)
def test_rows_past_32_bits_odd_scales(kernel):
    far_rows(*FAR_ROWS_ODD[kernel])


@gpu
@pytest.mark.parametrize("kernel", FAR_WEIGHTS)
def test_weights_past_32_bits(kernel):
    """Weights whose codes pass 2^32 bytes; rows for the last two experts alone."""
    R, E, N, K = FAR_WEIGHTS[kernel]
    x, tail = operands(R, R, 2, N, K)
    w = Q.empty_mxfp4(E, N, K, "cuda")
    w.codes.zero_()
    w.scales.fill_(127)
    w.codes[-2:], w.scales[-2:] = tail.codes, tail.scales
    assert (E - 2) * N * (K // 2) >= 2 ** 32
    ends, offs = offsets([0] * (E - 2) + [R // 3, R - R // 3])
    y = Q.moe_mxfp4_gemm(x, w, offs)
    xv, wv = values(x), values(tail).view(2, N, K)
    for e, (a, b) in enumerate(zip(ends[-3:-1], ends[-2:])):
        for i in range(a, b, 1024):
            j = min(b, i + 1024)
            want, tol = product(xv[i:j], wv[e:e + 1], [0, j - i], torch.arange(j - i, device="cuda"))
            assert bool(((y[i:j].double() - want).abs() <= tol).all()), (e, i)


def block(kernel):
    R, E, H, I = BLOCKS[kernel]
    gen = seeded(R)
    counts = [R // E] * E
    counts[1] += counts[0] - 1
    counts[0] = 1
    counts[-1] += R - sum(counts)
    ends, offs = offsets(counts)
    wg = Q.quantize_mxfp4(torch.randn(E, 2 * I, H, generator=gen, device="cuda") * 0.05)
    wd = Q.quantize_mxfp4(torch.randn(E, H, I, generator=gen, device="cuda") * 0.05)
    token = torch.randint(0, R // 2, (R,), generator=gen, device="cuda").to(torch.int32)
    xs = [torch.randn(R // 2, H, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2)]
    return xs, wg, wd, ends, offs, token


@gpu
@pytest.mark.parametrize("kernel", BLOCKS)
def test_two_streams_and_replays(kernel):
    """Two blocks in flight on two streams, and one captured and replayed between eager calls, each with its own
    output and workspace; one of them against 64-bit products."""
    xs, wg, wd, ends, offs, token = block(kernel)
    R, E, H, I = BLOCKS[kernel]
    want = [Q.moe_mxfp4_ffn(x, wg, wd, offs, token) for x in xs]
    xq = Q.quantize_mxfp4(xs[0])
    gu, tol = product(values(xq), values(wg).view(E, 2 * I, H), ends, token)
    pre = Q.moe_mxfp4_gemm(xq, wg, offs, token)
    assert bool(((pre.double() - gu).abs() <= tol).all())
    g, u = pre.double().chunk(2, 1)
    hv = g * torch.sigmoid(g) * u
    h = Q.moe_mxfp4_gemm(xq, wg, offs, token, epilogue=Q.EPI_SWIGLU, y_dtype=Q.MXFP4)
    check_block(h, hv, (7 + 1.23 * g.abs()) * U * hv.abs() + 2.0 ** -125)
    y, tol = product(values(h), values(wd).view(E, H, I), ends, torch.arange(R, device="cuda"))
    assert bool(((want[0].double() - y).abs() <= tol).all())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(4):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k] = Q.moe_mxfp4_ffn(xs[k], wg, wd, offs, token)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    x, out = xs[0].clone(), torch.empty_like(want[0])
    ws = torch.empty(Q.mxfp4_ffn_workspace_bytes(R // 2, R, H, I), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.moe_mxfp4_ffn(x, wg, wd, offs, token, y=out, ws=ws)
    for k in (0, 1, 1, 0):
        x.copy_(xs[k])
        out.zero_()
        graph.replay()
        assert torch.equal(Q.moe_mxfp4_ffn(xs[1 - k], wg, wd, offs, token), want[1 - k])
        torch.cuda.synchronize()
        assert torch.equal(out, want[k])
