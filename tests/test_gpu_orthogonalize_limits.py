"""GPU: orthogonalised updates of long thin matrices, and of more steps than a trainer takes.
Bit for bit and by the emulated roundings as in test_gpu_orthogonalize.py."""
import pytest
import torch

from fp4_quantized_moe_amd import _lib as Q
from test_gpu_orthogonalize import MUON, emulated, formula, gradient, relative, signs, whole_step

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("batch, rows, cols", [(2, 16, 1048560), (2, 1048560, 16), (300, 65536, 32), (17, 64, 262144), (17, 262144, 64)])
def test_batches_of_long_thin_matrices(batch, rows, cols):
    """Sides near 2^20, and batches whose longer sides' squares together pass 2^40 elements though the matrices do not."""
    g, p = signs(rows + cols, 2, rows, cols)
    want, largest = whole_step(g, 1.0, 1, -1)
    assert largest < 2 ** 11
    pick = torch.arange(batch) % 2
    want = (want / 2 ** p).to(torch.bfloat16).cuda()[pick]
    x = g.to(torch.bfloat16).cuda()[pick]
    got = Q.orthogonalize(x, steps=1, coefficients=(1.0, 4.0 ** p / 64, -(16.0 ** p) / 64), eps=0.0)
    assert torch.equal(got, want)


def with_singular_values(seed, rows, cols, s):
    """A matrix of the given singular values, the shorter side of them."""
    gen = torch.Generator().manual_seed(seed)
    side = lambda n: torch.linalg.qr(torch.randn(n, len(s), generator=gen, dtype=torch.float64))[0]  # noqa: E731
    return ((side(rows) * torch.tensor(s, dtype=torch.float64)) @ side(cols).T)[None].float()


def inputs(rows, cols):
    """Full rank, one direction ten and sixty times as loud as the others, a wide range, low ranks, and a norm of 1e-4 eps."""
    m = min(rows, cols)
    faint = gradient(8, 1, rows, cols, m)
    return {"gradient": gradient(1, 1, rows, cols, 4 * m), "random": torch.randn(1, rows, cols, generator=torch.Generator().manual_seed(2)),
            "loud": with_singular_values(3, rows, cols, [10.0] + [1.0] * (m - 1)),
            "louder": with_singular_values(3, rows, cols, [60.0] + [1.0] * (m - 1)),
            "wide": with_singular_values(4, rows, cols, [10.0 ** (-2 * i / m) for i in range(m)]),
            "tokens": gradient(5, 1, rows, cols, m // 3), "rank 16": gradient(6, 1, rows, cols, 16),
            "rank 1": gradient(7, 1, rows, cols, 1), "faint": faint / faint.norm() * 1e-11}


# By one workgroup, in slabs, and over tiles.
SIDES = [(96, 128), (64, 2048), (256, 512), (512, 256), (1024, 1040)]
STATED = {5: 4e-3, 10: 3e-2}  # of quads.h, before the result's rounding to bf16


@pytest.mark.parametrize("rows, cols", [(96, 128), (256, 512)])
def test_the_stated_error_covers_the_roundings(rows, cols):
    """quads.h's figures hold for the roundings that the kernel makes, carried through the steps on the CPU."""
    for name, g in inputs(rows, cols).items():
        for steps, stated in STATED.items():
            assert relative(emulated(g, steps, MUON, 1e-7), formula(g, steps, MUON, 1e-7)) <= stated, (name, steps)


@gpu
@pytest.mark.parametrize("rows, cols", SIDES)
def test_the_stated_error(rows, cols):
    """2^-8: half a step of the result's bf16."""
    for name, g in inputs(rows, cols).items():
        for steps, stated in STATED.items():
            want = formula(g.cuda(), steps, MUON, 1e-7)
            got = relative(Q.orthogonalize(g.cuda(), steps=steps), want)
            assert got <= stated + 2.0 ** -8, (name, steps, got)


@gpu
@pytest.mark.parametrize("rows, cols", SIDES)
@pytest.mark.parametrize("steps", [8, 9, 10])
def test_many_steps_as_far_as_their_roundings(rows, cols, steps):
    """Three times the emulated roundings' distance, for roundings of other signs, and bf16's half step."""
    for name, g in inputs(rows, cols).items():
        g = g.cuda()
        want = formula(g, steps, MUON, 1e-7)
        bound = 3 * relative(emulated(g, steps, MUON, 1e-7), want) + 2.0 ** -8
        got = relative(Q.orthogonalize(g, steps=steps), want)
        assert got <= bound < 0.1, (name, got, bound)


@gpu
def test_coefficients_are_three():
    g = torch.randn(2, 32, 48, device="cuda")
    for bad in ((), (1.0, 2.0), (1.0, 2.0, 3.0, 4.0)):
        with pytest.raises(Q.QuadsError, match="coefficients must be three"):
            Q.orthogonalize(g, coefficients=bad)
    assert torch.equal(Q.orthogonalize(g, coefficients=list(MUON)), Q.orthogonalize(g))
