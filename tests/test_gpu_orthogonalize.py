"""GPU: orthogonalised updates.

One step is tested bit for bit: G has 4^p entries of +-1 and the rest 0, so
|G|_F = 2^p and X = G / 2^p; with b = beta 4^p 2^-6 and c = gamma 16^p 2^-6 the
matrix b A + c A^2 is 2^-6 times whole numbers, which fp16 holds below 2^11 (the
test asserts it of its inputs), all sums are whole numbers below 2^24, and the
only rounding is the one to bf16.

Several steps are tested against the 64-bit oracle in the 2-norm.  Their error
is that of the roundings stated in quads.h, carried through the steps; how far
they reach depends on the singular values, so the test carries them itself: the
formula in fp32 on the CPU or GPU with X, A and B rounded as stated.  Roundings
of other signs reach as far: three times its distance from the formula is
allowed, and half a step of bf16, 2^-8, for the output."""
import numpy as np
import pytest
import torch

from fp4_quantized_moe_amd import _lib as Q
from oracle import layer_oracle as O

gpu = pytest.mark.gpu
MUON = (3.4445, -4.7750, 2.0315)


def signs(seed, batch, rows, cols):
    """[batch, rows, cols] with 4^p entries of +-1 in each matrix, about 12 in a row of the longer side at most."""
    gen = torch.Generator().manual_seed(seed)
    n = rows * cols
    p = 1
    while 4 ** (p + 1) <= min(n, 12 * min(rows, cols)):
        p += 1
    g = torch.zeros(batch, n)
    for m in g:
        at = torch.randperm(n, generator=gen)[:4 ** p]
        m[at] = torch.randint(0, 2, (4 ** p,), generator=gen).float() * 2 - 1
    return g.view(batch, rows, cols), p


def whole_step(g, a, beta, gamma):
    """The step's result in whole numbers times 2^-6 (times 2^-p), and the largest whole number on the way."""
    x = g.double()
    left = x.shape[1] <= x.shape[2]
    s = x @ x.transpose(1, 2) if left else x.transpose(1, 2) @ x
    b = beta * s + gamma * s @ s
    y = 64 * a * x + (b @ x if left else x @ b)
    return y / 64, max(s.abs().max().item(), b.abs().max().item())


# batch, rows, cols: both tiles of the kernel, one tile and several of a matrix, rows and columns that fill no tile, contractions
# of less than a stage, of a part of one and of several, wide, tall and square
STEP = [(1, 16, 16), (3, 16, 80), (3, 80, 16), (2, 64, 64), (5, 48, 144), (2, 128, 128), (1, 144, 272), (1, 272, 144), (7, 128, 512),
        (2, 656, 272), (12, 272, 656), (1, 400, 400), (1, 16, 4112), (1, 4112, 16), (40, 256, 512), (64, 512, 272), (40, 528, 784),
        (33, 784, 528), (20, 1040, 1040), (600, 32, 48)]


@gpu
@pytest.mark.parametrize("batch, rows, cols", STEP)
@pytest.mark.parametrize("step", [(0.0, 1, 0), (0.0, 0, 1), (1.0, 1, -1)])
def test_one_step_bit_for_bit(batch, rows, cols, step):
    g, p = signs(rows + cols, min(batch, 3), rows, cols)
    a, beta, gamma = step
    want, largest = whole_step(g, a, beta, gamma)
    assert largest < 2 ** 11
    pick = torch.arange(batch) % len(g)
    want = (want / 2 ** p).to(torch.bfloat16).cuda()[pick]
    coefficients = (a, beta * 4.0 ** p / 64, gamma * 16.0 ** p / 64)
    for dtype in (torch.float32, torch.bfloat16):
        x = g.cuda()[pick].to(dtype)
        got = Q.orthogonalize(x, steps=1, coefficients=coefficients, eps=0.0)
        assert torch.equal(got, want), (dtype, (got != want).sum().item())
    # a power of two in front of g leaves X as it is
    assert torch.equal(Q.orthogonalize(x.float() * 2.0 ** 80, steps=1, coefficients=coefficients, eps=0.0), want)
    assert torch.equal(Q.orthogonalize(x.float() * 2.0 ** -100, steps=1, coefficients=coefficients, eps=0.0), want)


# Both sides of the sizes that one workgroup holds, and of those of which five, two and one fit a CU.
SMALL = [(16, 16), (32, 32), (32, 224), (32, 240), (16, 608), (32, 624), (32, 1248), (32, 1264), (48, 48), (64, 64), (64, 80), (48, 256),
         (64, 272), (64, 576), (64, 592), (96, 96), (96, 128), (80, 144), (96, 352), (96, 368), (128, 128), (112, 224), (128, 224), (128, 240),
         (144, 144)]
SMALL += [(c, r) for r, c in SMALL if r != c]


@gpu
@pytest.mark.parametrize("rows, cols", SMALL)
def test_small_matrices(rows, cols):
    for step in ((0.0, 1, 0), (0.0, 0, 1), (1.0, 1, -1)):
        test_one_step_bit_for_bit(3, rows, cols, step)
    test_steps_that_keep_the_matrix(2, rows, cols)
    test_several_steps(3, rows, cols, 2 * min(rows, cols), torch.float32)
    test_several_steps(2, rows, cols, max(4, min(rows, cols) // 4), torch.bfloat16)


# Long matrices in slabs of columns: both sides of the sizes and batches that take them, whole and partial last slabs.
@gpu
@pytest.mark.parametrize("batch, rows, cols", [(2, 32, 2048), (3, 16, 8192), (1, 16, 8208), (2, 64, 4096), (1, 64, 4112), (2, 48, 640), (300, 64, 592),
                                               (1, 96, 2048), (1, 96, 2064), (32, 96, 512), (33, 96, 512), (2, 128, 240), (64, 112, 256),
                                               (65, 112, 256), (1, 128, 1040)])
def test_slabs(batch, rows, cols):
    for r, c in ((rows, cols), (cols, rows)):
        for step in ((0.0, 1, 0), (1.0, 1, -1)):
            test_one_step_bit_for_bit(batch, r, c, step)
        test_several_steps(min(batch, 40), r, c, max(4, rows // 4), torch.float32)
        test_several_steps(batch, r, c, 2 * rows, torch.bfloat16)


@gpu
def test_many_small_matrices():
    """More matrices than the card holds workgroups; each has the bits that it has alone, on the side of other values."""
    for rows, cols in ((32, 96), (96, 32), (128, 208)):
        g = gradient(9, 3000, rows, cols, 40, "cuda")
        g[7], g[8, 3, 5] = 0, float("nan")
        got = Q.orthogonalize(g)
        assert (got[7] == 0).all() and got[8].isnan().all() and got[9:].isfinite().all()
        for i in (0, 6, 9, 1500, 2999):
            assert torch.equal(Q.orthogonalize(g[i]), got[i])
        assert relative(got[9:40], formula(g[9:40], 5, MUON, 1e-7)) <= 3 * relative(emulated(g[9:40], 5, MUON, 1e-7), formula(g[9:40], 5, MUON, 1e-7)) + 2.0 ** -8


@gpu
@pytest.mark.parametrize("batch, rows, cols", [(2, 64, 96), (2, 96, 64), (6, 272, 400), (6, 400, 272), (70, 512, 528), (70, 528, 512)])
def test_steps_that_keep_the_matrix(batch, rows, cols):
    """a = 1, b = c = 0 gives X back: to 22 bits through hi + lo in one step, to fp16's 11 where the last step's X is hi alone."""
    g = torch.randn(batch, rows, cols, generator=torch.Generator().manual_seed(1))
    x = g.double() / (g.double().square().sum((1, 2), keepdim=True).sqrt())
    for steps in (1, 2, 3):
        got = Q.orthogonalize(g.cuda(), steps=steps, coefficients=(1.0, 0.0, 0.0), eps=0.0).cpu()
        # half a step of the output's bf16, 2^-8 relative; X's own rounding leaves 2^-20 of it, or 2^-35 where lo is subnormal
        # (2^-25 of 2^11); hi alone half a step of fp16, 2^-11, or 2^-36
        own = 2.0 ** -20 if steps == 1 else 2.0 ** -11 + 2.0 ** -20
        assert ((got.double() - x).abs() <= (2.0 ** -8 + own) * x.abs() + 2.0 ** -34).all()
        if steps == 1:
            differ = (got != x.to(torch.bfloat16)).double().mean().item()
            assert differ <= 2.0 ** -12, differ  # values within 2^-20 of a tie: 2^-11 of them if they were random, some on the right side


def emulated(g, steps, coefficients, eps):
    """The formula with X, A and B rounded as the kernel rounds them, in fp32 (products in 64 bits)."""
    a, b, c = coefficients
    half = lambda v: v.to(torch.float16).double()  # noqa: E731
    x = g.double()
    if tall := g.shape[1] > g.shape[2]:
        x = x.transpose(1, 2).contiguous()
    x = 2048 * x / (x.square().sum((1, 2), keepdim=True).sqrt() + eps)
    for step in range(steps):
        hi = half(x)
        x = hi + half(x - hi) if step == 0 or step + 1 < steps else hi
        s = half(torch.matmul(hi, hi.transpose(1, 2).contiguous()) / 4096) / 1024
        x = a * x + torch.matmul(half(b * s + c * torch.matmul(s, s)), hi)
    x = x / 2048
    return x.transpose(1, 2).contiguous() if tall else x


def formula(g, steps, coefficients, eps):
    a, b, c = coefficients
    x = g.double()
    if tall := g.shape[1] > g.shape[2]:
        x = x.transpose(1, 2).contiguous()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + eps)
    for _ in range(steps):
        s = torch.matmul(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.matmul(b * s + c * torch.matmul(s, s), x)
    return x.transpose(1, 2).contiguous() if tall else x


def gradient(seed, batch, rows, cols, rank, device="cpu"):
    """Output gradients times activations of `rank` tokens, a few channels loud."""
    gen = torch.Generator(device=device).manual_seed(seed)
    x = torch.randn(batch, rank, cols, generator=gen, device=device)
    x[:, :, ::max(cols // 4, 1)] *= 30
    return torch.bmm(torch.randn(batch, rows, rank, generator=gen, device=device), x)


def test_formula_is_the_oracles():
    g = gradient(0, 2, 32, 48, 20)
    for h in (g, g.transpose(1, 2).contiguous()):
        want = O.newton_schulz(h.numpy(), 3, MUON, 1e-7)
        assert np.abs(formula(h, 3, MUON, 1e-7).numpy() - want).max() <= 1e-12


def relative(got, want):
    return ((got.double() - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)).max().item()


@gpu
@pytest.mark.parametrize("batch, rows, cols, rank", [(1, 16, 16, 64), (3, 32, 128, 8), (2, 272, 656, 83), (2, 656, 272, 83), (1, 512, 512, 16),
                                                     (2, 128, 2048, 1000), (1, 1024, 2048, 512), (1, 2048, 1024, 4096), (40, 512, 784, 60),
                                                     (40, 784, 512, 600), (1, 1536, 2048, 4096), (2, 64, 64, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_several_steps(batch, rows, cols, rank, dtype):
    g = gradient(rows + rank, batch, rows, cols, rank, "cuda").to(dtype)
    for steps, coefficients in ((5, MUON), (2, MUON), (8, (1.5, -0.5, 0.0))):
        want = formula(g, steps, coefficients, 1e-7)
        bound = 3 * relative(emulated(g, steps, coefficients, 1e-7), want) + 2.0 ** -8
        got = Q.orthogonalize(g, steps=steps, coefficients=coefficients)
        assert relative(got, want) <= bound, (steps, bound)
        assert bound < 0.02  # and the bound says something


@gpu
def test_the_singular_values():
    """Five steps bring all singular values of a full-rank gradient between 0.6 and 1.3: there s (a + b s^2 + c s^4) moves
    them (0.68 to 1.13, and 0.02 for the error)."""
    g = torch.randn(2, 256, 384, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    s = torch.linalg.svdvals(Q.orthogonalize(g).double().cpu())
    assert s.max() < 1.3 and s.min() > 0.6


@gpu
@pytest.mark.parametrize("rows, cols", [(272, 528), (528, 272)])
def test_matrices_do_not_touch_each_other(rows, cols):
    """Zeros, NaN and infinities stay in their matrix; a matrix's result does not depend on the others or on its place."""
    g = gradient(4, 6, rows, cols, 300, "cuda")
    plain = Q.orthogonalize(g)
    g[1], g[3, 5, 7], g[4, 100, 200] = 0, float("nan"), float("inf")
    got = Q.orthogonalize(g)
    assert (got[1] == 0).all() and got[3].isnan().all() and got[4].isnan().all()
    assert torch.equal(got[[0, 2, 5]], plain[[0, 2, 5]])
    assert torch.equal(Q.orthogonalize(g[2]), plain[2])
    assert Q.orthogonalize(g[1], eps=0.0).isnan().all()


@gpu
def test_out_and_workspace():
    g = gradient(5, 3, 144, 208, 50, "cuda")
    want = Q.orthogonalize(g)
    out = torch.empty_like(want)
    ws = torch.empty(Q.orthogonalize_workspace_bytes(3, 144, 208), dtype=torch.uint8, device="cuda")
    for fill in (0, 255):  # what the workspace holds does not matter
        ws.fill_(fill)
        assert Q.orthogonalize(g, out=out, ws=ws) is out and torch.equal(out, want)
    assert Q.orthogonalize(g[:0]).shape == (0, 144, 208)
    for call, word in ((lambda: Q.orthogonalize(g, ws=ws[:-16]), "workspace"), (lambda: Q.orthogonalize(g, out=out[:2]), "out must"),
                       (lambda: Q.orthogonalize(g[0, 0]), "expected"), (lambda: Q.orthogonalize(g.half()), "bfloat16"),
                       (lambda: Q.orthogonalize(g.transpose(1, 2)), "contiguous"), (lambda: Q.orthogonalize(g, steps=0), "steps"),
                       (lambda: Q.orthogonalize(g[:, :, :200].contiguous()[:, :, :8].contiguous()), "multiples of 16")):
        with pytest.raises(Q.QuadsError, match=word):
            call()


@gpu
def test_past_32_bit_offsets():
    """Stacks whose last matrices begin past 2^32 bytes, wide and tall: the same bits as the stack's first (one matrix
    alone takes the other tile, whose sums may differ in their last bits), and the formula's values."""
    for rows, cols in ((1024, 2048), (2048, 1024)):
        g = gradient(6, 1, rows, cols, 256, "cuda").to(torch.bfloat16)
        stack = torch.zeros(1100, rows, cols, dtype=torch.bfloat16, device="cuda")
        stack[0], stack[-1] = g[0], g[0]
        got = Q.orthogonalize(stack, steps=2)
        assert torch.equal(got[-1], got[0]) and (got[1:-1] == 0).all()
        want = formula(g, 2, MUON, 1e-7)
        assert relative(got[-1:], want) <= 3 * relative(emulated(g, 2, MUON, 1e-7), want) + 2.0 ** -8
        del stack, got
