"""GPU: the norm's gradient against differences of the norm's own output, and
both sides of the sizes at which the kernels' lanes of a row change: up to 128,
1024 (a wave, where there are 2048 rows), 2048, 4096 and 8192 columns, 16384 the
most.  Tolerances as in test_gpu_norm.py, u = 2^-24."""
import numpy as np
import pytest
import torch

import test_gpu_norm as N
from fp4_quantized_moe_amd import _lib as Q
from oracle import layer_oracle as O
from test_gpu_norm import BF16, EPS, U, bf, f32, host

pytestmark = pytest.mark.gpu

SIDES = [(3, 112), (3, 128), (3, 144), (2048, 128), (2047, 160), (2047, 512), (2048, 512), (2048, 528), (2047, 1024), (2048, 1024), (2048, 1040),
         (5, 2048), (5, 2064), (5, 4096), (5, 4112), (5, 8192), (5, 8208), (2, 16368), (2, 16384)]


@pytest.mark.parametrize("rows, cols", SIDES)
def test_both_sides_of_a_rows_lanes(rows, cols):
    for types in ((f32, bf, f32), (bf, None, bf)):
        N.test_norm(rows, cols, types)


@pytest.mark.parametrize("rows, cols", SIDES + [(1024, 128), (1025, 144), (1025, 4096), (1025, 4112), (1025, 8208)])
def test_both_sides_of_a_rows_lanes_backward(rows, cols):
    for types in ((f32, bf, bf), (bf, f32, f32)):
        N.test_norm_backward(rows, cols, types)


@pytest.mark.parametrize("rows, cols", [(4, 96), (4, 256), (2100, 96), (2100, 400), (2100, 1008), (9, 2000), (9, 4096), (5, 8192), (3, 16384)])
@pytest.mark.parametrize("residual", [False, True])
def test_gradient_by_differences_of_the_kernels_norm(rows, cols, residual):
    """f(s) = <dy, y(s)> with y as rms_norm writes it, moved by h along v = dx, where f falls or grows fastest:
    (f(s + h v) - f(s - h v)) / 2h = <dx, v>, up to
      - the formula's own third derivative: the same difference of the 64-bit oracle, less its slope,
      - y's rounding, 2^-8 + e_y of each |dy y|, over h,
      - the points' rounding to fp32, u |s + h v| times the slope there, taken as twice |dx|, over h,
      - dx's own error, test_norm_backward's."""
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    s, dy = (torch.randn(rows, cols, generator=gen, device="cuda") for _ in range(2))
    w = torch.rand(cols, generator=gen, device="cuda") + 0.5
    kept = Q.rms_norm(torch.zeros_like(s), w, residual=s, eps=EPS, keep=True) if residual else Q.rms_norm(s, w, eps=EPS, keep=True)
    assert torch.equal(kept.sum, s)
    dx, _ = Q.rms_norm_backward(dy, kept.sum, w, kept.rstd)
    h, v = 0.25, dx
    points, values, size, moved = [], [], 0.0, 0.0
    for sign in (h, -h):
        r = Q.rms_norm(sign * v, w, residual=s, eps=EPS) if residual else Q.rms_norm(s + sign * v, w, eps=EPS)
        values.append((host(dy) * host(r.y)).sum())
        size += np.abs(host(dy) * host(r.y)).sum()
        moved += 2 * U * (np.abs(host(r.sum)) * np.abs(host(dx))).sum()
        points.append((host(dy) * O.rms_norm(host(s) + sign * host(v), host(w), EPS)[0]).sum())
    slope = (host(dx) * host(v)).sum()
    want, _ = O.rms_norm_grad(host(dy), host(s), host(w), EPS)
    curve = abs((points[0] - points[1]) / (2 * h) - (want * host(v)).sum())
    e_y, e_dx = (cols / 2 + 6) * U, (cols + 20) * U
    r, d = host(kept.rstd)[:, None], np.abs(host(dy) * host(w))
    own = (e_dx * r * (d + np.abs(host(s)) * r * (d * np.abs(host(s)) * r).mean(1, keepdims=True)) * np.abs(host(v))).sum()
    bound = curve + ((BF16 + e_y) * size + moved) / (2 * h) + own
    assert bound < 0.1 * slope  # and the bound says something
    assert abs((values[0] - values[1]) / (2 * h) - slope) <= bound, (bound / slope)
