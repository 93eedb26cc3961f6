"""The MXFP4 / gated-block oracle against hand-worked values and differences."""
import numpy as np
import pytest

from oracle import mxfp4_oracle as M


def _block(*vals):
    x = np.zeros(32)
    x[:len(vals)] = vals
    return x


@pytest.mark.parametrize("rule, amax, byte", [
    ("floor", 1.0, 125), ("floor", 6.0, 127), ("floor", 7.9, 127), ("floor", 8.0, 128), ("floor", 0.0, 0),
    ("even", 6.9, 127), ("even", 7.0, 128), ("even", 1.7499, 125), ("even", 1.75, 126), ("even", 0.0, 0),
    ("floor", 2.0 ** -149, 0), ("floor", 2.0 ** -125, 0), ("floor", 2.0 ** -124, 1),
    ("floor", 1.999 * 2.0 ** 127, 252), ("even", 1.999 * 2.0 ** 127, 252),
    ("floor", np.inf, 255), ("even", np.nan, 255),
])
def test_scale_bytes(rule, amax, byte):
    assert M.block_bytes(np.array([amax]), rule)[0] == byte


def test_ties_go_to_even_codes():
    v = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.9]
    codes, s = M.quantize(_block(*v, -0.0, -0.25, -5.0)[None])
    assert s[0, 0] == 127
    assert codes[0, :12].tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7, 8, 8, 14]


def test_nearest_by_distance():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 64)) * np.exp2(rng.integers(-20, 20, (50, 1)))
    for rule in ("floor", "even"):
        codes, s = M.quantize(x, rule)
        unit = np.repeat(np.exp2(s.astype(float) - 127), 32, -1)
        d = np.abs(np.minimum(np.abs(x) / unit, 6)[..., None] - M.LEVELS)
        assert (np.take_along_axis(d, (codes & 7)[..., None].astype(int), -1)[..., 0] <= d.min(-1)).all()
    assert np.array_equal(M.unpack(M.pack(codes)), codes)


def test_values_survive_a_second_pass():
    rng = np.random.default_rng(1)
    v = M.dequantize(*M.quantize(rng.standard_normal((9, 96))))
    assert np.array_equal(M.dequantize(*M.quantize(v)), v)


def test_gated_gradient_against_differences():
    rng = np.random.default_rng(2)
    gu, dh = rng.standard_normal((5, 24)) * 2, rng.standard_normal((5, 12))
    got, eps = M.gated_grad(dh, gu), 1e-5
    for i in range(24):
        step = np.zeros((5, 24))
        step[:, i] = eps
        num = (dh * (M.gated(gu + step) - M.gated(gu - step))).sum(1) / (2 * eps)
        assert np.allclose(got[:, i], num, rtol=1e-8, atol=1e-8)  # eps^2 and 2^-53 / eps
