"""The oracle of the operators around the experts against differences, bit
patterns and singular values."""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as O


def numeric(f, x, h=1e-6):
    """Central differences of the scalar f; error O(h^2) and 1e-16 / h."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + h
        up = f()
        x[i] = old - h
        g[i] = (up - f()) / (2 * h)
        x[i] = old
    return g


def test_norm_gradient():
    rng = np.random.default_rng(1)
    s, w, dy, dsum = rng.normal(size=(3, 16)), rng.normal(size=16), rng.normal(size=(3, 16)), rng.normal(size=(3, 16))
    loss = lambda: float((O.rms_norm(s, w, 1e-3)[0] * dy).sum() + (s * dsum).sum())  # noqa: E731
    dx, dw = O.rms_norm_grad(dy, s, w, 1e-3, dsum)
    assert np.abs(dx - numeric(loss, s)).max() < 1e-8
    assert np.abs(dw - numeric(loss, w)).max() < 1e-8


def test_e4m3_is_torchs():
    v = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, O.E4M3)
    x = np.abs(np.random.default_rng(2).normal(size=20000)) * np.exp2(np.random.default_rng(3).integers(-12, 9, 20000))
    mid = (O.E4M3[1:] + O.E4M3[:-1]) / 2
    x = np.concatenate((np.minimum(x, 448), mid, mid * (1 + 1e-6), mid * (1 - 1e-6))).astype(np.float32)
    assert np.array_equal(O.round_e4m3(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_mxfp8_blocks():
    x = np.zeros((1, 5 * 32))
    x[0, 32:64] = 500.0          # 2^8 <= a < 2^9: unit 1, saturates
    x[0, 64:96] = 2.0 ** -140    # below the smallest scale
    x[0, 96] = np.nan
    x[0, 128] = -448 * 2.0 ** 100
    codes, scales = O.quantize_mxfp8(x)
    v = O.dequantize_mxfp8(codes, scales)
    assert scales.tolist() == [[0, 127, 0, 255, 227]]
    assert (v[0, :32] == 0).all() and (v[0, 32:64] == 448).all() and (v[0, 64:96] == 0).all()
    assert np.isnan(v[0, 96:128]).all() and v[0, 128] == x[0, 128] and (codes[0, 96:128] == 0).all()


@pytest.mark.parametrize("masked", [False, True])
def test_router_gradient(masked):
    rng = np.random.default_rng(4)
    T, E, top = 7, 5, 2
    logits = rng.normal(size=(T, E))
    ids = np.argsort(-logits, 1)[:, :top]
    dw = rng.normal(size=(T, top))
    mask = np.array([1, 0, 1, 1, 0, 1, 1], bool) if masked else None
    keep = np.ones(T, bool) if mask is None else mask

    def loss():  # the counts are constants, and so is the choice
        w = np.take_along_axis(O.softmax(logits), ids, 1)
        return 1.7 * O.balance_loss(logits, ids, 0.3, mask)[0] + float((w * dw)[keep].sum())

    slope = O.balance_loss(logits, ids, 0.3, mask)[2]
    assert np.abs(O.route_grad(logits, ids, dw, slope, 1.7, mask) - numeric(loss, logits)).max() < 1e-8


def test_balance_is_coef_when_even():
    ids = np.arange(8).reshape(8, 1) % 4
    loss, counts, _ = O.balance_loss(np.zeros((8, 4)), ids, 0.01)
    assert abs(loss - 0.01) < 1e-15 and counts.tolist() == [2, 2, 2, 2]
    assert O.balance_loss(np.zeros((8, 4)), ids, 0.01, np.zeros(8, bool))[0] == 0
    assert (O.softmax(np.full((1, 4), -np.inf)) == 0).all()


def test_newton_schulz_moves_singular_values_alone():
    rng = np.random.default_rng(5)
    g = rng.normal(size=(6, 10))
    u, s, v = np.linalg.svd(g, full_matrices=False)
    a, b, c = 3.4445, -4.7750, 2.0315
    s = s / np.linalg.norm(g)
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.abs(O.newton_schulz(g, 5, (a, b, c), 0.0) - (u * s) @ v).max() < 1e-12
    assert np.abs(O.newton_schulz(g.T, 5, (a, b, c), 0.0) - ((u * s) @ v).T).max() < 1e-12
