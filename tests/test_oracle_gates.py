"""The gated-block oracle's sigmoid and its gradient where the gate is far from
0, against 60-digit decimals."""
from decimal import Decimal, getcontext

import numpy as np
import pytest

from oracle import mxfp4_oracle as M

getcontext().prec = 60
EPS = 2.0 ** -53


def sigmoid(z):
    return 1 / (1 + (-Decimal(z)).exp())


@pytest.mark.parametrize("z", [0.0, 0.5, -0.5, 5.0, -5.0, 20.0, -20.0, 37.0, -37.0, 80.0, -80.0, -95.0, 300.0, -300.0, 700.0, -700.0])
def test_sigmoid(z):
    want = sigmoid(z)
    # exp, a sum and a quotient, each within a step
    assert abs(Decimal(float(M.sigmoid(z))) - want) <= Decimal(4 * EPS) * want
    assert abs(Decimal(float(M.silu(z))) - Decimal(z) * want) <= abs(Decimal(5 * EPS) * want * Decimal(z))


@pytest.mark.parametrize("z", [-700.0, -95.0, -40.0, -20.0, -1.0, 1.0, 20.0, 40.0, 95.0])
def test_gradient(z):
    s, u, dh = sigmoid(z), 1.5, -0.75
    dg, du = M.gated_grad(np.array([dh]), np.array([z, u]))
    part = abs(Decimal(dh * u) * s) * (1 + abs(Decimal(z)))
    want = Decimal(dh * u) * s * (1 + Decimal(z) * (1 - s))
    assert abs(Decimal(float(dg)) - want) <= Decimal(16 * EPS) * part
    assert abs(Decimal(float(du)) - Decimal(dh) * Decimal(z) * s) <= Decimal(8 * EPS) * abs(Decimal(dh) * Decimal(z) * s)


def test_limits():
    with np.errstate(over="raise", invalid="raise", divide="raise"):
        z = np.array([-700.0, 0.0, 800.0, -3e38, 3e38])
        assert M.sigmoid(z).tolist()[1:] == [0.5, 1.0, 0.0, 1.0]
