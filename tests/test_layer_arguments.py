"""What the operators around the experts take and refuse at the edges of their
documented arguments, before anything is enqueued: the C ABI on the CPU host.
Addresses are never dereferenced there; calls that would launch are not made."""
import ctypes
import os

import pytest

from fp4_quantized_moe_amd import _lib as Q

ARG, SHAPE, WORKSPACE = -1, -2, -3
P = 1 << 20  # an address


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(Q.LIB_PATH):
        pytest.fail("libquads.so is not built (python -m fp4_quantized_moe_amd.build)")
    return Q.load()


# up to 2^39 elements, however long their longer side
@pytest.mark.parametrize("batch, rows, cols", [(2, 16, 1048560), (300, 65536, 32), (17, 262144, 64), (65535, 16, 32768), (1, 1 << 19, 1 << 19),
                                               (32768, 4096, 4096)])
def test_orthogonalize_takes_the_documented_sizes(L, batch, rows, cols):
    assert batch * rows * cols <= 2 ** 39
    for r, c in ((rows, cols), (cols, rows)):
        assert L.quads_orthogonalize_workspace_bytes(batch, r, c) > 0
        d = (P, 1, batch, r, c, 5, (ctypes.c_float * 3)(3.4, -4.8, 2.0), 1e-7, P, None, 0, None)
        assert L.quads_orthogonalize(*d) == WORKSPACE  # the last check


@pytest.mark.parametrize("batch, rows, cols", [(32769, 4096, 4096), (2, 1 << 19, (1 << 19) + 16), (65535, 32, (1 << 18) + 16)])
def test_orthogonalize_refuses_more(L, batch, rows, cols):
    for r, c in ((rows, cols), (cols, rows)):
        assert L.quads_orthogonalize_workspace_bytes(batch, r, c) == 0 and b"overflow" in L.quads_last_error()
