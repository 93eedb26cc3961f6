"""GPU: orthogonalised updates of long thin matrices, bit for bit as in
test_gpu_orthogonalize.py."""
import pytest
import torch

from fp4_quantized_moe_amd import _lib as Q
from test_gpu_orthogonalize import signs, whole_step

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
