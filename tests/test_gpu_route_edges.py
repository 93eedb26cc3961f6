"""GPU: the router's and the combine's training side at ids and rows that name
nothing or the same thing twice, at arrays that begin anywhere, and the balance
loss's last bits.  Tolerances as in test_gpu_route_grad.py, u = 2^-24."""
import numpy as np
import pytest
import torch

from fp4_quantized_moe_amd import _lib as Q
from oracle import layer_oracle as O
from test_gpu_route_grad import COEF, U, combine_inputs, host, make

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("E", [3, 10, 17, 40, 100, 130, 300, 1000])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), -float("inf")])
def test_ids_past_the_experts_take_no_gradient(E, value):
    """An id of E or more is passed over, whatever its slot's gradient holds: also where the token's lanes have a place of that number."""
    logits, ids, dw, mask = make(E, 70, E, 3)
    b = Q.moe_balance_loss(logits, ids, COEF)
    places = 1 << (E - 1).bit_length()
    gone, quiet, loud = ids.clone(), dw.clone(), dw.clone()
    for t, e in enumerate((E, E + 1, places - 1, places, 1023, 1024, 2 ** 31 - 1, -1, -E, -2 ** 31)):
        if e < 0 or e >= E:
            ids[3 * t, t % 3] = e
            gone[3 * t, t % 3], quiet[3 * t, t % 3], loud[3 * t, t % 3] = -1, 0.0, value
    want = Q.moe_route_backward(logits, gone, dw=quiet, slope=b.slope)
    assert want.isfinite().all()
    assert torch.equal(Q.moe_route_backward(logits, ids, dw=loud, slope=b.slope), want)
    assert torch.equal(Q.moe_route_backward(logits, ids, dw=loud, slope=b.slope, mask=mask), torch.where(mask[:, None], want, 0.0))
