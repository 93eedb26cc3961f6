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


@pytest.mark.parametrize("T", [20, 1200])
@pytest.mark.parametrize("want_dw", [True, False])
def test_dropped_slots_into_the_callers_rows(T, want_dw):
    """With `out` the rows that no slot names keep what the caller put there, here zeros; without drops it is the same call."""
    dout, y, inverse, w = combine_inputs(11, T, 4, 176, f32, bf)
    full, dw_full = Q.moe_combine_backward(dout, y, inverse, w)
    gone = torch.rand(T, 4, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") < 0.3
    rows = inverse[gone].long()
    dropped = inverse.clone()
    dropped[gone] = torch.where(torch.arange(len(rows), device="cuda") % 2 == 0, -5, 2 ** 31 - 1).int()
    out = torch.zeros(4 * T, 176, dtype=bf, device="cuda")
    dy, dw = Q.moe_combine_backward(dout, y if want_dw else None, dropped, w, out=out)
    assert dy is out
    want = full.clone()
    want[rows] = 0
    assert torch.equal(dy, want) and (dw is None if not want_dw else torch.equal(dw, torch.where(gone, 0.0, dw_full)))
    assert torch.equal(Q.moe_combine_backward(dout, None, inverse, w, out=out)[0], full)
    for bad, word in ((out[:-1], "out must"), (out.float(), "out must"), (out.t().contiguous().t(), "contiguous"), (out[:, :160].contiguous(), "out must")):
        with pytest.raises(Q.QuadsError, match=word):
            Q.moe_combine_backward(dout, y, inverse, w, out=bad)


@pytest.mark.parametrize("T, N", [(30, 160), (30, 2064), (1500, 160), (1500, 2064)])
def test_a_row_named_by_several_slots(T, N):
    """Each of its elements is that of one of them; rows named once and every dw are as without it."""
    dout, y, inverse, w = combine_inputs(12, T, 4, N, f32, f32)
    inverse[1::2, 3] = inverse[0::2, 0]  # two tokens name the row
    inverse[0::3, 2] = inverse[0::3, 1]  # one token names it twice
    dy, dw = Q.moe_combine_backward(dout, y, inverse, w)
    rows = inverse.long()
    fit, named = torch.zeros(4 * T, N, dtype=torch.bool, device="cuda"), torch.zeros(4 * T, dtype=torch.bool, device="cuda")
    for j in range(4):  # a slot of every other token at a time: no row occurs twice
        want = (w[:, j, None] * dout).to(bf)
        for half in (0, 1):
            r = rows[half::2, j]
            assert len(r.unique()) == len(r)
            fit[r] |= dy[r] == want[half::2]
            named[r] = True
        terms = dout.double() * y[rows[:, j]].double()
        assert ((dw[:, j].double() - terms.sum(1)).abs() <= (N + 2) * U * terms.abs().sum(1)).all()
    assert fit[named].all()


@pytest.mark.parametrize("T", [1, 37, 3000])
def test_masks_and_loss_gradients_that_begin_anywhere(T):
    """A row of a batch's mask, and one number out of a buffer of the losses' gradients."""
    logits, ids, dw, mask = make(T, T, 24, 3)
    b = Q.moe_balance_loss(logits, ids, COEF, mask=mask)
    buffer, masks = torch.linspace(-2, 2, 9, device="cuda"), torch.ones(T + 20, dtype=torch.bool, device="cuda")
    for at in (1, 2, 3, 7, 16):
        m, g = masks[at:at + T], buffer[at % 9:at % 9 + 1]
        m.copy_(mask)
        got = Q.moe_balance_loss(logits, ids, COEF, mask=m)
        assert all(torch.equal(x, y) for x, y in zip(got, b))
        want = Q.moe_route_backward(logits, ids, dw=dw, slope=b.slope, dloss=g.clone(), mask=mask)
        assert torch.equal(Q.moe_route_backward(logits, ids, dw=dw, slope=b.slope, dloss=g, mask=m), want)


# tokens whose number, its reciprocal and the square of that all round, for one workgroup and for several
@pytest.mark.parametrize("T, E, top", [(7, 4, 1), (333, 12, 3), (6554, 128, 8), (8191, 100, 7), (100003, 8, 2), (3001, 1000, 16)])
@pytest.mark.parametrize("coef", [0.01, 1.0, 0.3])
def test_slope_is_rounded_once(T, E, top, coef):
    """slope is the fp32 value nearest to coef E counts / (top n^2): half a step, u, and what the 64-bit quotients add (4 times
    2^-53).  coef enters as the fp32 value that the call takes."""
    logits, ids, _, mask = make(T + E, T, E, top)
    c32 = float(np.float32(coef))
    for m in (None, mask):
        got = Q.moe_balance_loss(logits, ids, coef, mask=m)
        _, counts, slope = O.balance_loss(host(logits), ids.cpu().numpy(), c32, None if m is None else m.cpu().numpy())
        assert got.counts.tolist() == counts.tolist()
        assert (np.abs(host(got.slope) - slope) <= (U + 2.0 ** -51) * slope).all()
