"""GPU: the balance loss with its counts, the gradient of the router's logits
and the combine's gradient against the 64-bit oracle.

Tolerances, with u = 2^-24.  A probability: the exponent's argument is off by
u |l - m|, expf by 2 u (one ulp), the sum of E terms by E u, the reciprocal and
the product by u each: e_p = (E + S + 5) u relative, S the largest |l - m| of a
row.  The loss is a sum of positive terms: over T tokens, then E experts, with
8 more roundings: (T + E) u + e_p + 8 u relative; slope has 6 roundings.
dlogits = p (dp - sum p dp): with M = |dloss slope| + sum |dw| per expert, dp is
off by (top + 7) u M, the sum by (E + top + 8) u + e_p of sum p M, the result by
three roundings: (E + top + 16) u + 2 e_p of p (M + sum p M).
Combine: dy is one fp32 product rounded to bf16, bit for bit; dw is a sum of N
products: (N + 2) u sum |dout y|."""
import numpy as np
import pytest
import torch

from fp4_quantized_moe_amd import _lib as Q
from oracle import layer_oracle as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
COEF = 0.01


def host(t):
    return t.detach().double().cpu().numpy()


def make(seed, T, E, top, spread=2.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    logits = spread * torch.randn(T, E, generator=gen, device="cuda")
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :top].int().contiguous()
    dw = torch.randn(T, top, generator=gen, device="cuda")
    mask = torch.rand(T, generator=gen, device="cuda") < 0.7
    return logits, ids, dw, mask


def probability_error(logits):
    l = host(logits)
    m = l.max(1, keepdims=True)
    S = np.abs(np.where(np.isfinite(l), l, m) - np.where(np.isfinite(m), m, 0)).max() if l.size else 0
    return (logits.shape[1] + S + 5) * U


def check_balance(logits, ids, mask):
    got = Q.moe_balance_loss(logits, ids, COEF, mask=mask)
    m = None if mask is None else mask.cpu().numpy() != 0
    loss, counts, slope = O.balance_loss(host(logits), ids.cpu().numpy(), COEF, m)
    assert got.counts.tolist() == counts.tolist()
    assert (np.abs(host(got.slope) - slope) <= 6 * U * slope).all()
    T, E = logits.shape
    assert abs(got.loss.item() - loss) <= ((T + E + 8) * U + probability_error(logits)) * loss
    return got


def check_grad(logits, ids, dw, slope, dloss, mask):
    got = host(Q.moe_route_backward(logits, ids, dw=dw, slope=slope, dloss=dloss, mask=mask))
    T, E = logits.shape
    m = None if mask is None else mask.cpu().numpy() != 0
    i, g = ids.cpu().numpy(), 1.0 if dloss is None else dloss.item()
    arrays = [None if t is None else host(t) for t in (dw, slope)]
    want = O.route_grad(host(logits), i, *arrays, g, m)
    p = O.softmax(host(logits))
    M = np.zeros((T, E))  # magnitudes of dp, by the oracle's own linear form
    if slope is not None:
        M += abs(g) * host(slope)
    if dw is not None:
        for j in range(i.shape[1]):
            ok = (i[:, j] >= 0) & (i[:, j] < E)
            np.add.at(M, (np.nonzero(ok)[0], i[ok, j]), np.abs(host(dw))[ok, j])
    tol = ((E + i.shape[1] + 16) * U + 2 * probability_error(logits)) * p * (M + (p * M).sum(1, keepdims=True))
    assert (np.abs(got - want) <= tol).all()
    if m is not None:
        assert (got[~m] == 0).all()
    return got


# tokens, experts, choices: every number of experts a lane, one workgroup and several (by 512, or 128 past 128 experts), whole
# and partial groups
SIZES = [(1, 1, 1), (1, 4, 1), (3, 16, 16), (511, 12, 3), (513, 17, 8), (2000, 32, 2), (512, 64, 8), (9000, 64, 6), (1000, 65, 5),
         (8192, 128, 8), (130, 129, 8), (127, 256, 16), (700, 300, 8), (33, 512, 8), (3000, 1000, 16), (129, 1024, 4),
         (100003, 8, 2)]


@pytest.mark.parametrize("T, E, top", SIZES)
def test_router(T, E, top):
    logits, ids, dw, mask = make(T + E, T, E, top)
    for m in (None, mask, mask.to(torch.uint8) * 255):
        b = check_balance(logits, ids, m)
        check_grad(logits, ids, dw, b.slope, None, m)
    check_grad(logits, ids, dw, None, None, None)
    check_grad(logits, ids, None, b.slope, torch.full((1,), -3.5, device="cuda"), mask)
    assert (Q.moe_route_backward(logits, ids) == 0).all()


@pytest.mark.parametrize("T, E, top", [(512, 16, 2), (513, 16, 2), (128, 128, 8), (129, 128, 8), (64, 200, 3), (65, 200, 3), (17, 1024, 16),
                                       (32768, 17, 3), (32769, 17, 3), (8193, 200, 4), (9001, 1000, 2)])
def test_balance_loss_by_one_workgroup_and_many(T, E, top):
    """Both sides of the sizes at which one workgroup, 128 and 256 take the tokens."""
    logits, ids, _, mask = make(T, T, E, top)
    for m in (None, mask):
        check_balance(logits, ids, m)


def test_the_routers_own_choice():
    """counts are the differences of moe_route's offsets, and its weights are the probabilities differentiated."""
    logits, _, dw, _ = make(1, 3000, 64, 8)
    ids, w, offsets, _, _ = Q.moe_route(logits, 8)
    assert torch.equal(check_balance(logits, ids, None).counts, offsets.diff())
    p = torch.from_numpy(O.softmax(host(logits))).cuda()
    assert ((w - p.gather(1, ids.long())).abs() <= probability_error(logits) * w).all()
    check_grad(logits, ids, dw, None, None, None)


@pytest.mark.parametrize("T", [40, 5000])
@pytest.mark.parametrize("E", [9, 128, 200])
def test_rows_without_experts(T, E):
    """Experts shut off by -inf and by the lowest fp32, rows with no expert left, large logits, equal ones."""
    logits, _, dw, mask = make(T + E, T, E, 4)
    logits[:, 3] = -float("inf")
    logits[:, 5] = torch.finfo(torch.float32).min
    logits[0] = -float("inf")
    logits[1] = torch.finfo(torch.float32).min
    logits[2] = 7.25
    logits[4] *= 40
    ids = Q.moe_route(logits, 4)[0]
    l, S = host(logits), 2.0 ** 8  # exponents far below -104 are 0 in both, whatever the argument's error
    p = O.softmax(l)
    e_p = (E + S + 5) * U
    b = Q.moe_balance_loss(logits, ids, COEF, mask=mask)
    loss, counts, slope = O.balance_loss(l, ids.cpu().numpy(), COEF, mask.cpu().numpy())
    assert b.counts.tolist() == counts.tolist() and abs(b.loss.item() - loss) <= ((T + E + 8) * U + e_p) * loss
    got = host(Q.moe_route_backward(logits, ids, dw=dw, slope=b.slope))
    want = O.route_grad(l, ids.cpu().numpy(), host(dw), slope)
    M = slope + np.abs(host(dw)).sum(1, keepdims=True)
    # results below the smallest normal number of fp32 lose bits: 2^-126 absolute
    tol = ((E + 20) * U + 2 * e_p) * p * (M + (p * M).sum(1, keepdims=True)) + 2.0 ** -126
    assert (np.abs(got - want) <= tol).all()
    assert (got[0] == 0).all() and (got[3:, 3] == 0).all()  # rows 1 and 2 have been written over


def test_padding_may_hold_anything():
    """Tokens that take no part: NaN logits, wrong ids and infinite gradients do not reach the others."""
    T, E, top = 700, 20, 4
    logits, ids, dw, mask = make(2, T, E, top)
    b, g = check_balance(logits, ids, mask), None
    g = Q.moe_route_backward(logits, ids, dw=dw, slope=b.slope, mask=mask)
    off = ~mask
    logits[off], ids[off], dw[off] = float("nan"), -7, float("inf")
    ids[off.nonzero()[0]] = 2 ** 31 - 1
    c = Q.moe_balance_loss(logits, ids, COEF, mask=mask)
    assert torch.equal(b.loss, c.loss) and torch.equal(b.counts, c.counts) and torch.equal(b.slope, c.slope)
    assert torch.equal(g, Q.moe_route_backward(logits, ids, dw=dw, slope=b.slope, mask=mask))


def test_nan_and_infinite_logits():
    logits, ids, dw, _ = make(3, 600, 24, 3)
    b = Q.moe_balance_loss(logits, ids, COEF)
    want = Q.moe_route_backward(logits, ids, dw=dw, slope=b.slope)
    logits[5, 2], logits[9, 23] = float("nan"), float("inf")
    got = Q.moe_route_backward(logits, ids, dw=dw, slope=b.slope)
    assert got[5].isnan().all() and got[9].isnan().all()
    keep = [i for i in range(600) if i not in (5, 9)]
    assert torch.equal(got[keep], want[keep])
    c = Q.moe_balance_loss(logits, ids, COEF)
    assert c.loss.isnan().all() and torch.equal(c.counts, b.counts) and torch.equal(c.slope, b.slope)


def test_ids_twice_and_outside():
    """The same expert twice in a token counts twice; ids outside [0, E) are passed over."""
    logits, ids, dw, mask = make(4, 900, 10, 4)
    ids[:, 1] = ids[:, 0]
    ids[7, 2], ids[8, 3], ids[9] = -1, 10, 1 << 30
    for m in (None, mask):
        b = check_balance(logits, ids, m)
        check_grad(logits, ids, dw, b.slope, None, m)


@pytest.mark.parametrize("T", [0, 1, 2000])
def test_no_token_takes_part(T):
    logits, ids, dw, mask = make(5, T, 40, 2)
    b = Q.moe_balance_loss(logits, ids, COEF, mask=torch.zeros_like(mask))
    assert b.loss.item() == 0 and (b.counts == 0).all() and (b.slope == 0).all()
    assert (Q.moe_route_backward(logits, ids, dw=dw, slope=b.slope, mask=torch.zeros_like(mask)) == 0).all()


def test_gradient_by_differences_of_the_kernels_loss():
    """The loss of the kernel itself, moved by h along v: h <g, v> up to O(h^2) and its own rounding."""
    logits, ids, _, mask = make(6, 64, 8, 2)
    v = torch.randn(64, 8, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    b = Q.moe_balance_loss(logits, ids, 1.0, mask=mask)
    g = Q.moe_route_backward(logits, ids, slope=b.slope, mask=mask)
    h = 2.0 ** -5
    up, down = (Q.moe_balance_loss(logits + s * h * v, ids, 1.0, mask=mask).loss.item() for s in (1, -1))
    slope = (g.double() * v.double()).sum().item()
    curve = (host(b.slope)[None] * np.abs(host(v)) ** 3).sum() * h * h  # third derivatives of p are at most 1
    rounding = 2 * ((64 + 8 + 8) * U + probability_error(logits)) * up / h
    assert abs((up - down) / (2 * h) - slope) <= curve + rounding


def combine_inputs(seed, T, top, N, d_type, y_type):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    inverse = torch.randperm(T * top, generator=gen, device="cuda").int().view(T, top)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return randn(T, N).to(d_type), randn(T * top, N).to(y_type), inverse, torch.rand(T, top, generator=gen, device="cuda")


bf, f32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("T, top, N", [(1, 1, 16), (1, 8, 2048), (3, 2, 4112), (333, 3, 656), (17, 16, 528), (1023, 5, 512), (1024, 1, 64),
                                       (1025, 4, 1040), (2000, 8, 2048), (1500, 12, 496), (1100, 7, 16)])
@pytest.mark.parametrize("types", [(f32, f32), (bf, f32), (f32, bf), (bf, bf)])
def test_combine_backward(T, top, N, types):
    dout, y, inverse, w = combine_inputs(T + top, T, top, N, *types)
    dy, dw = Q.moe_combine_backward(dout, y, inverse, w)
    rows = inverse.long()
    want = torch.empty_like(dy)
    want[rows.view(-1)] = (w[:, :, None] * dout.float()[:, None]).to(bf).flatten(0, 1)
    assert torch.equal(dy, want)
    for j in range(top):
        terms = dout.double() * y[rows[:, j]].double()
        assert ((dw[:, j].double() - terms.sum(1)).abs() <= (N + 2) * U * terms.abs().sum(1)).all()
    alone, none = Q.moe_combine_backward(dout, None, inverse, w)
    assert none is None and torch.equal(alone, dy)


@pytest.mark.parametrize("T", [20, 1200])
def test_combine_slots_without_a_row(T):
    dout, y, inverse, w = combine_inputs(8, T, 4, 160, f32, f32)
    full, dw_full = Q.moe_combine_backward(dout, y, inverse, w)
    gone = torch.rand(T, 4, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") < 0.3
    rows = inverse[gone].long()
    y[rows] = float("nan")  # what no slot names does not matter
    inverse[gone] = torch.where(torch.arange(len(rows), device="cuda") % 2 == 0, -1, 4 * T).int()
    dy = torch.full((4 * T, 160), 3.0, dtype=bf, device="cuda")
    dw = torch.empty(T, 4, device="cuda")
    L = Q.load()
    assert L.quads_moe_combine_backward(dout.data_ptr(), 0, y.data_ptr(), 0, inverse.data_ptr(), w.data_ptr(), T, 4, 160,
                                        dy.data_ptr(), dw.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    full[rows] = 3.0  # left as they were
    assert torch.equal(dy, full) and torch.equal(dw, torch.where(gone, 0.0, dw_full))


def test_combine_of_no_tokens_and_past_32_bit_offsets():
    z = torch.zeros(0, 64, device="cuda")
    dy, dw = Q.moe_combine_backward(z, z, torch.zeros(0, 2, dtype=torch.int32, device="cuda"), torch.zeros(0, 2, device="cuda"))
    assert dy.shape == (0, 64) and dw.shape == (0, 2)
    T, top, N = 40000, 8, 8192  # y of 10 GB, dy of 5
    y = torch.zeros(T * top, N, device="cuda")
    dout = torch.zeros(T, N, dtype=bf, device="cuda")
    inverse = torch.arange(T * top, dtype=torch.int32, device="cuda").flip(0).view(T, top).contiguous()
    w = torch.rand(T, top, device="cuda")
    y[:8], dout[-1] = 2.0, 0.5
    y[-8:], dout[0] = 3.0, 1.0
    dy, dw = Q.moe_combine_backward(dout, y, inverse, w)
    assert (dw[-1] == N).all() and (dw[0] == 3.0 * N).all() and (dw[1:-1] == 0).all()
    assert torch.equal(dy[0], (0.5 * w[-1, 7]).to(bf).expand(N)) and torch.equal(dy[-1], w[0, 0].to(bf).expand(N))


def test_checks_of_tensors():
    logits, ids, dw, mask = make(9, 20, 8, 2)
    b = Q.moe_balance_loss(logits, ids, COEF)
    for call, word in ((lambda: Q.moe_balance_loss(logits, ids[:3], COEF), "must be"), (lambda: Q.moe_balance_loss(logits.half(), ids, COEF), "float32"),
                       (lambda: Q.moe_balance_loss(logits, ids.long(), COEF), "int32"), (lambda: Q.moe_balance_loss(logits, ids, COEF, mask=mask[:4]), "mask"),
                       (lambda: Q.moe_balance_loss(logits, ids, COEF, mask=mask.float()), "mask"),
                       (lambda: Q.moe_route_backward(logits, ids, dw=dw[:, :1].contiguous()), "dw must"),
                       (lambda: Q.moe_route_backward(logits, ids, slope=b.slope[:4]), "slope must"),
                       (lambda: Q.moe_route_backward(logits, ids, dloss=b.loss), "without slope"),
                       (lambda: Q.moe_balance_loss(logits[:, :1].contiguous(), ids, COEF), "top must"),
                       (lambda: Q.moe_combine_backward(dw, logits, ids, dw), "must be"),
                       (lambda: Q.moe_combine_backward(torch.zeros(20, 24, device="cuda"), None, ids, dw), "multiple of 16")):
        with pytest.raises(Q.QuadsError, match=word):
            call()
