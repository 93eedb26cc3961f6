"""GPU: a training step of the MoE layer from the residual stream to the masters'
update, as a trainer calls it, against a 64-bit autograd of the same layer; the
same step on another stream and in a replayed graph; calls at once.

Tolerance.  Against 64 bits every activation and gradient that is kept in bf16 is
off by half a step, 2^-8, at most: y, gate | up, h; dy, d gate | d up; dx.  Each
enters the following ones linearly (silu's slope is at most 1.1), so in the
2-norm a result behind n of them is off by 1.1 n 2^-8 to first order; n <= 6.
The choice of experts and the counts are the kernel's own in both."""
import pytest
import torch

from fp4_quantized_moe_amd import _lib as Q

pytestmark = pytest.mark.gpu
T, H, I, E, TOP, COEF, EPS = 700, 256, 128, 12, 3, 0.02, 1e-6
bf, f32 = torch.bfloat16, torch.float32


def inputs(seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return dict(stream=randn(T, H).to(bf), delta=(0.5 * randn(T, H)).to(bf), weight=(1 + 0.2 * randn(H)).to(bf),
                router=0.1 * randn(E, H), w_gate_up=(0.06 * randn(E, 2 * I, H)).to(bf), w_down=(0.08 * randn(E, H, I)).to(bf),
                dout=randn(T, H), dsum=randn(T, H).to(bf), mask=(torch.arange(T, device="cuda") < T - 100))


def step(d):
    """Forward, backward and the update, by the library's calls (and torch's for the router's projection)."""
    n = Q.rms_norm(d["delta"], d["weight"], residual=d["stream"], eps=EPS, keep=True)
    logits = n.y.float() @ d["router"].t()
    ids, w, offs, rt, inv = Q.moe_route(logits, TOP)
    R = T * TOP
    h, gu = Q.moe_gated_forward(n.y, d["w_gate_up"], offs, rt)
    y = Q.GemmCall(N=H, K=I, expert_offsets=offs, num_rows=R, x_bf16=h, w_bf16=d["w_down"])()
    out = Q.moe_combine(y, inv, w)
    balance = Q.moe_balance_loss(logits, ids, COEF, mask=d["mask"])

    dy, dw = Q.moe_combine_backward(d["dout"], y, inv, w)
    dgu = Q.moe_gated_backward(dy, d["w_down"], gu, offs)
    dx, _, dw_gate_up = Q.QatBackward(d["w_gate_up"], dgu, n.y, offs, rt, inv)()
    dw_down = Q.WgradCall(dy, h, offs)()
    # padding takes no part in the balance loss; its combine weights do, as its output does
    dlogits = Q.moe_route_backward(logits, ids, dw=dw) + Q.moe_route_backward(logits, ids, slope=balance.slope, mask=d["mask"])
    dstream, dweight = Q.rms_norm_backward(dx + dlogits @ d["router"], n.sum, d["weight"], n.rstd, dsum=d["dsum"])
    return dict(out=out, loss=balance.loss, counts=balance.counts, ids=ids, offsets=offs, dstream=dstream, dweight=dweight,
                dlogits=dlogits, dw_gate_up=dw_gate_up, dw_down=dw_down,
                update_gate_up=Q.orthogonalize(dw_gate_up.view(2 * E, I, H)), update_down=Q.orthogonalize(dw_down))


def reference(d, ids):
    """The same layer in 64 bits with autograd; the experts' choice is given."""
    p = {k: d[k].double().requires_grad_(True) for k in ("weight", "w_gate_up", "w_down")}
    s = (d["stream"].float() + d["delta"].float()).to(bf).double().requires_grad_(True)
    y = s / torch.sqrt(s.square().mean(1, keepdim=True) + EPS) * p["weight"]
    logits = y @ d["router"].double().t()
    logits.retain_grad()
    prob = torch.softmax(logits, 1)
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, slot = (ids == e).nonzero(as_tuple=True)
        z = y[t] @ p["w_gate_up"][e].t()
        g, u = z.chunk(2, 1)
        out = out.index_add(0, t, prob[t, e, None] * ((g * torch.sigmoid(g) * u) @ p["w_down"][e].t()))
    m, n = d["mask"], int(d["mask"].sum())
    counts = torch.bincount(ids[m].flatten().long(), minlength=E)
    loss = COEF * E * (counts / (TOP * n) * prob[m].sum(0) / n).sum()
    ((out * d["dout"].double()).sum() + loss + (s * d["dsum"].double()).sum()).backward()
    return dict(out=out.detach(), loss=loss.detach().reshape(1), counts=counts, dstream=s.grad, dweight=p["weight"].grad,
                dlogits=logits.grad, dw_gate_up=p["w_gate_up"].grad, dw_down=p["w_down"].grad)


def test_a_training_step():
    d = inputs(1)
    got = step(d)
    want = reference(d, got["ids"])
    assert got["counts"].tolist() == want["counts"].tolist()
    assert (got["offsets"].diff() >= got["counts"]).all()
    for name in ("out", "loss", "dstream", "dweight", "dlogits", "dw_gate_up", "dw_down"):
        off = (got[name].double() - want[name]).norm() / want[name].norm()
        assert off <= 1.1 * 6 * 2.0 ** -8, (name, off.item())
    for name, g in (("update_gate_up", got["dw_gate_up"].view(2 * E, I, H)), ("update_down", got["dw_down"])):
        # descent: an orthogonalised update has the gradient's direction, <g, u> = sum of s f(s) / |g| > 0, and about unit singular values
        u = got[name].double()
        assert ((g.double() * u).sum((1, 2)) > 0).all()
        assert torch.linalg.svdvals(u.cpu()).max() < 1.3


def test_the_step_on_another_stream_and_in_a_graph():
    """The bits of the default stream on another one, and in each of several replays with eager work between them."""
    d = inputs(2)
    want = step(d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step(d)
    side.synchronize()
    for k in want:
        assert torch.equal(again[k], want[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(d)
    for replay in range(4):
        for t in out.values():
            t.fill_(3)
        other = step(inputs(10 + replay))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(out[k], want[k]), (replay, k)
        assert not torch.equal(other["out"], want["out"])
    # new values in the captured inputs
    new = inputs(3)
    for k in d:
        d[k].copy_(new[k])
    graph.replay()
    torch.cuda.synchronize()
    fresh = step(new)
    for k in fresh:
        assert torch.equal(out[k], fresh[k]), k


def test_two_calls_at_once():
    """Calls of each operator on two streams, unordered, each with a workspace of its own."""
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    gen = torch.Generator(device="cuda").manual_seed(5)
    g = [torch.randn(6, 272, 528, generator=gen, device="cuda") for _ in sides]
    x = [torch.randn(5000, 512, generator=gen, device="cuda") for _ in sides]
    ids = [Q.moe_route(t[:, :64].contiguous(), 8)[0] for t in x]
    w = torch.ones(512, dtype=bf, device="cuda")

    def calls(i):
        n = Q.rms_norm(x[i], w, quantize=Q.MXFP8, keep=True, bf16=True)
        dx, dw = Q.rms_norm_backward(x[i], n.sum, w, n.rstd)
        b = Q.moe_balance_loss(x[i][:, :64].contiguous(), ids[i], 0.1)
        return [Q.orthogonalize(g[i]), n.y, n.q.codes, dx, dw, b.loss, b.counts, b.slope]

    want = [calls(0), calls(1)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for i, s in enumerate(sides):
            with torch.cuda.stream(s):
                got.append(calls(i))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_the_norm_feeds_the_mxfp4_block():
    """The norm's MXFP4 output is what the products take: the same bits as quantizing the fp32 norm, and as moe_mxfp4_gemm's own rows."""
    d = inputs(4)
    n = Q.rms_norm(d["delta"], d["weight"], residual=d["stream"], quantize=Q.MXFP4, bf16=True)
    assert n.q.codes.shape == (T, H // 2) and n.q.scales.shape == (T, H // 32)
    offs = torch.tensor([0, 300, 300, T], dtype=torch.int32, device="cuda")
    w = Q.quantize_mxfp4(d["w_gate_up"][:3].contiguous())
    y = Q.moe_mxfp4_gemm(n.q, w, offs, epilogue=Q.EPI_SWIGLU, y_dtype=bf)
    values, weights = Q.dequantize_mxfp4(n.q, f32), Q.dequantize_mxfp4(w, f32)
    for e, (a, b) in enumerate(((0, 300), (300, 300), (300, T))):
        z = values[a:b].double() @ weights[e].double().t()
        g, u = z.chunk(2, 1)
        want = g * torch.sigmoid(g) * u
        # fp32 sums of H products: H u sum |x w| each, carried through h = silu(g) u; then half a step of bf16
        z_off = H * 2.0 ** -24 * (values[a:b].abs().double() @ weights[e].abs().double().t())
        g_off, u_off = z_off.chunk(2, 1)
        off = 1.1 * g_off * (u.abs() + u_off) + (g * torch.sigmoid(g)).abs() * u_off + (7 + 1.23 * g.abs()) * 2.0 ** -24 * want.abs()
        assert ((y[a:b].double() - want).abs() <= 2.0 ** -8 * (want.abs() + off) + off).all()
