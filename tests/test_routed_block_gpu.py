"""The layers together, as examples/routed_block.py runs them: norm, router, routing
index, experts, combine, and back; and the same layer in 4 bits.

Tolerances (2-norms).  The gradients pass up to six BF16 roundings (2^-9 of the
values each, the sums' terms independent) and the 8-bit checkpoint: z off by up to
2^-4 of its value, 2^-4 / sqrt(3) of its norm, through slopes of order one in two
factors.  2 * 2^-4 / sqrt(3) + 6 * 2^-9 = 0.084."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

D = torch.float64


def _block(d=256, experts=8, f=128, k=3, T=333, seed=0):
    import routed_block
    gen = torch.Generator().manual_seed(seed)
    b = routed_block.RoutedBlock(d, experts, f, k, gen)
    b.norm_w.copy_(1 + 0.1 * torch.randn(d, generator=gen))
    b.norm_b.copy_(0.1 * torch.randn(d, generator=gen))
    x, res, dout = (torch.randn((T, d), generator=gen).to(torch.bfloat16).cuda() for _ in range(3))
    return b, x, res, dout


def _reference(b, x, res, ids):
    """The layer's formula in 64 bits with the choices given; (leaves, output, score shares)."""
    leaves = {n: getattr(b, n).to(D).requires_grad_(True) for n in b.grads}
    xs = x.to(D).requires_grad_(True)
    s = xs + res.to(D)
    m = s.mean(1, keepdim=True)
    y = (s - m) * ((s - m).square().mean(1, keepdim=True) + 1e-5).rsqrt() * leaves["norm_w"] + leaves["norm_b"]
    p = torch.softmax(y @ leaves["wr"].T, 1)
    w = p.gather(1, ids.long())
    w = w / w.sum(1, keepdim=True)
    out = s
    for j in range(ids.shape[1]):
        w1, w2 = leaves["w1"][ids[:, j].long()], leaves["w2"][ids[:, j].long()]
        g, u = torch.einsum("td,tfd->tf", y, w1).chunk(2, 1)
        out = out + w[:, j:j + 1] * torch.einsum("tf,tdf->td", g * torch.sigmoid(g) * u, w2)
    return leaves, xs, out, p.sum(0)


def _off(got, ref):
    return float((got.to(D) - ref).norm() / ref.norm())


def test_forward_and_gradients(cuda_lib):
    b, x, res, dout = _block()
    out = b.forward(x, res)
    _, dshare = b.balance(0.5)
    dx = b.backward(dout, dshare)
    leaves, xs, ref, share = _reference(b, x, res, b.ids)
    assert _off(out, ref.detach()) < 0.02 and _off(b.share, share.detach()) < 0.01
    loss = (ref * dout.to(D)).sum() + (share * dshare.to(D)).sum()
    grads = dict(zip(list(leaves) + ["x"], torch.autograd.grad(loss, list(leaves.values()) + [xs])))
    for name, g in b.grads.items():
        assert _off(g, grads[name]) < 0.084, name
    assert _off(dx, grads["x"]) < 0.084
    assert cuda_lib.mx_get_device_status() == "MX_OK"


def test_gradients_add_up(cuda_lib):
    b, x, res, dout = _block(T=100)
    b.forward(x, res)
    b.backward(dout)
    once = {n: g.clone() for n, g in b.grads.items()}
    b.backward(dout)
    for n, g in b.grads.items():
        assert torch.equal(g, once[n] + once[n]), n


def test_gradient_of_the_router_against_differences(cuda_lib):
    """sum(dout * out) moves by the router's gradient when its logits do: the choices
    stay, the weights and so the combine move (64-bit differences of the formula
    against the layer's own backward pass)."""
    b, x, res, dout = _block(T=64, seed=3)
    b.forward(x, res)
    b.backward(dout)
    step = torch.randn(b.wr.shape, generator=torch.Generator().manual_seed(4)).cuda().to(D) * 1e-4
    wr = b.wr
    values = []
    for sign in (1, -1):
        b.wr = wr.to(D) + sign * step
        _, _, ref, _ = _reference(b, x, res, b.ids)
        values.append(float((ref.detach() * dout.to(D)).sum()))
    b.wr = wr
    moved = values[0] - values[1]
    assert abs(moved - 2 * float((b.grads["wr"].to(D) * step).sum())) < 0.084 * 2 * float(
        b.grads["wr"].to(D).norm() * step.norm())


@pytest.mark.parametrize("T", [1, 5, 128, 700])
def test_served_in_4_bits(cuda_lib, T):
    """Against the layer computed from the 4-bit values: the products' operands are
    exactly those, what lies between is rounded to BF16 (and again to 4 bits)."""
    b, x, res, _ = _block(T=T)
    full = b.forward(x, res).float()
    b.quantize()
    four = b.serve(x, res).float()
    assert torch.isfinite(four).all()
    own = full - b.s.float()
    assert float((four - full).norm() / own.norm()) < 0.35  # three quantizations of 0.1 each, one behind the other
    again = b.serve(x, res).float()
    assert torch.equal(four, again)


def test_served_tokens_do_not_depend_on_their_batch(cuda_lib):
    b, x, res, _ = _block(T=90)
    b.quantize()
    whole, some = b.serve(x, res), b.serve(x[30:47].contiguous(), res[30:47].contiguous())
    assert torch.equal(whole[30:47], some)


def test_trains(cuda_lib):
    import routed_block
    losses, block, _, _ = routed_block.train(steps=3, tokens=600, d=256, experts=8, f=128)
    assert len(losses) == 3 and all(v == v for v in losses)


def test_a_captured_step(cuda_lib):
    """Forward and backward replayed from a graph on new inputs."""
    b, x, res, dout = _block(T=200)
    inputs = [(x.clone(), res.clone(), dout.clone()), tuple(t.flip(0).contiguous() for t in (x, res, dout))]
    want = []
    for i in inputs:
        out = b.forward(i[0], i[1])
        want.append((out, b.backward(i[2])))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.backward(dout) if b.forward(x, res) is not None else None
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.forward(x, res)
        dx = b.backward(dout)
    for i, w in zip(inputs, want):
        for t, v in zip((x, res, dout), i):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w[0]) and torch.equal(dx, w[1])
