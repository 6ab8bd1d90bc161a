"""The BF16 layers together (examples/bf16_block.py): the block's gradients
against autograd of the same block in fp64 without any quantization, a few
training steps, and one token through the layers as a decode step."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(cuda_lib):
    spec = importlib.util.spec_from_file_location("bf16_block", os.path.join(ROOT, "examples", "bf16_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _reference(block, x, topk, probs):
    """The block in fp64 with autograd leaves."""
    leaves = {n: getattr(block.dense, n).double().requires_grad_() for n in ("w1", "w2", "b1", "b2")}
    experts = {n: getattr(block.experts, n).double().requires_grad_() for n in ("w1", "w2")}
    x = x.double().requires_grad_()
    z = x @ leaves["w1"].T + leaves["b1"]
    t = x + torch.nn.functional.gelu(z, approximate="tanh") @ leaves["w2"].T + leaves["b2"]
    out = t
    for j in range(topk.shape[1]):
        w1, w2 = experts["w1"][topk[:, j].long()], experts["w2"][topk[:, j].long()]
        g, u = torch.einsum("tfd,td->tf", w1, t).chunk(2, -1)
        out = out + probs[:, j:j + 1].double() * torch.einsum("tdf,tf->td", w2, torch.nn.functional.silu(g) * u)
    return x, leaves, experts, out


def _off(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_block_gradients(example):
    """E4M3 keeps 4 bits: a relative error of at most 2^-4 per value of the
    checkpoint, 2^-5 in the mean square; it enters the slopes and the
    recomputed activations once, so gradients are within 5 % in the 2-norm
    (BF16 rounding, 2^-9, is below that).  The output has only BF16 roundings."""
    gen = torch.Generator().manual_seed(3)
    T, d, G, k = 97, 64, 6, 2
    block = example.Block(d, 160, G, 96, gen)
    block.dense.b1 += 0.1
    x = torch.randn((T, d), generator=gen).to(torch.bfloat16).cuda()
    probs, topk = torch.topk(torch.softmax(torch.randn((T, G - 1), generator=gen), -1), k)   # expert 5 gets no token
    topk, probs = topk.to(torch.int32).cuda(), probs.contiguous().cuda()
    dy = torch.randn((T, d), generator=gen).to(torch.bfloat16).cuda()
    out = block.forward(x, topk, probs)
    dx = block.backward(dy)
    rx, leaves, experts, rout = _reference(block, x, topk, probs)
    rout.backward(dy.double())
    assert _off(out, rout.detach()) < 0.01
    assert _off(dx, rx.grad) < 0.05
    for n, leaf in leaves.items():
        assert _off(block.dense.grads[n], leaf.grad) < 0.05, n
    for n, leaf in experts.items():
        assert _off(block.experts.grads[n], leaf.grad) < 0.05, n
        assert not bool(block.experts.grads[n][G - 1].any())


def test_training_reduces_the_loss(example):
    losses, block = example.train(steps=6, tokens=1000, d=128, f=512, experts=8, f_expert=96)
    assert losses[-1] < 0.9 * losses[0]
    kept, bf16 = block.saved_bytes()
    assert kept < 0.56 * bf16


def test_one_token(example, cuda_lib):
    """A decode step gives the same token the same result as a batch does, to
    the rounding of BF16 between the layers."""
    gen = torch.Generator().manual_seed(8)
    d, G, k, T = 256, 16, 4, 300
    block = example.Block(d, 512, G, 128, gen)
    x = torch.randn((T, d), generator=gen).to(torch.bfloat16).cuda()
    probs, topk = torch.topk(torch.softmax(torch.randn((T, G), generator=gen), -1), k)
    topk, probs = topk.to(torch.int32).cuda(), probs.contiguous().cuda()
    full = block.forward(x, topk, probs)
    one = block.forward(x[7:8], topk[7:8].contiguous(), probs[7:8].contiguous())
    assert _off(one, full[7:8].double()) < 0.01
