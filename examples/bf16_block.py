"""A transformer block's two MLPs in BF16, trained for a few steps.

A dense MLP with a residual (``mx_linear_fwd``: bias, activation and residual
in the products' epilogues, the pre-activation kept in 8 bits) and a routed
expert MLP (``mx_ragged_gemm`` on unpadded segments, SwiGLU with its input kept
in 8 bits), with their backward passes from the 8-bit checkpoints and fp32
main gradients accumulated over microbatches.

    python3 examples/bf16_block.py [--steps 8] [--tokens 4096]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mlp_gemms_gb300 as mx  # noqa: E402


class DenseMlp:
    """x + W2 gelu(W1 x + b1) + b2.  Keeps x, the activation's input in 8
    bits and nothing of its output: the backward pass computes it again."""

    def __init__(self, d, f, gen, device="cuda"):
        self.w1 = (torch.randn((f, d), generator=gen) * d ** -0.5).to(torch.bfloat16).to(device)
        self.w2 = (torch.randn((d, f), generator=gen) * f ** -0.5).to(torch.bfloat16).to(device)
        self.b1 = torch.zeros(f, dtype=torch.bfloat16, device=device)
        self.b2 = torch.zeros(d, dtype=torch.bfloat16, device=device)
        self.grads = {n: torch.zeros(getattr(self, n).shape, device=device) for n in ("w1", "w2", "b1", "b2")}

    def forward(self, x):
        self.x = x
        self.ckpt = mx.MX(x.shape[0], self.w1.shape[0])
        a = mx.mx_linear_fwd(x, self.w1, self.b1, mx.ACT_GELU_TANH, ckpt=self.ckpt)
        return mx.mx_linear_fwd(a, self.w2, self.b2, mx.ACT_NONE, residual=x)

    def backward(self, dy):
        da = mx.mx_ragged_gemm(dy, self.w2[None], None, layout=mx.W_KN)
        dz, a, db1 = mx.mx_act_ckpt_bwd(self.ckpt, mx.ACT_GELU_TANH, da, recompute=True, colsum=True)
        mx.mx_ragged_gemm_wgrad_f32(dy, a, 1, None, self.grads["w2"][None], accumulate=True)
        mx.mx_ragged_gemm_wgrad_f32(dz, self.x, 1, None, self.grads["w1"][None], accumulate=True)
        self.grads["b1"] += db1
        self.grads["b2"] += dy.float().sum(0)
        return mx.mx_ragged_gemm(dz, self.w1[None], None, layout=mx.W_KN) + dy


class ExpertMlp:
    """sum over a token's choices j of p_j W2[e_j] swiglu(W1[e_j] x), on
    segments of whatever length the routing gives."""

    def __init__(self, experts, d, f, gen, device="cuda"):
        self.G = experts
        self.w1 = (torch.randn((experts, 2 * f, d), generator=gen) * d ** -0.5).to(torch.bfloat16).to(device)
        self.w2 = (torch.randn((experts, d, f), generator=gen) * f ** -0.5).to(torch.bfloat16).to(device)
        self.grads = {n: torch.zeros(getattr(self, n).shape, device=device) for n in ("w1", "w2")}

    def forward(self, x, topk, probs):
        """topk [T, k] expert ids, probs [T, k] fp32."""
        T, k = topk.shape
        order = torch.argsort(topk.reshape(-1), stable=True)
        self.src = order // k
        self.row_of = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device=x.device)).to(
            torch.int32).view(T, k)
        self.offsets = torch.bincount(topk.reshape(-1), minlength=self.G).cumsum(0).to(torch.int32)
        self.p = probs.reshape(-1)[order].unsqueeze(1)
        self.xs = x[self.src]
        z = mx.mx_ragged_gemm(self.xs, self.w1, self.offsets)
        h, self.ckpt = mx.mx_act_ckpt_fwd(z, mx.ACT_SWIGLU)      # z and h end here
        y = mx.mx_ragged_gemm(h, self.w2, self.offsets)
        return mx.mx_moe_unpermute(y, self.row_of, probs)

    def backward(self, dout):
        dy = (dout[self.src] * self.p).to(torch.bfloat16)
        dh = mx.mx_ragged_gemm(dy, self.w2, self.offsets, layout=mx.W_KN)
        dz, h, _ = mx.mx_act_ckpt_bwd(self.ckpt, mx.ACT_SWIGLU, dh, recompute=True)
        mx.mx_ragged_gemm_wgrad_f32(dy, h, self.G, self.offsets, self.grads["w2"], accumulate=True)
        mx.mx_ragged_gemm_wgrad_f32(dz, self.xs, self.G, self.offsets, self.grads["w1"], accumulate=True)
        dxs = mx.mx_ragged_gemm(dz, self.w1, self.offsets, layout=mx.W_KN)
        return mx.mx_moe_unpermute(dxs, self.row_of)


class Block:
    """The dense MLP, then the experts with a residual."""

    def __init__(self, d, f, experts, f_expert, gen):
        self.dense, self.experts = DenseMlp(d, f, gen), ExpertMlp(experts, d, f_expert, gen)

    def forward(self, x, topk, probs):
        t = self.dense.forward(x)
        return t + self.experts.forward(t, topk, probs)

    def backward(self, dy):
        return self.dense.backward(dy + self.experts.backward(dy))

    def parameters(self):
        for part in (self.dense, self.experts):
            for name, grad in part.grads.items():
                yield getattr(part, name), grad

    def saved_bytes(self):
        """(of the two checkpoints, of the same tensors in BF16)"""
        cks = (self.dense.ckpt, self.experts.ckpt)
        return sum(c.data.numel() + c.scale.numel() for c in cks), sum(2 * c.rows * c.cols for c in cks)


def train(steps=8, tokens=4096, d=512, f=2048, experts=16, f_expert=256, k=2, microbatches=2, lr=0.01, seed=0):
    """Fits a fixed random target; returns the loss of every step and the block."""
    gen = torch.Generator().manual_seed(seed)
    block = Block(d, f, experts, f_expert, gen)
    batches = []
    for _ in range(microbatches):
        x = torch.randn((tokens, d), generator=gen).to(torch.bfloat16).cuda()
        target = (torch.randn((tokens, d), generator=gen) * 0.5).cuda()
        score = torch.randn((tokens, experts), generator=gen) + torch.arange(experts) * -0.2   # uneven experts
        probs, topk = torch.topk(torch.softmax(score, -1), k)
        batches.append((x, target, topk.to(torch.int32).cuda(), probs.contiguous().cuda()))
    losses = []
    for _ in range(steps):
        loss = 0.0
        for x, target, topk, probs in batches:
            err = block.forward(x, topk, probs).float() - target
            loss += float(err.square().mean()) / microbatches
            block.backward((err / (tokens * microbatches)).to(torch.bfloat16))
        for w, grad in block.parameters():
            w.copy_((w.float() - lr * grad).to(torch.bfloat16))
            grad.zero_()
        losses.append(loss)
    assert mx.mx_get_device_status() == "MX_OK"
    return losses, block


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=4096)
    a = ap.parse_args()
    losses, block = train(a.steps, a.tokens)
    for i, v in enumerate(losses):
        print("step %d loss %.4f" % (i, v))
    kept, bf16 = block.saved_bytes()
    print("activations kept: %.1f MB in 8 bits, %.1f MB in BF16" % (kept / 1e6, bf16 / 1e6))


if __name__ == "__main__":
    main()
