"""A routed expert layer with everything around it: the norm with the residual
stream, a learned router with a balancing term, the experts and their combine,
trained in BF16 and served in 4 bits.

    python3 examples/routed_block.py [--steps 8] [--tokens 4096]

``RoutedBlock.forward`` and ``backward`` train (the experts' products in BF16 on
the routing index's padded segments, the activation's input kept in 8 bits);
``serve`` runs the same layer with the experts' weights and activations in 4 bits.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mlp_gemms_gb300 as mx  # noqa: E402


class RoutedBlock:
    """s = x + residual; out = s + sum over a token's choices j of w_j
    W2[e_j] swiglu(W1[e_j] norm(s)), with experts e and weights w from Wr norm(s)."""

    def __init__(self, d, experts, f, k, gen, device="cuda"):
        self.G, self.k = experts, k

        def rand(*shape, std):
            return (torch.randn(shape, generator=gen) * std).to(torch.bfloat16).to(device)

        self.norm_w = torch.ones(d, dtype=torch.bfloat16, device=device)
        self.norm_b = torch.zeros(d, dtype=torch.bfloat16, device=device)
        self.wr = rand(experts, d, std=d ** -0.5)
        self.w1 = rand(experts, 2 * f, d, std=d ** -0.5)
        self.w2 = rand(experts, d, f, std=f ** -0.5)
        self.grads = {n: torch.zeros(getattr(self, n).shape, device=device) for n in ("norm_w", "norm_b", "wr", "w1", "w2")}

    def _route(self, y):
        """Weights and rows of the tokens' choices, and the experts' segments."""
        self.logits = mx.mx_linear_fwd(y, self.wr)
        self.weights, self.ids, self.load, self.share = mx.mx_moe_topk(self.logits, self.k, stats=True)
        self.offsets, self.src, self.row_of = mx.mx_moe_route_index(self.ids, self.G)

    def forward(self, x, residual):
        self.y, self.mean, self.rstd, self.s = mx.mx_layernorm_fwd(x, self.norm_w, self.norm_b, residual=residual)
        self._route(self.y)
        self.xs = self.y[self.src.clamp(min=0).long()] * (self.src >= 0).unsqueeze(1)
        z = mx.mx_ragged_gemm(self.xs, self.w1, self.offsets)
        h, self.ckpt = mx.mx_act_ckpt_fwd(z, mx.ACT_SWIGLU)
        self.o = mx.mx_ragged_gemm(h, self.w2, self.offsets)
        return self.s + mx.mx_moe_unpermute(self.o, self.row_of, self.weights)

    def balance(self, strength):
        """The balancing term strength * G * sum over experts of (share of the
        choices) * (share of the scores), and its gradient of the score sums."""
        T = self.logits.shape[0]
        chosen = self.load.float() / (T * self.k)
        return strength * self.G * (chosen * self.share / T).sum(), strength * self.G * chosen / T

    def backward(self, dout, dshare=None):
        """Returns the gradient of x (and of the residual: it is the same)."""
        do, dweights = mx.mx_moe_unpermute_bwd(dout, self.o, self.row_of, self.weights, src=self.src)
        dh = mx.mx_ragged_gemm(do, self.w2, self.offsets, layout=mx.W_KN)
        dz, h, _ = mx.mx_act_ckpt_bwd(self.ckpt, mx.ACT_SWIGLU, dh, recompute=True)
        mx.mx_ragged_gemm_wgrad_f32(do, h, self.G, self.offsets, self.grads["w2"], accumulate=True)
        mx.mx_ragged_gemm_wgrad_f32(dz, self.xs, self.G, self.offsets, self.grads["w1"], accumulate=True)
        dy = mx.mx_moe_unpermute(mx.mx_ragged_gemm(dz, self.w1, self.offsets, layout=mx.W_KN), self.row_of)
        dlogits = mx.mx_moe_topk_bwd(self.logits, self.ids, dweights, dscore_sum=dshare)
        mx.mx_ragged_gemm_wgrad_f32(dlogits, self.y, 1, None, self.grads["wr"][None], accumulate=True)
        dy = dy + mx.mx_ragged_gemm(dlogits, self.wr[None], None, layout=mx.W_KN)
        dx, _, _ = mx.mx_layernorm_bwd(dy, self.s, self.mean, self.rstd, self.norm_w, dres=dout, accumulate=True,
                                       dweight=self.grads["norm_w"], dbias=self.grads["norm_b"])
        return dx

    def quantize(self):
        """The experts' weights in 4 bits, once, for serve()."""
        self.q1 = mx.mx_nvfp4_quantize(self.w1.flatten(0, 1))
        self.q2 = mx.mx_nvfp4_quantize(self.w2.flatten(0, 1))

    def serve(self, x, residual):
        y, _, _, s = mx.mx_layernorm_fwd(x, self.norm_w, self.norm_b, residual=residual, stats=False)
        self._route(y)
        a = mx.mx_nvfp4_quantize(y, src=self.src, offsets=self.offsets)
        h, _ = mx.mx_act_ckpt_fwd(mx.mx_nvfp4_gemm(a, self.q1, self.G, self.offsets), mx.ACT_SWIGLU)
        o = mx.mx_nvfp4_gemm(mx.mx_nvfp4_quantize(h, offsets=self.offsets), self.q2, self.G, self.offsets)
        return s + mx.mx_moe_unpermute(o, self.row_of, self.weights)


def train(steps=8, tokens=4096, d=512, experts=16, f=256, k=2, lr=0.01, strength=0.01, seed=0):
    """Fits a fixed random target; returns the loss of every step and the block."""
    gen = torch.Generator().manual_seed(seed)
    block = RoutedBlock(d, experts, f, k, gen)
    x, residual = ((torch.randn((tokens, d), generator=gen)).to(torch.bfloat16).cuda() for _ in range(2))
    target = (torch.randn((tokens, d), generator=gen) * 0.5).cuda()
    losses = []
    for _ in range(steps):
        err = block.forward(x, residual).float() - target
        term, dshare = block.balance(strength)
        losses.append(float(err.square().mean() + term))
        block.backward((err / tokens).to(torch.bfloat16), dshare)
        for name, grad in block.grads.items():
            w = getattr(block, name)
            w.copy_((w.float() - lr * grad).to(torch.bfloat16))
            grad.zero_()
    assert mx.mx_get_device_status() == "MX_OK"
    return losses, block, x, residual


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=4096)
    a = ap.parse_args()
    losses, block, x, residual = train(a.steps, a.tokens)
    for i, v in enumerate(losses):
        print("step %d loss %.4f" % (i, v))
    block.quantize()
    full, four = block.forward(x, residual).float(), block.serve(x, residual).float()
    print("served in 4 bits: off by %.3f of the layer's own output" % float((full - four).norm() / (full - block.s).norm()))


if __name__ == "__main__":
    main()
