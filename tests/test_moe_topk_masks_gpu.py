"""Routing of logits masked by large finite values, of logits in the millions and of
BF16 logits all below 0: softmax weights depend on differences alone, so they are
finite, those of tokens masked throughout equal shares.

Tolerances, in roundings U = 2^-24.  exp(x - top): the difference, its product with
log2 e and that constant, each |x - top| U, and the hardware's power of two, 4 U.  A
sum of n such terms: their errors weighed by their shares, and n / 32 + 5 additions;
the quotient: 4.  So a weight w_j is off by w_j (3 |d_j| + 3 sum w |d| + 20 + n / 32) U,
d the distance from the largest, and by nothing more than 2^-125 where exp leaves
fp32's normal range."""
import pytest
import torch

from test_moe_topk_gpu import _choose

pytestmark = pytest.mark.gpu

BF, F, D = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24
INF = float("inf")


def _masked(G, k, dtype, low):
    """Ordinary tokens, tokens masked throughout, and tokens with fewer than k experts left."""
    gen = torch.Generator(device="cuda").manual_seed(G + k)
    x = torch.randn((24, G), device="cuda", generator=gen)
    x[3], x[17], x[23] = low, low, low
    x[5, 1:], x[11, :G - 1] = low, low
    x[8, max(1, k - 1):] = low
    return x.to(dtype)


def _expect(x, ids, renorm):
    """(weights, their bound, score sums, their bound) in 64 bits."""
    d = x.to(D)
    p = torch.softmax(d, 1)
    gap = (d.max(1, keepdim=True).values - d).clamp(max=1e4)
    # shares of closed terms are 0, so their distance does not count
    row = (p * gap).sum(1, keepdim=True)
    rel = (3 * gap + 3 * row + 20 + x.shape[1] / 32) * U
    s = p.gather(1, ids)
    w = s / s.sum(1, keepdim=True) if renorm else s
    return w, w * rel.gather(1, ids) * 2 + 2.0 ** -125, p.sum(0), (p * (rel + x.shape[0] * U)).sum(0) + 2.0 ** -120


def _check(mx, x, k):
    want = _choose(x.to(D), k, False, None, 1, 1, 1)
    for renorm in (True, False):
        for stats in (True, False):
            w, ids, load, total = mx.mx_moe_topk(x, k, renorm=renorm, stats=stats)
            assert torch.equal(ids.long(), want)
            ref, bound, sums, sums_bound = _expect(x, want, renorm)
            assert torch.isfinite(w).all()
            assert ((w.to(D) - ref).abs() <= bound).all(), (renorm, stats)
            if stats:
                assert torch.equal(load.long(), torch.bincount(want.reshape(-1), minlength=x.shape[1]))
                assert ((total.to(D) - sums).abs() <= sums_bound).all()


@pytest.mark.parametrize("low", [-1e9, -1e30, "lowest"])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("G,k", [(8, 3), (31, 4), (128, 8), (256, 8), (384, 6), (1024, 32)])
def test_finite_masks(cuda_lib, G, k, dtype, low):
    _check(cuda_lib, _masked(G, k, dtype, torch.finfo(dtype).min if low == "lowest" else low), k)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("G,k", [(8, 2), (128, 8), (256, 8), (1024, 4)])
def test_logits_in_the_millions(cuda_lib, G, k, dtype):
    """Steps of one and less around 5e6 and -5e6, as far as the type tells them apart."""
    gen = torch.Generator(device="cuda").manual_seed(G)
    x = torch.randint(-6, 7, (40, G), device="cuda", generator=gen) * 0.5
    x[:20] += 5e6
    x[20:] -= 5e6
    x[30:] *= 2
    _check(cuda_lib, x.to(dtype), k)


@pytest.mark.parametrize("G", [8, 128, 256, 1024])
def test_negative_bf16_maxima(cuda_lib, G):
    gen = torch.Generator(device="cuda").manual_seed(G)
    x = -(torch.rand((40, G), device="cuda", generator=gen) + 1) * torch.logspace(-3, 8, 40, device="cuda")[:, None]
    _check(cuda_lib, x.to(BF), 4)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("G", [8, 128, 1024])
def test_a_row_of_one_value_is_a_row_of_zeros(cuda_lib, G, dtype):
    """Weights, score sums and gradients to the bit, with and without a bias and groups."""
    values = [0.0, -1e9, -1e30, 1e7, float(torch.finfo(dtype).min), float(torch.finfo(dtype).max)]
    gen = torch.Generator(device="cuda").manual_seed(2)
    a = torch.randn((1, 4), device="cuda", generator=gen)
    bias, v = (torch.randn(G, device="cuda", generator=gen) for _ in range(2))
    for kw in (dict(), dict(renorm=False), dict(bias=bias), dict(bias=bias, groups=4, topk_groups=2, group_top=2)):
        first = None
        for value in values:
            x = torch.full((1, G), value, device="cuda").to(dtype)
            w, ids, load, total = cuda_lib.mx_moe_topk(x, 4, stats=True, **kw)
            renorm = kw.get("renorm", True)
            got = (w, ids, load, total, cuda_lib.mx_moe_topk_bwd(x, ids, a, renorm=renorm),
                   cuda_lib.mx_moe_topk_bwd(x, ids, a, renorm=renorm, dscore_sum=v))
            first = got if first is None else first
            assert all(torch.equal(p, q) for p, q in zip(got, first)), (kw, value)
