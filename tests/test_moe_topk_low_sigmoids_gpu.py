"""Sigmoid routing of tokens whose logits are all far below 0 (padding behind a
finite mask, a router that closes everything): the chosen scores over their sum, and
the scores' shares of the row, stay what the definition gives, although the scores
themselves leave fp32's range.

The definition in 64 bits by logarithms: sigmoid(x_j) / sum = softmax of log
sigmoid(x).  Tolerances, in roundings U = 2^-24, of a share: 3 |d| + 3 sum w |d| for exp
of differences (d the distance from the largest log sigmoid), 64 for the sums and
quotients, and 2^-26 = U / 4 where exp(x) stands for the sigmoid; shares below 2^-99
may be 0."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F, D = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24
INF = float("inf")


def _rows(G, dtype):
    gen = torch.Generator(device="cuda").manual_seed(G)
    x = 3.0 * torch.randn((14, G), device="cuda", generator=gen)
    for i, low in enumerate((-17, -20, -60, -87.5, -95, -103, -200, -5000)):
        x[i] += low
    x[8], x[9], x[10] = -100.0, -1e9, torch.finfo(dtype).min
    x[11] = -200.0
    x[11, G // 2:] = -INF
    x[12] = -INF
    return x.to(dtype)


def _shares(l):
    return torch.where(torch.isneginf(l).all(1, keepdim=True), torch.zeros_like(l), torch.softmax(l, 1))


def _bound(w, l):
    gap = (l.max(1, keepdim=True).values - l).nan_to_num(nan=0.0, posinf=1e4).clamp(max=1e4)
    return w * (3 * gap + 3 * (w * gap).sum(1, keepdim=True) + 66) * U + 2.0 ** -99


@pytest.mark.parametrize("with_bias", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("G,k", [(8, 2), (100, 6), (256, 8), (1024, 32)])
def test_shares(cuda_lib, G, k, dtype, with_bias):
    x = _rows(G, dtype)
    bias = torch.linspace(0.1, 0, G, device="cuda") if with_bias else None
    l = torch.nn.functional.logsigmoid(x.to(D))
    w, ids, _, total = cuda_lib.mx_moe_topk(x, k, cuda_lib.SCORE_SIGMOID, bias, stats=True)
    again, _, _, _ = cuda_lib.mx_moe_topk(x, k, cuda_lib.SCORE_SIGMOID, bias)
    assert torch.equal(again, w)
    c = l.gather(1, ids.long())
    ref = _shares(c)
    assert ((w.to(D) - ref).abs() <= _bound(ref, c)).all()
    q = _shares(l)
    assert ((total.to(D) - q.sum(0)).abs() <= (_bound(q, l) + len(x) * U * q).sum(0)).all()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("G,k", [(8, 2), (100, 6), (256, 8), (1024, 32)])
def test_gradient(cuda_lib, G, k, dtype):
    x = _rows(G, dtype)
    gen = torch.Generator(device="cuda").manual_seed(1)
    a, v = torch.randn((len(x), k), device="cuda", generator=gen), torch.randn(G, device="cuda", generator=gen)
    _, ids, _, _ = cuda_lib.mx_moe_topk(x, k, cuda_lib.SCORE_SIGMOID)
    l = torch.nn.functional.logsigmoid(x.to(D))
    slope = torch.sigmoid(-x.to(D))
    w, q = _shares(l.gather(1, ids.long())), _shares(l)
    for dsum in (None, v):
        got = cuda_lib.mx_moe_topk_bwd(x, ids, a, cuda_lib.SCORE_SIGMOID, dscore_sum=dsum)
        b = a.to(D)
        parts, off_w = w * (b - (w * b).sum(1, keepdim=True)), _bound(w, l.gather(1, ids.long()))
        # w_j's error times |b_j - A|, and w_j times that of A = sum w b
        err = b.abs().max() * (2 * off_w + w * (2 * off_w.sum(1, keepdim=True) + 64 * U))
        ref = torch.zeros_like(q).scatter_add_(1, ids.long(), parts)
        bound = torch.zeros_like(q).scatter_add_(1, ids.long(), err)
        if dsum is not None:
            d = v.to(D)
            ref = ref + q * (d - (q * d).sum(1, keepdim=True))
            off_q = _bound(q, l)
            bound = bound + d.abs().max() * (2 * off_q + q * (2 * off_q.sum(1, keepdim=True) + 64 * U))
        ref, bound = ref * slope, bound * slope
        off = (got.to(D) - ref).abs()
        assert (off <= bound + (2.0 ** -8 if dtype == BF else U) * ref.abs() + 2.0 ** -98).all()
