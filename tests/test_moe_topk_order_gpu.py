"""The order of exact values where a value away from the border has the largest
error: a group whose biases cancel beside two ordinary ones at the border, and an expert
of a large score, cancelled by its bias, behind two of scores near 0."""
import pytest
import torch

from test_moe_topk_gpu import _choose

pytestmark = pytest.mark.gpu

D = torch.float64


def _same(mx, x, k, sigmoid, bias, groups, kept, top):
    score = mx.SCORE_SIGMOID if sigmoid else mx.SCORE_SOFTMAX
    _, ids, _, _ = mx.mx_moe_topk(x, k, score, bias, groups, kept, top)
    return int((ids.long() != _choose(x.to(D), k, sigmoid, bias, groups, kept, top)).any(1).sum())


@pytest.mark.parametrize("G", [64, 60])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_a_cancelling_group_behind_two_ordinary_ones(cuda_lib, sigmoid, G):
    """Groups of two.  The border lies between two ordinary groups 1.6e-5 apart; a third
    group's biases of 1000 and -999 leave its fp32 value off by up to 6e-5."""
    step = 2.0 ** -14                      # of fp32 values near 1000
    bias = torch.full((G,), -1.0, device="cuda")
    bias[:8] = 1.0                         # four groups far above
    bias[20], bias[21] = 0.5, 0.5 + 1.7e-5
    bias[22], bias[23] = 0.5, 0.5 + 1e-6
    bias[40], bias[41] = 1000.0, -999.0
    x = torch.zeros((64, 64, G), device="cuda")
    sweep = torch.linspace(-step, step, 64, device="cuda") * (4 if sigmoid else G)
    x[:, :, 40], x[:, :, 41] = sweep[:, None], sweep
    assert _same(cuda_lib, x.view(-1, G), 10, sigmoid, bias, G // 2, 5, 2) == 0


@pytest.mark.parametrize("G,groups", [(64, 1), (256, 1), (64, 4), (60, 5)])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_a_large_score_that_its_bias_cancels(cuda_lib, sigmoid, G, groups):
    """Experts 0 and 16 have scores of exp(-100) and biases of 3e-8 and 1e-8; expert
    40's score is about 0.6 and its bias as much below 0: an fp32 sum in steps of 6e-8."""
    x = torch.full((160, G), -float("inf"), device="cuda")
    x[:, 0] = x[:, 16] = -100.0
    x[:, G - 5] = 0.0
    wrong = 0
    for i in range(16):
        s = 0.55 + 0.01 * i
        logit = torch.tensor(s / (1 - s), dtype=D).log().item()
        x[:, 40] = logit + torch.linspace(-80, 80, 160, device="cuda") * 2.0 ** -25
        bias = torch.full((G,), -5.0, device="cuda")
        bias[0], bias[16], bias[40] = 3e-8, 1e-8, -s
        wrong += _same(cuda_lib, x, 1, sigmoid, bias, groups, max(1, groups - 1), 1)
    assert wrong == 0, "%d tokens" % wrong
