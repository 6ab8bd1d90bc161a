"""The order of exact values where a value away from the border has the largest
error: a group whose biases cancel beside two ordinary ones at the border."""
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
