"""Equal logits with equal biases are equal, whichever of a lane's experts they are: the
lowest index comes first, in every layout of the experts and with groups."""
import pytest
import torch

from test_moe_topk_gpu import _choose

pytestmark = pytest.mark.gpu

D = torch.float64


@pytest.mark.parametrize("G,groups,kept", [(8, 1, 1), (60, 1, 1), (64, 1, 1), (128, 1, 1), (256, 1, 1), (1000, 1, 1), (64, 32, 9),
                                           (60, 30, 9), (256, 8, 4), (160, 8, 3), (384, 8, 4), (1024, 16, 3), (96, 3, 2)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_rows_of_few_values(cuda_lib, sigmoid, dtype, G, groups, kept):
    """Every row holds one to three values, and so do the biases: ties everywhere."""
    gen = torch.Generator(device="cuda").manual_seed(G)
    T = 600
    few = torch.randn((T, 3), device="cuda", generator=gen)
    pick = torch.randint(0, 3, (T, G), device="cuda", generator=gen)
    pick[:200] = 0
    pick[200:400] %= 2
    x = few.gather(1, pick).to(dtype)
    score = cuda_lib.SCORE_SIGMOID if sigmoid else cuda_lib.SCORE_SOFTMAX
    k = min(8, G // groups * kept)
    for values in (1, 2):
        level = torch.randn(values, device="cuda", generator=gen)
        bias = level[torch.arange(G, device="cuda") * values // G].contiguous()
        for top in (1, 2) if groups > 1 else (1,):
            _, ids, _, _ = cuda_lib.mx_moe_topk(x, k, score, bias, groups, kept, top)
            want = _choose(x.to(D), k, sigmoid, bias, groups, kept, top)
            wrong = (ids.long() != want).any(1)
            assert not wrong.any(), "%d rows, values %d, top %d" % (int(wrong.sum()), values, top)
