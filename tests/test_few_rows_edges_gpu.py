"""The product of a few rows at the ends of its range."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [2 ** 31 - 8, 2 ** 31 - 776])
def test_longest_contraction(cuda_lib, K):
    """K up to the largest the entry point takes: the last chunks' column
    indexes pass 2^31.  Few nonzero weights, small integers: exact."""
    mx = cuda_lib
    x = torch.ones((1, K), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((8, K), dtype=torch.bfloat16, device="cuda")
    for n in range(8):
        w[n, K - 1 - n] = n + 1
        w[n, K - 700 + 64 * n] = 16
        w[n, 1 << (20 + n)] = 32
        w[n, n] = 64
    x[0, K - 8:] = 2
    out = mx.mx_linear_fwd(x, w)
    assert mx.mx_get_device_status() == "MX_OK"
    want = [2 * (n + 1) + 16 + 32 + 64 for n in range(8)]
    assert out[0].tolist() == want
