"""The checkpoint's backward pass where a gradient or a pre-activation is not
an ordinary number."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R", [40, 600])
def test_relu_selects_the_gradient(cuda_lib, R):
    """A closed gate (z <= 0) passes nothing on, whatever the gradient
    behind it: dz is exactly dh or 0, and the column sums stay those of the open
    gates (fp32 sums of R terms, in any order: R 2^-23 of the magnitudes)."""
    mx = cuda_lib
    gen = torch.Generator().manual_seed(R)
    C = 320
    z = torch.randn((R, C), generator=gen)
    z[:, ::5] = 0.0
    z = z.to(torch.bfloat16).cuda()
    _, ck = mx.mx_act_ckpt_fwd(z, mx.ACT_RELU)
    dh = torch.randn((R, C), generator=gen).to(torch.bfloat16).cuda()
    shut, bad = z <= 0, torch.rand((R, C), generator=gen).cuda()
    for i, v in enumerate((float("inf"), float("-inf"), float("nan"))):
        dh[shut & (bad > 0.1 * i) & (bad < 0.1 * i + 0.1)] = v
    first = int((z[:, 1] > 0).nonzero()[0])
    dh[first, 1] = float("inf")
    want = torch.where(z > 0, dh, torch.zeros_like(dh))
    dz, h, db = mx.mx_act_ckpt_bwd(ck, mx.ACT_RELU, dh, recompute=True, colsum=True)
    assert torch.equal(dz, want)
    assert bool(h.isfinite().all())
    assert float(db[1]) == float("inf")
    d = torch.cat([want[:, :1], want[:, 2:]], 1).double()
    got = torch.cat([db[:1], db[2:]]).double()
    assert bool(((got - d.sum(0)).abs() <= R * 2.0 ** -23 * d.abs().sum(0)).all())
