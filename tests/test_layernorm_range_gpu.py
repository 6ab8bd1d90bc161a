"""Rows that fp32 cannot normalise: an infinity, a NaN, or squares whose sum passes
fp32's range.  The whole row, its rstd and its gradients are NaN in both forms of
the norm, wherever in the row it stands; the other rows are as without it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [8, 64, 2048, 5120, 8192, 16384])
def test_rows_out_of_range(cuda_lib, D, dtype, rms):
    gen = torch.Generator(device="cuda").manual_seed(D)
    x = torch.randn((11, D), device="cuda", generator=gen).to(dtype)
    dy = torch.randn((11, D), device="cuda", generator=gen).to(BF)
    w, b = ((1 + torch.rand(D, device="cuda", generator=gen)).to(BF) for _ in range(2))
    clean = cuda_lib.mx_layernorm_fwd(x, w, b, rms=rms)
    y = x.clone()
    bad = [0, 2, 4, 5, 6, 8]
    y[0, 0], y[2, D // 2], y[4, D - 1], y[5, D // 2 - 1] = float("inf"), float("inf"), -float("inf"), float("nan")
    y[6, D // 3], y[8, ::2] = 1e30, -3e38
    got = cuda_lib.mx_layernorm_fwd(y, w, b, rms=rms)
    good = [i for i in range(11) if i not in bad]
    assert torch.isnan(got[0][bad]).all() and torch.isnan(got[2][bad]).all()
    assert torch.equal(got[0][good], clean[0][good]) and torch.equal(got[2][good], clean[2][good])
    dx, dw, _ = cuda_lib.mx_layernorm_bwd(dy, y, got[1], got[2], w, rms=rms)
    ref, _, _ = cuda_lib.mx_layernorm_bwd(dy, x, clean[1], clean[2], w, rms=rms)
    assert torch.isnan(dx[bad]).all() and torch.equal(dx[good], ref[good]) and torch.isnan(dw).all()


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("D", [64, 2048, 16384])
def test_large_rows_within_range(cuda_lib, D, rms):
    """Squares that sum up to 2^126 still normalise: y is that of the row scaled by a power of two."""
    gen = torch.Generator(device="cuda").manual_seed(D)
    x = torch.randn((5, D), device="cuda", generator=gen).clamp(-4, 4)
    up = 2.0 ** (61 - (D.bit_length() + 1) // 2)        # |x| <= 4: D 16 up^2 <= 2^126
    small = cuda_lib.mx_layernorm_fwd(x, eps=0.0, rms=rms)
    large = cuda_lib.mx_layernorm_fwd(x * up, eps=0.0, rms=rms)
    assert torch.equal(small[0], large[0]) and torch.equal(small[2], large[2] * up)
