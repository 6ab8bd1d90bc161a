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


def _slope(z, act):
    """act and act' in fp64, for any finite fp32 z."""
    if act == "RELU":
        return z.clamp(min=0), (z > 0).double()
    k, b = (1.0, 0.0) if act in ("SILU", "SWIGLU") else (2 * (2 / torch.pi) ** 0.5, 0.044715)
    s = torch.sigmoid(k * (z + b * z ** 3))
    return z * s, s + z * s * (1 - s) * k * (1 + 3 * b * z * z)


@pytest.mark.parametrize("act", ["SWIGLU", "GELU_TANH", "SILU", "RELU"])
@pytest.mark.parametrize("recompute,colsum", [(False, False), (True, True)])
def test_slopes_over_the_whole_range(cuda_lib, act, recompute, colsum):
    """Pre-activations of every magnitude that BF16 and the checkpoint hold,
    of both signs: the slope is 1 or 0 far out, never NaN.  Powers of two are
    exact in the checkpoint.  Bounds: one rounding to BF16 (2^-9, doubled) and
    2^-18 of the factors for the fp32 arithmetic, |z| counted up to 16, where
    the gate has closed or opened to within fp32."""
    mx = cuda_lib
    a = getattr(mx, "ACT_" + act)
    exps = torch.arange(-100, 128)
    z = torch.ldexp(torch.ones(()), exps.float())[:, None].repeat(1, 64)
    z = torch.cat([z, -z]).double()
    if act == "SWIGLU":
        z = torch.cat([z, torch.ones_like(z)], 1)
    gen = torch.Generator().manual_seed(1)
    dh = torch.ldexp(torch.randint(0, 2, (z.shape[0], 64), generator=gen) * 2.0 - 1.0,
                     torch.randint(-3, 0, (z.shape[0], 64), generator=gen).float()).to(torch.bfloat16).cuda()
    zb = z.to(torch.bfloat16).cuda()
    z = z.cuda()
    assert torch.equal(zb.double(), z)
    _, ck = mx.mx_act_ckpt_fwd(zb, a)
    dz, h, db = mx.mx_act_ckpt_bwd(ck, a, dh, recompute=recompute, colsum=colsum)
    g = z[:, :64]
    rh, slope = _slope(g, act)
    d = dh.double()
    ref = d * slope
    err = (dz[:, :64].double() - ref).abs()
    assert bool((err <= 2.0 ** -8 * ref.abs() + 2.0 ** -18 * d.abs() * (1 + g.abs().clamp(max=16))).all())
    # e^-32 |z| is below half a unit of 1 in BF16, and e^-128 |z| below BF16's smallest value
    assert torch.equal(dz[:, :64][g >= 32].double(), d[g >= 32]) and not bool(dz[:, :64][g <= -128].any())
    if act == "SWIGLU":
        ref_u = d * rh
        err = (dz[:, 64:].double() - ref_u).abs()
        assert bool((err <= 2.0 ** -8 * ref_u.abs() + 2.0 ** -18 * d.abs() * g.abs().clamp(max=16) + 2.0 ** -126).all())
    if recompute:
        err = (h.double() - rh).abs()
        assert bool((err <= 2.0 ** -8 * rh.abs() + 2.0 ** -18 * g.abs().clamp(max=16) + 2.0 ** -126).all())
    if colsum:
        n = z.shape[0]
        bound = n * 2.0 ** -23 * ref.abs().sum(0) + 2.0 ** -18 * (d.abs() * (1 + g.abs().clamp(max=16))).sum(0)
        assert bool(((db[:64].double() - ref.sum(0)).abs() <= bound).all())
