"""8-bit activation checkpoints: bytes against the oracle's quantizer, the
backward pass against a plain fp64 implementation of the formulas and against
differences, special values, odd row counts, strides.

Tolerances: results are fp32 expressions rounded once to BF16 (half a unit:
2^-9 relative, doubled), plus 2^-18 of the factors' magnitude for the fp32
arithmetic of the activation; the fp32 column sums add R * 2^-23 of the
summed magnitudes.
"""
import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu

ACTS = ["SWIGLU", "GELU_TANH", "SILU", "RELU"]


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _z(R, C, seed):
    """Rows of mixed magnitude, with zeros and a zero block."""
    gen = torch.Generator().manual_seed(seed)
    z = torch.randn((R, C), generator=gen) * torch.exp2(torch.randint(-6, 4, (R, 1), generator=gen).float())
    z[:, ::37] = 0
    z[R // 2, :32] = 0
    return z.to(torch.bfloat16).cuda()


def _f(z, act):
    if act == "RELU":
        return z.clamp(min=0), (z > 0).double()
    k, b = (1.0, 0.0) if act == "SILU" else (2 * np.sqrt(2 / np.pi), 0.044715)
    s = torch.sigmoid(k * (z + b * z ** 3))
    return z * s, s + z * s * (1 - s) * k * (1 + 3 * b * z * z)


def _bwd_ref(z, dh, act):
    """(dz, h, magnitude of dz's terms)"""
    if act == "SWIGLU":
        g, u = z.chunk(2, 1)
        h, d = _f(g, "SILU")
        dz = torch.cat([dh * u * d, dh * h], 1)
        mag = torch.cat([(dh * u).abs() * (1 + g.abs()), dh.abs() * g.abs()], 1)
        return dz, h * u, mag
    h, d = _f(z, act)
    return dh * d, h, dh.abs() * (1 + z.abs())


def _close(got, ref, mag, rel=2.0 ** -8, fp32=2.0 ** -18):
    got = got.double()
    bound = rel * ref.abs() + fp32 * mag + 2.0 ** -126
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), "%d of %d off, worst %.3g x the bound" % (
        int(bad.sum()), bad.numel(), float(((got - ref).abs() / bound).max()))


def _values(mx, ck):
    return torch.from_numpy(O.dequantize_rows(ck.data.cpu().numpy(), ck.scale.cpu().numpy(), ck.rows, ck.cols,
                                              O.E4M3)).cuda()


SHAPES = [(1, 64), (3, 128), (31, 192), (129, 64), (256, 512), (300, 1536), (512, 1088), (513, 1088), (1000, 2240)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("R,C", SHAPES)
def test_save(cuda_lib, act, R, C):
    mx = cuda_lib
    z = _z(R, C, R + C)
    ck = mx.MX(R, C)
    ck.scale.fill_(0xCD)
    h, _ = mx.mx_act_ckpt_fwd(z, getattr(mx, "ACT_" + act), ckpt=ck)
    payload, scales = O.quantize_rows(O.bf16_to_f64(_bits(z)), O.E4M3)
    assert np.array_equal(ck.data.cpu().numpy(), payload)
    assert np.array_equal(ck.scale.cpu().numpy(), scales)
    d = z.double()
    if act == "SWIGLU":
        g, u = d.chunk(2, 1)
        ref, mag = _f(g, "SILU")[0] * u, (g * u).abs()
    else:
        ref, mag = _f(d, act)[0], d.abs()
    _close(h, ref, mag)


@pytest.mark.parametrize("act", ACTS)
def test_save_special_values(cuda_lib, act):
    """NaN, infinities, subnormals and the largest values: payload and scales
    as the oracle's quantizer; h is the formula's where that is finite."""
    mx = cuda_lib
    z = _z(64, 256, 5)
    z[3, 7], z[4, 40], z[5, 200] = float("nan"), float("inf"), float("-inf")
    z[6, :32] = 1e-40
    z[7, :64] = 3e38
    z[8, 64:96] = -3e38
    h, ck = mx.mx_act_ckpt_fwd(z, getattr(mx, "ACT_" + act))
    payload, scales = O.quantize_rows(O.bf16_to_f64(_bits(z)), O.E4M3)
    assert np.array_equal(ck.data.cpu().numpy(), payload)
    assert np.array_equal(ck.scale.cpu().numpy(), scales)
    clean = torch.ones(64, dtype=torch.bool)
    clean[3:9] = False
    d = z.double()[clean.cuda()]
    ref = _f(d.chunk(2, 1)[0], "SILU")[0] * d.chunk(2, 1)[1] if act == "SWIGLU" else _f(d, act)[0]
    _close(h[clean.cuda()], ref, d.abs().chunk(2, 1)[0] * d.abs().chunk(2, 1)[1] if act == "SWIGLU" else d.abs())
    assert bool(h[3].isnan().any())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("recompute,colsum", [(False, False), (True, True)])
def test_backward(cuda_lib, act, R, C, recompute, colsum):
    mx = cuda_lib
    a = getattr(mx, "ACT_" + act)
    z = _z(R, C, 2 * R + C)
    _, ck = mx.mx_act_ckpt_fwd(z, a)
    gen = torch.Generator().manual_seed(R)
    dh = torch.randn((R, C // 2 if act == "SWIGLU" else C), generator=gen).to(torch.bfloat16).cuda()
    dz, h, db = mx.mx_act_ckpt_bwd(ck, a, dh, recompute=recompute, colsum=colsum)
    assert mx.mx_get_device_status() == "MX_OK"
    zq = _values(mx, ck)
    rdz, rh, mag = _bwd_ref(zq, dh.double(), act)
    _close(dz, rdz, mag)
    assert (h is not None) == recompute and (db is not None) == colsum
    if recompute:
        hm = zq.abs() if act != "SWIGLU" else zq.abs().chunk(2, 1)[0] * zq.abs().chunk(2, 1)[1]
        _close(h, rh, hm)
    if colsum:
        _close(db, rdz.sum(0), mag.sum(0), rel=0, fp32=R * 2.0 ** -23 + 2.0 ** -18)
        again = mx.mx_act_ckpt_bwd(ck, a, dh, colsum=True)[2]
        assert torch.equal(db, again)


@pytest.mark.parametrize("act", ACTS)
def test_strides(cuda_lib, act):
    mx = cuda_lib
    a = getattr(mx, "ACT_" + act)
    R, C = 70, 320
    H = C // 2 if act == "SWIGLU" else C
    z = _z(R, C + 24, 9)[:, 8:8 + C]
    hb = torch.full((R, H + 16), 5.0, dtype=torch.bfloat16, device="cuda")
    _, ck = mx.mx_act_ckpt_fwd(z, a, h=hb[:, 8:8 + H])
    h0, ck0 = mx.mx_act_ckpt_fwd(z.contiguous(), a)
    assert torch.equal(ck.data, ck0.data) and torch.equal(ck.scale, ck0.scale) and torch.equal(hb[:, 8:8 + H], h0)
    assert bool((hb[:, :8] == 5).all()) and bool((hb[:, 8 + H:] == 5).all())
    dhb = _z(R, H + 8, 3)
    dzb = torch.full((R, C + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    mx.mx_act_ckpt_bwd(ck, a, dhb[:, :H], dz=dzb[:, :C], h=hb[:, 8:8 + H])
    dz0, h1, _ = mx.mx_act_ckpt_bwd(ck, a, dhb[:, :H].contiguous(), recompute=True)
    assert torch.equal(dzb[:, :C], dz0) and torch.equal(hb[:, 8:8 + H], h1) and bool((dzb[:, C:] == 5).all())


def test_no_rows(cuda_lib):
    mx = cuda_lib
    e = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    h, ck = mx.mx_act_ckpt_fwd(e, mx.ACT_GELU_TANH)
    dz, _, db = mx.mx_act_ckpt_bwd(ck, mx.ACT_GELU_TANH, e, colsum=True)
    assert h.shape == dz.shape == (0, 128) and not bool(db.any())


@pytest.mark.parametrize("act", ACTS)
def test_backward_is_the_derivative(cuda_lib, act):
    """dz against central differences of the fp64 activation at the
    checkpoint's values: error of the difference h^2 / 6 of the third
    derivative (below 5), plus dz's own rounding."""
    mx = cuda_lib
    a = getattr(mx, "ACT_" + act)
    z = _z(40, 128, 77).clamp(-6, 6)
    _, ck = mx.mx_act_ckpt_fwd(z, a)
    zq = _values(mx, ck)
    dh = torch.ones((40, 64 if act == "SWIGLU" else 128), dtype=torch.bfloat16, device="cuda")
    dz = mx.mx_act_ckpt_bwd(ck, a, dh)[0].double()
    step = 1e-4

    def f(v):
        if act == "SWIGLU":
            g, u = v.chunk(2, 1)
            return _f(g, "SILU")[0] * u
        return _f(v, act)[0]

    far = zq.abs() > 2 * step                      # away from ReLU's corner
    parts = [slice(0, 64), slice(64, 128)] if act == "SWIGLU" else [slice(0, 128)]
    for p in parts:
        e = torch.zeros_like(zq)
        e[:, p] = step
        diff = (f(zq + e) - f(zq - e)) / (2 * step)
        want = dz[:, p]
        bound = 2.0 ** -8 * diff.abs() + 1e-6 * (1 + zq.abs().max() ** 2)
        ok = ((want - diff).abs() <= bound) | ~far[:, p]
        assert bool(ok.all())


def test_a_layer_from_its_checkpoint(cuda_lib):
    """mx_linear_fwd's checkpoint feeds mx_act_ckpt_bwd and the products: the
    gradients of a dense layer against fp64 at the checkpoint's values."""
    mx = cuda_lib
    gen = torch.Generator().manual_seed(0)
    M, N, K = 150, 192, 136
    x = torch.randn((M, K), generator=gen).to(torch.bfloat16).cuda()
    w = (torch.randn((N, K), generator=gen) * K ** -0.5).to(torch.bfloat16).cuda()
    b = torch.randn(N, generator=gen).to(torch.bfloat16).cuda()
    dout = torch.randn((M, N), generator=gen).to(torch.bfloat16).cuda()
    ck = mx.MX(M, N)
    mx.mx_linear_fwd(x, w, b, mx.ACT_GELU_TANH, ckpt=ck)
    z = x.double() @ w.double().T + b.double()
    zq = _values(mx, ck)
    # E4M3: half a unit of 2^-4 relative to the element, 2^-10 of the block's scale for subnormals (448 >= amax / 2 scales)
    assert bool(((zq - z).abs() <= 2.0 ** -4 * z.abs() + 2.0 ** -16 * z.abs().max()).all())
    dz, _, db = mx.mx_act_ckpt_bwd(ck, mx.ACT_GELU_TANH, dout, colsum=True)
    dx = mx.mx_ragged_gemm(dz, w[None], None, layout=mx.W_KN)
    dw = mx.mx_ragged_gemm_wgrad(dz, x, 1, None)[0]
    rdz, _, mag = _bwd_ref(zq, dout.double(), "GELU_TANH")
    _close(dz, rdz, mag)
    _close(db, rdz.sum(0), mag.sum(0), rel=0, fp32=2.0 ** -15)
    d = dz.double()
    _close(dx, d @ w.double(), d.abs() @ w.double().abs(), fp32=N * 2.0 ** -23)
    _close(dw, d.T @ x.double(), d.abs().T @ x.double().abs(), fp32=M * 2.0 ** -23)
