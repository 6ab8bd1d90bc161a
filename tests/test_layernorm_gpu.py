"""The layer norm and its backward pass against the formulas in 64 bits and
against differences: both types, rows of one warp to sixteen, odd row counts,
strides, residuals, large offsets, infinities, streams, graphs.

Tolerances.  y and BF16 results are fp32 expressions rounded once (2^-8 / 2 of
the value, eps / 2 = 2^-9 in BF16's significand, doubled).  The fp32 arithmetic: a row's
sums of D terms are off by at most (8 + log2 D) roundings of 2^-24 of the summed
magnitudes (a lane's values in turn, then a tree), mean and rstd likewise; sums
over R rows add R / blocks sequential roundings, bounded here by R * 2^-24 of
the summed magnitudes."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
U = 2.0 ** -24


def _inputs(R, D, dtype, seed=0, offset=0.5, res=False, wtype=BF, pad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + R * 7 + D)

    def rand(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    def rows(v):  # with a row stride of D + pad
        t = torch.full((R, D + pad), float("nan"), dtype=v.dtype, device="cuda")
        t[:, :D] = v
        return t[:, :D]

    x = rows((rand(R, D) * (0.2 + rand(D).abs()) + offset).to(dtype))
    return dict(x=x, w=(1 + 0.2 * rand(D)).to(wtype), b=(0.2 * rand(D)).to(wtype), dy=rows(rand(R, D).to(BF)),
                res=rows(rand(R, D).to(dtype)) if res else None)


def _close(got, ref, bound, what):
    got = got.double()
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of the bound" % (
        what, int(bad.sum()), bad.numel(), float(((got - ref).abs() / bound).max()))


def _ref(s, w, b, eps, rms):
    d = s.double()
    mean = torch.zeros_like(d[:, :1]) if rms else d.mean(1, keepdim=True)
    rstd = ((d - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    y = (d - mean) * rstd
    y = y if w is None else y * w.double()
    return mean, rstd, y if b is None else y + b.double()


def _check_fwd(t, got, eps, rms, w, b):
    y, mean, rstd, s = got
    R, D = s.shape
    m, r, want = _ref(s, w, b, eps, rms)
    k = 16 + torch.tensor(float(D)).log2().item()
    size = s.double().abs().mean(1, keepdim=True) + s.double().square().mean(1, keepdim=True).sqrt()
    if not rms:
        _close(mean[:, None], m, k * U * size, "mean")
    # the centred squares are relative to themselves; the mean's error enters them squared
    _close(rstd[:, None], r, 2 * k * U * r + 2.0 ** -120, "rstd")
    fp32 = 4 * k * U * ((s.double().abs() + m.abs() + size) * r * (1 if w is None else w.double().abs())
                        + (0 if b is None else b.double().abs()))
    _close(y, want, 2.0 ** -8 * want.abs() + fp32 + 2.0 ** -126, "y")


SHAPES = [(1, 8), (3, 64), (5, 200), (37, 256), (129, 264), (64, 1000), (7, 2048), (33, 2056), (9, 4096), (2, 5120),
          (5, 7168), (3, 8192), (2, 8200), (3, 12288 + 8), (2, 16384), (700, 512)]


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,D", SHAPES)
def test_forward(cuda_lib, R, D, dtype):
    t = _inputs(R, D, dtype)
    _check_fwd(t, cuda_lib.mx_layernorm_fwd(t["x"], t["w"], t["b"]), 1e-5, False, t["w"], t["b"])
    _check_fwd(t, cuda_lib.mx_layernorm_fwd(t["x"], t["w"], rms=True, eps=1e-6), 1e-6, True, t["w"], None)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [1280, 1288, 2560, 3584, 4088, 4104, 5112, 6136, 6144, 6152, 8184, 8208, 10240, 12288, 16376])
def test_row_lengths(cuda_lib, D, dtype):
    """Every number of warps and pieces a row takes, with and without lanes past its
    end, and the sizes where shared memory passes what a launch has unasked."""
    for R, res in ((2, True), (161, False)):
        t = _inputs(R, D, dtype, seed=7, res=res)
        s = cuda_lib.mx_layernorm_fwd(t["x"], t["w"], t["b"], residual=t["res"])
        _check_fwd(t, s, 1e-5, False, t["w"], t["b"])
        got = cuda_lib.mx_layernorm_bwd(t["dy"], t["x"], s[1], s[2], t["w"], dres=t["res"])
        if not res:
            _check_bwd(t, got, s[1], s[2], False, t["w"], dtype)
        else:  # the forward's sum is what the backward pass takes
            u = dict(t, x=s[3])
            _check_bwd(u, cuda_lib.mx_layernorm_bwd(t["dy"], s[3], s[1], s[2], t["w"], dres=t["res"]), s[1], s[2], False,
                       t["w"], dtype)


@pytest.mark.parametrize("wtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,D", [(3, 64), (5, 1000), (131, 2048), (2, 8200), (2, 16384)])
def test_forward_with_residual_and_strides(cuda_lib, R, D, dtype, wtype):
    t = _inputs(R, D, dtype, res=True, wtype=wtype, pad=24)
    got = cuda_lib.mx_layernorm_fwd(t["x"], t["w"], t["b"], residual=t["res"])
    want = (t["x"].float() + t["res"].float()).to(dtype)
    assert torch.equal(got[3], want)
    _check_fwd(t, got, 1e-5, False, t["w"], t["b"])
    # in place: the sum takes x's memory, then the residual's
    for name in ("x", "res"):
        u = _inputs(R, D, dtype, res=True, wtype=wtype, pad=24)
        again = cuda_lib.mx_layernorm_fwd(u["x"], u["w"], u["b"], residual=u["res"], sum_out=u[name])
        assert again[3] is u[name]
        assert all(torch.equal(p, q) for p, q in zip(again, got))


def test_forward_without_weights_and_statistics(cuda_lib):
    t = _inputs(6, 320, BF)
    _check_fwd(t, cuda_lib.mx_layernorm_fwd(t["x"]), 1e-5, False, None, None)
    y, mean, rstd, s = cuda_lib.mx_layernorm_fwd(t["x"], bias=t["b"], stats=False)
    assert mean is None and rstd is None and s is t["x"]
    assert torch.equal(y, cuda_lib.mx_layernorm_fwd(t["x"], bias=t["b"])[0])


@pytest.mark.parametrize("D", [64, 1000, 4096, 16384])
def test_large_offset_keeps_the_variance(cuda_lib, D):
    """Values around 2^12 with steps of 2^-8: squares minus the mean's square
    would lose the variance."""
    t = _inputs(5, D, F)
    x = 4096.0 + t["x"]
    got = cuda_lib.mx_layernorm_fwd(x, eps=0.0)
    m, r, _ = _ref(x, None, None, 0.0, False)
    # the mean is off by at most k 2^-24 * 4096, whose square joins the variance
    k = 16 + 14
    err = (k * U * 4096) ** 2 * r.square() + 2 * k * U
    _close(got[2][:, None], r, err * r, "rstd")


def test_constant_rows_and_zero_rows(cuda_lib):
    x = torch.tensor([[3.0], [0.0], [-2.5]], device="cuda").expand(3, 1024).contiguous()
    y, mean, rstd, _ = cuda_lib.mx_layernorm_fwd(x)
    assert (y == 0).all() and mean.tolist() == [3.0, 0.0, -2.5]
    _close(rstd, torch.full((3,), 1e-5, dtype=torch.float64, device="cuda").rsqrt(), 0.01, "rstd")
    y, _, rstd, _ = cuda_lib.mx_layernorm_fwd(torch.zeros((2, 72), dtype=BF, device="cuda"), rms=True, eps=0.0)
    assert torch.isinf(rstd).all() and torch.isnan(y).all()  # 0 * (1 / 0)


@pytest.mark.parametrize("D", [64, 2048, 8192])
def test_non_finite_rows_stay_alone(cuda_lib, D):
    t = _inputs(9, D, BF)
    clean = cuda_lib.mx_layernorm_fwd(t["x"], t["w"], t["b"])
    x = t["x"].clone()
    x[2, D // 2], x[5, 3], x[7, D - 1] = float("nan"), float("inf"), float("-inf")
    y, mean, rstd, _ = cuda_lib.mx_layernorm_fwd(x, t["w"], t["b"])
    bad = [2, 5, 7]
    assert torch.isnan(y[bad]).all()
    good = [i for i in range(9) if i not in bad]
    assert torch.equal(y[good], clean[0][good]) and torch.equal(rstd[good], clean[2][good])


# ---------------------------------------------------------------- backward

def _bwd_ref(t, mean, rstd, rms, w):
    x, dy = t["x"].double(), t["dy"].double()
    D = x.shape[1]
    r = rstd.double()[:, None]
    xh = (x if rms else x - mean.double()[:, None]) * r
    g = dy if w is None else dy * w.double()
    c1 = 0 if rms else g.mean(1, keepdim=True)
    c2 = (g * xh).mean(1, keepdim=True)
    dx = r * (g - c1 - xh * c2)
    mag = r * (g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True)
               + xh.abs() * c2.abs())
    if t["res"] is not None:
        dx, mag = dx + t["res"].double(), mag + t["res"].double().abs()
    return dx, mag, (dy * xh).sum(0), (dy * xh).abs().sum(0), dy.sum(0), dy.abs().sum(0)


def _check_bwd(t, got, mean, rstd, rms, w, dtype):
    dx, dw, db = got
    R, D = t["x"].shape
    want, mag, w_ref, w_mag, b_ref, b_mag = _bwd_ref(t, mean, rstd, rms, w)
    k = 24 + torch.tensor(float(D)).log2().item()
    _close(dx, want, (2.0 ** -8 if dtype == BF else U) * want.abs() + 2 * k * U * mag + 2.0 ** -126, "dx")
    if dw is not None:
        _close(dw, w_ref, (R + 8) * U * w_mag + 2.0 ** -126, "dweight")
    if db is not None:
        _close(db, b_ref, (R + 8) * U * b_mag + 2.0 ** -126, "dbias")


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,D", SHAPES + [(2500, 384), (160, 8192), (155, 4096)])
def test_backward(cuda_lib, R, D, dtype, rms):
    for res in (False, True):
        t = _inputs(R, D, dtype, seed=1, res=res, pad=8 if res else 0)
        _, mean, rstd, _ = cuda_lib.mx_layernorm_fwd(t["x"], t["w"], rms=rms)
        got = cuda_lib.mx_layernorm_bwd(t["dy"], t["x"], mean, rstd, t["w"], dres=t["res"], rms=rms)
        _check_bwd(t, got, mean, rstd, rms, t["w"], dtype)
        again = cuda_lib.mx_layernorm_bwd(t["dy"], t["x"], mean, rstd, t["w"], dres=t["res"], rms=rms)
        assert all(torch.equal(p, q) for p, q in zip(got, again))
        only = cuda_lib.mx_layernorm_bwd(t["dy"], t["x"], mean, rstd, t["w"], dres=t["res"], rms=rms, wgrad=False,
                                         bias=False)
        assert torch.equal(only[0], got[0]) and only[1] is None and only[2] is None


@pytest.mark.parametrize("D", [512, 8192, 16384])
def test_backward_parts(cuda_lib, D):
    """fp32 weights, no weights, one gradient without the other, dx in dres's memory."""
    t = _inputs(40, D, F, seed=2, res=True, wtype=F)
    _, mean, rstd, _ = cuda_lib.mx_layernorm_fwd(t["x"])
    full = cuda_lib.mx_layernorm_bwd(t["dy"], t["x"], mean, rstd, t["w"], dres=t["res"])
    _check_bwd(t, full, mean, rstd, False, t["w"], F)
    one = cuda_lib.mx_layernorm_bwd(t["dy"], t["x"], mean, rstd, t["w"], dres=t["res"], bias=False)
    assert one[2] is None and torch.equal(one[1], full[1]) and torch.equal(one[0], full[0])
    one = cuda_lib.mx_layernorm_bwd(t["dy"], t["x"], mean, rstd, t["w"], dres=t["res"], wgrad=False)
    assert one[1] is None and torch.equal(one[2], full[2])
    _check_bwd(t, cuda_lib.mx_layernorm_bwd(t["dy"], t["x"], mean, rstd, dres=t["res"]), mean, rstd, False, None, F)
    dres = t["res"].clone()
    inplace = cuda_lib.mx_layernorm_bwd(t["dy"], t["x"], mean, rstd, t["w"], dres=dres, dx=dres)
    assert inplace[0] is dres and torch.equal(dres, full[0])


@pytest.mark.parametrize("R", [0, 1, 50])
def test_backward_accumulates(cuda_lib, R):
    t = _inputs(R, 640, BF, seed=3)
    mean, rstd = torch.zeros(R, device="cuda"), torch.ones(R, device="cuda")
    _, dw, db = cuda_lib.mx_layernorm_bwd(t["dy"], t["x"], mean, rstd, t["w"])
    if R == 0:
        assert (dw == 0).all() and (db == 0).all()
    old_w, old_b = torch.randn(640, device="cuda"), torch.randn(640, device="cuda")
    gw, gb = old_w.clone(), old_b.clone()
    cuda_lib.mx_layernorm_bwd(t["dy"], t["x"], mean, rstd, t["w"], dweight=gw, dbias=gb, accumulate=True)
    assert torch.equal(gw, old_w + dw) and torch.equal(gb, old_b + db)


def test_no_rows(cuda_lib):
    x = torch.empty((0, 64), dtype=BF, device="cuda")
    y, mean, rstd, _ = cuda_lib.mx_layernorm_fwd(x)
    assert y.shape == (0, 64) and mean.shape == (0,)
    assert cuda_lib.mx_layernorm_bwd(y, x, mean, rstd, wgrad=False, bias=False)[0].shape == (0, 64)


def test_gradient_against_differences(cuda_lib):
    """sum(c y) moves by dx along a direction: fp32 input, central differences.
    y is rounded to BF16 (2^-9 of its values), so the sum over 3 x 256 of them in a
    step of 2^-4 is off by at most 2^-9 sum |c y| * 2^4 / 1, in practice its root."""
    t = _inputs(3, 256, F, seed=4)
    c = torch.randn((3, 256), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).to(BF)
    v = torch.randn((3, 256), device="cuda", generator=torch.Generator(device="cuda").manual_seed(6))
    _, mean, rstd, _ = cuda_lib.mx_layernorm_fwd(t["x"], t["w"])
    dx, _, _ = cuda_lib.mx_layernorm_bwd(c, t["x"], mean, rstd, t["w"])
    h = 2.0 ** -4

    def f(x):
        return (cuda_lib.mx_layernorm_fwd(x, t["w"])[0].double() * c.double()).sum()

    def f64(x):
        return (_ref(x, t["w"], None, 1e-5, False)[2] * c.double()).sum()

    moved = float((f(t["x"] + h * v) - f(t["x"] - h * v)) / (2 * h))
    moved64 = float((f64(t["x"] + h * v) - f64(t["x"] - h * v)) / (2 * h))
    curve = abs(moved64 - float((f64(t["x"] + h / 8 * v) - f64(t["x"] - h / 8 * v)) / (h / 4)))
    noise = 2.0 ** -9 * float((_ref(t["x"], t["w"], None, 1e-5, False)[2] * c.double()).abs().sum()) / h
    assert abs(float((dx.double() * v.double()).sum()) - moved) <= noise + 2 * curve


def test_rows_behind_and_beside_are_left_alone(cuda_lib):
    buf = torch.full((12, 136), 7.0, dtype=BF, device="cuda")
    t = _inputs(10, 128, BF)
    cuda_lib.mx_layernorm_fwd(t["x"], out=buf[:10, :128])
    assert (buf[10:] == 7).all() and (buf[:, 128:] == 7).all() and not (buf[:10, :128] == 7).all()
    dx = torch.full((12, 136), 7.0, dtype=BF, device="cuda")
    mean, rstd = torch.zeros(10, device="cuda"), torch.ones(10, device="cuda")
    cuda_lib.mx_layernorm_bwd(t["dy"], t["x"], mean, rstd, dx=dx[:10, :128])
    assert (dx[10:] == 7).all() and (dx[:, 128:] == 7).all()


def test_streams_and_graphs(cuda_lib):
    """Two streams at once, and a captured forward and backward replayed on new inputs."""
    t = [_inputs(300, 2048, BF, seed=i, res=True) for i in range(2)]

    def both(u, stream=None):
        y, mean, rstd, s = cuda_lib.mx_layernorm_fwd(u["x"], u["w"], u["b"], residual=u["res"], stream=stream)
        return (y, mean, rstd, s) + cuda_lib.mx_layernorm_bwd(u["dy"], s, mean, rstd, u["w"], dres=u["res"],
                                                              stream=stream)

    want = [both(u) for u in t]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in t]
    for _ in range(20):
        got = [both(u, s) for u, s in zip(t, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(g, w))
    u = {k: v.clone() for k, v in t[0].items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(u)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(u)
    for i in (1, 0, 1):
        for k in u:
            u[k].copy_(t[i][k])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want[i]))
