"""4-bit tensors with E4M3 scales per 16: the quantization value for value against
its definition in 64 bits (ties, subnormals, infinities, gathered rows), the
product against 64-bit sums of the operands' values.

Tolerance of the product: one rounding to BF16 (2^-8 / 2 of the value, doubled) and the
fp32 accumulation: a step of 64 products joins the running sum with its terms
cut at a few units of 2^-24 of the largest, so K / 64 + 8 steps are off by less than
(K / 64 + 8) * 2^-21 of the summed magnitudes."""
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu

BF, D = torch.bfloat16, torch.float64
GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=D)


def _blocked(rows, cols):
    """Offsets of the scales [rows, cols / 16] in the blocked layout."""
    return torch.from_numpy(O.blocked_index(rows, cols // 16, range(rows))).reshape(rows, cols // 16)


def _parts(t):
    """(signed code values [R, K], scales [R, K / 16], row scales [R]) in 64 bits, on the CPU."""
    data = t.data.cpu().view(t.rows, t.cols // 2)
    codes = torch.stack((data & 15, data >> 4), -1).view(t.rows, t.cols).long()
    v = GRID[codes & 7] * torch.where(codes >= 8, -1.0, 1.0)
    s = t.scale.cpu()[_blocked(t.rows, t.cols)].view(torch.float8_e4m3fn).to(D)
    return v, s, (torch.ones(t.rows, dtype=D) if t.row_scale is None else t.row_scale.cpu().to(D))


def _values(t):
    v, s, r = _parts(t)
    return v * s.repeat_interleave(16, 1) * r[:, None]


def _want(x):
    """The definition for finite BF16 rows x (64 bits, CPU)."""
    R, K = x.shape
    amax = x.abs().view(R, -1, 16).amax(2)
    top = amax.amax(1)
    mant, exp = torch.frexp(top / (6 * 448))          # in [0.5, 1): 2^exp is above, 2^(exp - 1) only if mant is 0.5
    e = torch.where(top == 0, -100, torch.where(mant == 0.5, exp - 1, exp)).clamp(min=-100)
    row = torch.exp2(e.to(D))
    s = (amax / row[:, None] / 6).float().to(torch.float8_e4m3fn).to(D)  # exact in fp32 up to the division, whose
    step = (s * row[:, None]).repeat_interleave(16, 1)                   # ties are exact
    q = torch.where(step == 0, torch.zeros_like(x), x.abs() / torch.where(step == 0, 1.0, step))
    n = torch.where(q < 2, torch.round(2 * q) / 2, torch.where(q < 4, torch.round(q), 2 * torch.round(q / 2))).clamp(max=6)
    return torch.sign(x) * n, s, row


def _check_quantized(t, x):
    v, s, r = _parts(t)
    wv, ws, wr = _want(x)
    assert torch.equal(r, wr) and torch.equal(s, ws)
    bad = v != wv
    assert not bad.any(), "%d codes differ, first at %s: %s for %s" % (
        int(bad.sum()), bad.nonzero()[0].tolist(), float(v[bad][0]), float(x[bad][0]))


def _rand(shape, seed, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (std * torch.randn(shape, generator=gen) * torch.exp2(torch.randint(-8, 8, (shape[0], 1), generator=gen).float())
            ).to(BF)


@pytest.mark.parametrize("R,K", [(1, 32), (3, 64), (130, 96), (5, 512), (128, 1024), (300, 2048), (2, 2080), (4, 4096),
                                 (3, 8192), (2, 16416), (1, 32768)])
def test_quantize(cuda_lib, R, K):
    x = _rand((R, K), R + K)
    x[0, : K // 2] *= 2.0 ** -9          # blocks far below the row's largest: subnormal and zero scales
    x[R // 2, 16:32] = 0
    t = cuda_lib.mx_nvfp4_quantize(x.cuda())
    _check_quantized(t, x.to(D))
    used = torch.zeros(t.scale.numel(), dtype=torch.bool)
    used[_blocked(R, K).reshape(-1)] = True
    assert (t.scale.cpu()[~used] == 0).all()          # padding rows and columns


def test_quantize_every_bf16_value(cuda_lib):
    """All finite BF16 values beside every kind of block maximum: ties and the
    values next to them."""
    bits = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16)
    every = bits.view(BF)
    every = every[torch.isfinite(every)]
    every = every[(every.abs() <= 8) & (every.abs() >= 2.0 ** -12)]
    n = every.numel() // 15
    rows = []
    for top in (6.0, 5.25, 7.0, 3.75, 4.03125, 1.0, 2688.0 / 256, 0.013):
        b = every[: n * 15].view(n, 15)
        rows.append(torch.cat([torch.full((n, 1), top, dtype=BF), b.clamp(-top, top)], 1))
    x = torch.cat(rows).view(-1, 16)
    pad = -x.shape[0] % 4
    x = torch.cat([x, x[:pad]]).view(-1, 64)
    for scale in (1.0, 2.0 ** -40, 2.0 ** 40):
        y = (x.float() * scale).to(BF)
        _check_quantized(cuda_lib.mx_nvfp4_quantize(y.cuda()), y.to(D))


def test_quantize_the_ends_of_the_range(cuda_lib):
    x = torch.zeros((6, 64), dtype=BF)
    x[0, 3] = 3.38953139e38               # the largest BF16 value
    x[1, :] = 2.0 ** -133                 # subnormal
    x[2, 5] = -2.0 ** -126
    x[3, ::2] = 2.0 ** -100
    x[4, 7], x[4, 40] = 2688.0, -1.0      # 6 * 448: the row's power is 1
    x[5, 7] = 2704.0                      # just above
    t = cuda_lib.mx_nvfp4_quantize(x.cuda())
    _check_quantized(t, x.to(D))
    assert t.row_scale[4] == 1 and t.row_scale[5] == 2


def test_quantize_non_finite_rows(cuda_lib):
    x = _rand((8, 2112), 1)              # eight: as weights they are N = 8 columns
    want = cuda_lib.mx_nvfp4_quantize(x.cuda())
    bad = x.clone()
    bad[1, 700], bad[3, 0], bad[4, 2111] = float("nan"), float("inf"), float("-inf")
    t = cuda_lib.mx_nvfp4_quantize(bad.cuda())
    assert torch.isnan(t.row_scale[[1, 3, 4]]).all() and (t.data[[1, 3, 4]] == 0).all()
    good = [0, 2, 5, 6, 7]
    assert torch.equal(t.row_scale[good], want.row_scale[good]) and torch.equal(t.data[good], want.data[good])
    w = cuda_lib.mx_nvfp4_quantize(_rand((64, 2112), 2).cuda())
    y = cuda_lib.mx_nvfp4_gemm(t, w)
    clean = cuda_lib.mx_nvfp4_gemm(want, w)
    assert torch.isnan(y[[1, 3, 4]]).all() and torch.equal(y[good], clean[good])
    z = cuda_lib.mx_nvfp4_gemm(w, t)      # and as weights: their columns
    assert torch.isnan(z[:, [1, 3, 4]]).all() and torch.isfinite(z[:, good]).all()


def test_quantize_gathered_rows(cuda_lib):
    x = _rand((20, 160), 3).cuda()
    src = torch.tensor([3, -1, 19, 0, 0, -7, 11] + [-1] * 121, dtype=torch.int32, device="cuda")
    wide = torch.full((20, 200), float("nan"), dtype=BF, device="cuda")
    wide[:, :160] = x
    for rows in (x, wide[:, :160]):
        t = cuda_lib.mx_nvfp4_quantize(rows, src=src)
        _check_quantized(t, torch.where((src < 0)[:, None], 0.0, x[src.clamp(min=0).long()].to(D)).cpu())
    offsets = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    out = cuda_lib.NVFP4(128, 160)
    out.data.fill_(0x55), out.row_scale.fill_(7)
    part = cuda_lib.mx_nvfp4_quantize(x, src=src, offsets=offsets, out=out)
    assert torch.equal(part.data[:4], t.data[:4]) and (part.data[4:] == 0x55).all() and (part.row_scale[4:] == 7).all()
    src[2] = 20
    t = cuda_lib.mx_nvfp4_quantize(x, src=src)
    assert cuda_lib.mx_get_device_status() == "MX_ERR_INVALID_ARG"
    assert (t.data[2] == 0).all() and cuda_lib.mx_get_device_status() == "MX_OK"


@pytest.mark.parametrize("ends", [None, [200, 700], [0, 900]], ids=["all", "whole", "part"])
@pytest.mark.parametrize("T,K,R", [(70, 32768, 1030), (64, 16416, 1152), (1000, 2080, 9100), (3000, 1024, 20000)])
def test_quantize_copied_rows(cuda_lib, T, K, R, ends):
    """Rows that name tokens many times, copied from the tokens' quantization: the
    bytes of each row quantized for itself."""
    import ctypes
    gen = torch.Generator().manual_seed(T)
    x = _rand((T, K), T).cuda()
    x[T // 2, 5] = float("nan")
    src = torch.randint(-1, T, (R,), generator=gen, dtype=torch.int32).cuda()
    need = cuda_lib.mx_nvfp4_quantize_workspace_bytes(T, K, R)
    assert need > 0
    offsets = None if ends is None else torch.tensor([ends[0], ends[1] * R // 1000], dtype=torch.int32, device="cuda")

    def fresh():
        t = cuda_lib.NVFP4(R, K)
        t.data.fill_(0x55), t.scale.fill_(0x2A), t.row_scale.fill_(7)
        return t

    copied, itself = fresh(), fresh()
    cuda_lib.mx_nvfp4_quantize(x, src=src, offsets=offsets, out=copied)
    L = cuda_lib.load()
    assert L.mx_nvfp4_quantize(x.data_ptr(), T, K, K, src.data_ptr(), None if offsets is None else offsets.data_ptr(),
                               0 if offsets is None else 2, ctypes.byref(itself.struct()), None, 0, None) == 0
    assert torch.equal(copied.data, itself.data) and torch.equal(copied.scale, itself.scale)
    assert torch.equal(copied.row_scale.nan_to_num(-1.0), itself.row_scale.nan_to_num(-1.0))
    src[0] = T
    again = cuda_lib.mx_nvfp4_quantize(x, src=src, offsets=offsets)
    assert cuda_lib.mx_get_device_status() == "MX_ERR_INVALID_ARG" and (again.data[0] == 0).all()
    assert cuda_lib.mx_get_device_status() == "MX_OK"


def test_quantize_a_row_does_not_depend_on_the_others(cuda_lib):
    x = _rand((50, 512), 4).cuda()
    t, one = cuda_lib.mx_nvfp4_quantize(x), cuda_lib.mx_nvfp4_quantize(x[33:34])
    assert torch.equal(t.data[33:34], one.data) and torch.equal(t.row_scale[33:34], one.row_scale)


# ---------------------------------------------------------------- product

def _operand(mx, rows, cols, seed, exact=False, row_scale=True):
    """Random codes and scales (exact: small values whose sums fp32 holds)."""
    gen = torch.Generator().manual_seed(seed)
    data = torch.randint(0, 256, (rows, cols // 2), generator=gen, dtype=torch.uint8)
    if exact:
        data = data & 0x99                           # codes 0, 1, 8, 9: 0, 1/2 with either sign
        s8 = torch.tensor([0x38, 0x40, 0x30, 0x00], dtype=torch.uint8)[torch.randint(0, 4, (rows, cols // 16), generator=gen)]
        row = torch.exp2(torch.randint(-3, 4, (rows,), generator=gen).float())
    else:
        s8 = torch.randint(0, 0x7F, (rows, cols // 16), generator=gen, dtype=torch.uint8)
        row = torch.rand(rows, generator=gen) + 0.5
    scale = torch.zeros(mx.layers.nvfp4_scale_bytes(rows, cols), dtype=torch.uint8)
    scale[_blocked(rows, cols).reshape(-1)] = s8.reshape(-1)
    return mx.NVFP4(rows, cols, data=data.cuda(), scale=scale.cuda(), row_scale=row.cuda() if row_scale else None)


def _check_product(y, a, b, G, ends, exact=False):
    av, bv = _values(a).cuda(), _values(b).cuda()
    N, K = b.rows // G, a.cols
    begin = 0
    for g, end in enumerate(ends):
        if end > begin:
            w = bv[g * N:(g + 1) * N]
            ref, mag = av[begin:end] @ w.T, av[begin:end].abs() @ w.abs().T
            if exact:
                assert torch.equal(y[begin:end], ref.float().to(BF)), (g, begin, end)
            else:
                bound = 2.0 ** -8 * ref.abs() + (K / 64 + 8) * 2.0 ** -21 * mag + 2.0 ** -126
                bad = ~((y[begin:end].to(D) - ref).abs() <= bound)
                assert not bad.any(), "%d off in expert %d, worst %.3g" % (
                    int(bad.sum()), g, float(((y[begin:end].to(D) - ref).abs() / bound).max()))
        begin = end


@pytest.mark.parametrize("exact", [True, False], ids=["exact", "random"])
@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (1, 256, 64), (5, 136, 96), (128, 128, 256), (129, 264, 288), (300, 504, 320),
                                   (64, 1000, 1056), (257, 512, 2048), (1, 4096, 4096), (16, 2304, 512), (700, 776, 544),
                                   (2000, 2560, 256)])
def test_product(cuda_lib, M, N, K, exact):
    a, b = _operand(cuda_lib, M, K, M + N, exact), _operand(cuda_lib, N, K, K, exact)
    y = cuda_lib.mx_nvfp4_gemm(a, b)
    _check_product(y, a, b, 1, [M], exact)
    assert torch.equal(y, cuda_lib.mx_nvfp4_gemm(a, b)) and cuda_lib.mx_get_device_status() == "MX_OK"


def test_product_without_row_scales_and_with_a_row_stride(cuda_lib):
    a, b = _operand(cuda_lib, 70, 128, 1, row_scale=False), _operand(cuda_lib, 72, 128, 2, row_scale=False)
    buf = torch.full((75, 96), 7.0, dtype=BF, device="cuda")
    cuda_lib.mx_nvfp4_gemm(a, b, out=buf[:70, :72])
    _check_product(buf[:70, :72], a, b, 1, [70])
    assert (buf[70:] == 7).all() and (buf[:, 72:] == 7).all()


@pytest.mark.parametrize("N,K", [(128, 64), (256, 288), (384, 512), (640, 1024)])
@pytest.mark.parametrize("ends", [[128], [0, 128, 128, 512], [256, 256, 384, 1024], [0, 0, 0], [384, 640, 768, 896, 1280]],
                         ids=str)
def test_grouped_product(cuda_lib, ends, N, K):
    G, R = len(ends), max(1280, ends[-1])
    a, b = _operand(cuda_lib, R, K, N, True), _operand(cuda_lib, G * N, K, K, True)
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    out = torch.full((R, N), 7.0, dtype=BF, device="cuda")
    y = cuda_lib.mx_nvfp4_gemm(a, b, G, offsets, out=out)
    _check_product(y, a, b, G, ends, True)
    assert (out[ends[-1]:] == 7).all()
    b.row_scale = None
    _check_product(cuda_lib.mx_nvfp4_gemm(a, b, G, offsets), a, b, G, ends, True)


def test_other_experts_values_stay_out(cuda_lib):
    """A tile of 256 columns meets the next expert's weights: NaN there goes nowhere."""
    a, b = _operand(cuda_lib, 256, 128, 1), _operand(cuda_lib, 2 * 128, 128, 2)
    offsets = torch.tensor([128, 256], dtype=torch.int32, device="cuda")
    want = cuda_lib.mx_nvfp4_gemm(a, b, 2, offsets)
    b.row_scale[128:] = float("nan")
    b.scale[b.scale.numel() // 2:] = 0x7F              # NaN scales of the second expert's rows
    got = cuda_lib.mx_nvfp4_gemm(a, b, 2, offsets)
    assert torch.equal(got[:128], want[:128]) and torch.isnan(got[128:]).all()


def test_malformed_segments_are_reported(cuda_lib):
    a, b = _operand(cuda_lib, 384, 64, 1, True), _operand(cuda_lib, 3 * 128, 64, 2, True)
    out = torch.full((384, 128), 7.0, dtype=BF, device="cuda")
    cuda_lib.mx_nvfp4_gemm(a, b, 3, torch.tensor([128, 200, 384], dtype=torch.int32, device="cuda"), out=out)
    assert cuda_lib.mx_get_device_status() == "MX_ERR_OFFSETS"
    _check_product(out, a, b, 3, [128, 128, 128], True)
    assert cuda_lib.mx_get_device_status() == "MX_OK"


def test_quantized_layer(cuda_lib):
    """BF16 through quantization and product: the result is the values' product, and
    close to the BF16 product (4 bits: a tenth of its norm)."""
    x, w = _rand((333, 1024), 5), _rand((768, 1024), 6, 0.02)
    x /= x.float().abs().amax(1, keepdim=True).to(BF)
    w /= w.float().abs().amax(1, keepdim=True).to(BF)
    a, b = cuda_lib.mx_nvfp4_quantize(x.cuda()), cuda_lib.mx_nvfp4_quantize(w.cuda())
    y = cuda_lib.mx_nvfp4_gemm(a, b)
    _check_product(y, a, b, 1, [333])
    full = x.double() @ w.double().T
    assert float((y.cpu().double() - full).norm() / full.norm()) < 0.2


def test_streams_and_graphs(cuda_lib):
    x = [_rand((500, 512), i).cuda() for i in (7, 8)]
    w = cuda_lib.mx_nvfp4_quantize(_rand((640, 512), 9).cuda())

    def call(x, stream=None):
        return cuda_lib.mx_nvfp4_gemm(cuda_lib.mx_nvfp4_quantize(x, stream=stream), w, stream=stream)

    want = [call(v) for v in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]
    for _ in range(10):
        got = [call(v, s) for v, s in zip(x, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, v) for g, v in zip(got, want))
    v = x[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(v)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(v)
    for i in (1, 0):
        v.copy_(x[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])


def test_no_rows(cuda_lib):
    t = cuda_lib.mx_nvfp4_quantize(torch.empty((0, 64), dtype=BF, device="cuda"))
    w = _operand(cuda_lib, 64, 64, 1)
    assert cuda_lib.mx_nvfp4_gemm(t, w).shape == (0, 64)
