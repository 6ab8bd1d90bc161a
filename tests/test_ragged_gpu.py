"""The BF16 ragged products and the linear layer against a plain fp64
implementation: segment lengths from none to long, odd sizes, strides,
non-finite neighbours, refusals on the device.

Tolerances.  Products of BF16 values are exact in fp32; the kernels add K of
them in fp32 with any order of sums.  With the sums' magnitudes S = sum |a b|
the fp32 error is at most K * 2^-23 * S per value (2^-23: an accumulator that
truncates), rounding to BF16 adds 2^-8 relative to the result, half a unit
being 2^-9, doubled to keep clear of the bound itself.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _bf16(shape, gen, std=1.0):
    return (torch.randn(shape, generator=gen, dtype=torch.float32) * std).to(torch.bfloat16).cuda()


def _offsets(counts):
    return torch.tensor(np.cumsum(counts), dtype=torch.int32).cuda()


def _check(got, ref, mag, K, rel):
    """|got - ref| <= rel |ref| + K 2^-23 mag (+ the smallest BF16 normal)."""
    got, ref = got.double(), ref.double()
    bound = rel * ref.abs() + K * 2.0 ** -23 * mag.double() + 2.0 ** -126
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), "%d of %d values off, worst %.3g x the bound" % (
        int(bad.sum()), bad.numel(), float(((got - ref).abs() / bound).max()))


def _ragged_ref(a, w, counts, kn):
    ref = torch.zeros((a.shape[0], w.shape[2 if kn else 1]), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    b = 0
    for g, c in enumerate(counts):
        m = w[g].double() if kn else w[g].double().T
        ref[b:b + c] = a[b:b + c].double() @ m
        mag[b:b + c] = a[b:b + c].double().abs() @ m.abs()
        b += c
    return ref, mag


COUNTS = {
    "one row": [1],
    "one row of many experts": [0] * 5 + [1] + [0] * 6,
    "eight single rows": [1, 0, 1, 1, 0, 0, 1, 1, 1, 1, 0, 1],
    "empty ends": [0, 3, 0, 0, 129, 0],
    "tile edges": [127, 128, 129, 255, 256, 257, 1, 31, 33],
    "one long": [0, 0, 1500, 0],
    "many": [(7 * i * i) % 41 for i in range(128)],
}


@pytest.mark.parametrize("kn", [False, True], ids=["NK", "KN"])
@pytest.mark.parametrize("N,K", [(8, 8), (64, 72), (200, 136), (256, 64), (328, 520), (1032, 264)])
@pytest.mark.parametrize("name", list(COUNTS))
def test_ragged_gemm(cuda_lib, name, N, K, kn):
    mx = cuda_lib
    counts = COUNTS[name]
    R, G = sum(counts), len(counts)
    gen = torch.Generator().manual_seed(R * 7 + N + K)
    a = _bf16((R, K), gen)
    w = _bf16((G, K, N) if kn else (G, N, K), gen)
    out = mx.mx_ragged_gemm(a, w, _offsets(counts), layout=mx.W_KN if kn else mx.W_NK)
    assert mx.mx_get_device_status() == "MX_OK"
    ref, mag = _ragged_ref(a, w, counts, kn)
    _check(out, ref, mag, K, 2.0 ** -8)


@pytest.mark.parametrize("kn", [False, True], ids=["NK", "KN"])
@pytest.mark.parametrize("R", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 100, 128, 129, 300])
def test_ragged_gemm_row_counts(cuda_lib, R, kn):
    """Every row count around the kernels' tile heights, one segment, no offsets."""
    mx = cuda_lib
    gen = torch.Generator().manual_seed(R)
    N, K = 264, 1096
    a = _bf16((R, K), gen)
    w = _bf16((1, K, N) if kn else (1, N, K), gen)
    out = mx.mx_ragged_gemm(a, w, None, layout=mx.W_KN if kn else mx.W_NK)
    ref, mag = _ragged_ref(a, w, [R], kn)
    _check(out, ref, mag, K, 2.0 ** -8)


@pytest.mark.parametrize("R", [5, 700])
@pytest.mark.parametrize("kn", [False, True], ids=["NK", "KN"])
def test_ragged_gemm_strides_and_untouched_rows(cuda_lib, kn, R):
    """Row strides wider than the rows; rows past the last segment and the
    columns past N of the output's rows keep what they held."""
    mx = cuda_lib
    counts = [R // 3, 0, R - R // 3]
    gen = torch.Generator().manual_seed(3 + R)
    K, N, tail = 152, 168, 9
    abuf = _bf16((R + tail, K + 24), gen)
    a = abuf[:, 8:8 + K]
    w = _bf16((3, K, N) if kn else (3, N, K), gen)
    obuf = torch.full((R + tail, N + 40), 7.0, dtype=torch.bfloat16, device="cuda")
    out = obuf[:, 16:16 + N]
    mx.mx_ragged_gemm(a, w, _offsets(counts), layout=mx.W_KN if kn else mx.W_NK, out=out)
    ref, mag = _ragged_ref(a[:R], w, counts, kn)
    _check(out[:R], ref, mag, K, 2.0 ** -8)
    obuf[:R, 16:16 + N] = 7.0
    assert bool((obuf == 7.0).all())


@pytest.mark.parametrize("kn", [False, True], ids=["NK", "KN"])
def test_ragged_gemm_nonfinite_neighbours(cuda_lib, kn):
    """NaN and Inf in one expert's rows, in its weights and past the last
    segment reach no other expert's results."""
    mx = cuda_lib
    counts = [5, 130, 3, 260]
    R, N, K = sum(counts), 136, 200
    gen = torch.Generator().manual_seed(11)
    a = _bf16((R + 4, K), gen)
    w = _bf16((4, K, N) if kn else (4, N, K), gen)
    a[5:135] = float("nan")
    w[1] = float("inf")
    a[R:] = float("nan")
    out = mx.mx_ragged_gemm(a, w, _offsets(counts), layout=mx.W_KN if kn else mx.W_NK)
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[5:135] = False
    a2, w2 = a[:R].clone(), w.clone()
    a2[5:135], w2[1] = 0, 0
    ref, mag = _ragged_ref(a2, w2, counts, kn)
    _check(out[:R][keep], ref[keep], mag[keep], K, 2.0 ** -8)
    assert bool(out[5:135].isnan().all())


def test_ragged_gemm_malformed_offsets(cuda_lib):
    """A decreasing segment and one past R are skipped and reported; the
    others are computed."""
    mx = cuda_lib
    gen = torch.Generator().manual_seed(2)
    R, N, K = 40, 64, 64
    a, w = _bf16((R, K), gen), _bf16((3, N, K), gen)
    out = torch.full((R, N), 3.0, dtype=torch.bfloat16, device="cuda")
    mx.mx_ragged_gemm(a, w, torch.tensor([10, 4, 99], dtype=torch.int32, device="cuda"), out=out)
    assert mx.mx_get_device_status() == "MX_ERR_OFFSETS"
    assert mx.mx_get_device_status() == "MX_OK"
    ref, mag = _ragged_ref(a[:10], w[:1], [10], False)
    _check(out[:10], ref, mag, K, 2.0 ** -8)
    assert bool((out[10:] == 3.0).all())


@pytest.mark.parametrize("ends,good", [([3, 1, 3, 9], [(0, 0, 3)]), ([2, 2, 5, 4, 7, 8], [(0, 0, 2), (2, 2, 5), (5, 7, 8)]),
                                       ([-4, 2, 6], [(2, 2, 6)]), ([0, 0, 8], [(2, 0, 8)])])
def test_ragged_gemm_malformed_offsets_few_rows(cuda_lib, ends, good):
    """The same for a few rows: (expert, begin, end) of the segments that count."""
    mx = cuda_lib
    gen = torch.Generator().manual_seed(2)
    R, N, K, G = 8, 72, 64, len(ends)
    a, w = _bf16((R, K), gen), _bf16((G, N, K), gen)
    out = torch.full((R, N), 3.0, dtype=torch.bfloat16, device="cuda")
    mx.mx_ragged_gemm(a, w, torch.tensor(ends, dtype=torch.int32, device="cuda"), out=out)
    bad = any(e < s or e > R or s < max([0] + ends[:g]) for g, (s, e) in enumerate(zip([0] + ends, ends)))
    assert mx.mx_get_device_status() == ("MX_ERR_OFFSETS" if bad else "MX_OK")
    rest = torch.ones(R, dtype=torch.bool, device="cuda")
    for g, b, e in good:
        ref, mag = _ragged_ref(a[b:e], w[g:g + 1], [e - b], False)
        _check(out[b:e], ref, mag, K, 2.0 ** -8)
        rest[b:e] = False
    assert bool((out[rest] == 3.0).all())


def test_ragged_gemm_validates_on_request(cuda_lib, monkeypatch):
    mx = cuda_lib
    a = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((2, 64, 64), dtype=torch.bfloat16, device="cuda")
    monkeypatch.setenv("MX_VALIDATE_OFFSETS", "1")
    for bad in ([5, 3], [4, 9]):
        with pytest.raises(mx.MXError, match="OFFSETS"):
            mx.mx_ragged_gemm(a, w, torch.tensor(bad, dtype=torch.int32, device="cuda"))
    mx.mx_ragged_gemm(a, w, torch.tensor([5, 8], dtype=torch.int32, device="cuda"))


def test_ragged_gemm_on_another_stream_and_graph(cuda_lib):
    """The call goes to the given stream only, and can be captured and
    replayed with other offsets in the same buffer."""
    mx = cuda_lib
    gen = torch.Generator().manual_seed(5)
    R, N, K, G = 333, 264, 128, 4
    a, w = _bf16((R, K), gen), _bf16((G, N, K), gen)
    off = _offsets([100, 0, 200, 33])
    out = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mx.mx_ragged_gemm(a, w, off, out=out)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mx_ragged_gemm(a, w, off, out=out)
    for counts in ([1, 2, 329, 1], [0, 0, 0, 333]):
        off.copy_(_offsets(counts))
        graph.replay()
        ref, mag = _ragged_ref(a, w, counts, False)
        _check(out, ref, mag, K, 2.0 ** -8)


def test_ragged_gemm_past_two_gib_of_elements(cuda_lib):
    """Row offsets past 2^31 elements: a strided view whose last rows lie
    beyond them."""
    mx = cuda_lib
    R, K, N, ld = 300, 64, 64, 1 << 23
    gen = torch.Generator().manual_seed(9)
    buf = torch.empty(R * ld, dtype=torch.bfloat16, device="cuda")
    a = buf.view(R, ld)[:, :K]
    a.copy_(_bf16((R, K), gen))
    w = _bf16((2, N, K), gen)
    out = buf.view(R, ld)[:, 128:128 + N]
    mx.mx_ragged_gemm(a, w, _offsets([17, 283]), out=out)
    ref, mag = _ragged_ref(a, w, [17, 283], False)
    _check(out, ref, mag, K, 2.0 ** -8)


# ------------------------------------------------------------------ gradients

@pytest.mark.parametrize("N,K", [(8, 8), (64, 136), (136, 64), (264, 200), (520, 392)])
@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("kind", ["bf16", "f32", "acc"])
def test_ragged_wgrad(cuda_lib, name, N, K, kind):
    mx = cuda_lib
    counts = COUNTS[name]
    R, G = sum(counts), len(counts)
    gen = torch.Generator().manual_seed(R + N * 3 + K)
    dy, x = _bf16((R, N), gen), _bf16((R, K), gen)
    off = _offsets(counts)
    if kind == "bf16":
        got = mx.mx_ragged_gemm_wgrad(dy, x, G, off)
    else:
        got = torch.randn((G, N, K), generator=gen).cuda()
        before = got.double()
        mx.mx_ragged_gemm_wgrad_f32(dy, x, G, off, got, accumulate=kind == "acc")
    assert mx.mx_get_device_status() == "MX_OK"
    b = 0
    for g, c in enumerate(counts):
        d, e = dy[b:b + c].double(), x[b:b + c].double()
        ref, mag = d.T @ e, d.abs().T @ e.abs()
        if kind == "acc":
            ref = ref + before[g]
        _check(got[g], ref, mag, max(c, 1), 2.0 ** -8 if kind == "bf16" else 2.0 ** -23)
        if c == 0:
            assert torch.equal(got[g].double(), ref)
        b += c


def test_ragged_wgrad_nonfinite_neighbours_and_strides(cuda_lib):
    """Rows of other experts and past the last segment that hold NaN and Inf,
    read through strided views, reach no other expert's gradient."""
    mx = cuda_lib
    counts = [3, 70, 129, 1, 64]
    R, N, K = sum(counts), 136, 72
    gen = torch.Generator().manual_seed(21)
    dy = _bf16((R + 20, N + 16), gen)[:, 8:8 + N]
    x = _bf16((R + 20, K + 8), gen)[:, :K]
    dy[3:73], x[3:73] = float("nan"), float("inf")
    dy[R:], x[R:] = float("inf"), float("nan")
    got = mx.mx_ragged_gemm_wgrad(dy, x, 5, _offsets(counts))
    b = 0
    for g, c in enumerate(counts):
        if g != 1:
            d, e = dy[b:b + c].double(), x[b:b + c].double()
            _check(got[g], d.T @ e, d.abs().T @ e.abs(), c, 2.0 ** -8)
        b += c
    assert bool(got[1].isnan().all())


def test_ragged_wgrad_is_deterministic_and_takes_no_rows(cuda_lib):
    mx = cuda_lib
    gen = torch.Generator().manual_seed(4)
    counts = [2000, 0, 3, 5000]
    R, N, K = sum(counts), 264, 520
    dy, x = _bf16((R, N), gen), _bf16((R, K), gen)
    first = mx.mx_ragged_gemm_wgrad(dy, x, 4, _offsets(counts))
    for _ in range(3):
        assert torch.equal(first, mx.mx_ragged_gemm_wgrad(dy, x, 4, _offsets(counts)))
    none = torch.empty((0, N), dtype=torch.bfloat16, device="cuda")
    g = mx.mx_ragged_gemm_wgrad(none, torch.empty((0, K), dtype=torch.bfloat16, device="cuda"), 2,
                                torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert not bool(g.any())


def test_ragged_wgrad_long_segment_fp32(cuda_lib):
    """A long sum in fp32: 2-norm error within 2e-5 of the result's."""
    mx = cuda_lib
    gen = torch.Generator().manual_seed(8)
    R, N, K = 65536, 64, 128
    dy, x = _bf16((R, N), gen), _bf16((R, K), gen)
    got = mx.mx_ragged_gemm_wgrad_f32(dy, x, 1, None, torch.empty((1, N, K), device="cuda"))[0].double()
    ref = dy.double().T @ x.double()
    assert float((got - ref).norm() / ref.norm()) < 2e-5


def test_gradients_are_the_products_derivatives(cuda_lib):
    """dX and dW of sum(out * dY) against finite differences.  out is linear
    in a and in w, so a difference over a step h has no error of its own but
    the rounding of the fp64 reference of out."""
    mx = cuda_lib
    counts = [5, 0, 12]
    R, N, K, G = 17, 40, 24, 3
    gen = torch.Generator().manual_seed(6)
    a, w, dy = _bf16((R, K), gen), _bf16((G, N, K), gen), _bf16((R, N), gen)
    off = _offsets(counts)
    dx = mx.mx_ragged_gemm(dy, w, off, layout=mx.W_KN)
    dw = mx.mx_ragged_gemm_wgrad(dy, a, G, off)

    def value(a, w):
        return float((_ragged_ref(a, w, counts, False)[0] * dy.double()).sum())

    rng = np.random.default_rng(0)
    for _ in range(12):
        r, k = int(rng.integers(R)), int(rng.integers(K))
        up, dn = a.double(), a.double()
        up[r, k] += 0.5
        dn[r, k] -= 0.5
        diff = value(up, w) - value(dn, w)
        assert abs(diff - float(dx[r, k])) <= 2.0 ** -8 * abs(diff) + 1e-3
        g, n = int(rng.choice([0, 2])), int(rng.integers(N))
        up, dn = w.double(), w.double()
        up[g, n, k] += 0.5
        dn[g, n, k] -= 0.5
        diff = value(a, up) - value(a, dn)
        assert abs(diff - float(dw[g, n, k])) <= 2.0 ** -8 * abs(diff) + 1e-3


# --------------------------------------------------------------- linear layer

def _act(z, act, mx):
    if act == mx.ACT_RELU:
        return z.clamp(min=0)
    if act == mx.ACT_SILU:
        return z * torch.sigmoid(z)
    if act == mx.ACT_GELU_TANH:
        return 0.5 * z * (1 + torch.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)))
    return z


@pytest.mark.parametrize("act", ["NONE", "GELU_TANH", "SILU", "RELU"])
@pytest.mark.parametrize("bias,res", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("M,N,K", [(1, 264, 520), (3, 8, 16), (33, 136, 72), (130, 512, 256), (300, 328, 1000)])
def test_linear(cuda_lib, act, bias, res, M, N, K):
    mx = cuda_lib
    act = getattr(mx, "ACT_" + act)
    gen = torch.Generator().manual_seed(M + N + K)
    x, w = _bf16((M, K), gen), _bf16((N, K), gen, K ** -0.5)
    b = _bf16((N,), gen) if bias else None
    r = _bf16((M, N), gen) if res else None
    out = mx.mx_linear_fwd(x, w, b, act, r)
    assert mx.mx_get_device_status() == "MX_OK"
    z = x.double() @ w.double().T
    mag = x.double().abs() @ w.double().abs().T
    if bias:
        z, mag = z + b.double(), mag + b.double().abs()
    h = _act(z, act, mx)
    ref = h + r.double() if res else h
    # activations: slope at most 1.13, and 2^-18 relative for their own fp32 arithmetic
    _check(out, ref, 1.13 * mag + h.abs() * (2.0 ** 5 / K) + (r.double().abs() / K if res else 0), K, 2.0 ** -8)


def test_linear_residual_in_place_and_strides(cuda_lib):
    mx = cuda_lib
    gen = torch.Generator().manual_seed(1)
    for M in (4, 200):
        N, K = 136, 264
        x, w = _bf16((M, K + 8), gen)[:, :K], _bf16((N, K), gen, 0.1)
        buf = _bf16((M, N + 24), gen)
        before = buf.clone()
        out = buf[:, 8:8 + N]
        mx.mx_linear_fwd(x, w, None, mx.ACT_NONE, out, out=out)
        ref = x.double() @ w.double().T + before[:, 8:8 + N].double()
        mag = x.double().abs() @ w.double().abs().T + before[:, 8:8 + N].double().abs()
        _check(out, ref, mag, K, 2.0 ** -8)
        buf[:, 8:8 + N] = before[:, 8:8 + N]
        assert torch.equal(buf, before)


@pytest.mark.parametrize("M,N,K", [(1, 32, 64), (5, 160, 136), (127, 256, 64), (129, 544, 72), (700, 1056, 128)])
def test_linear_checkpoint_bytes(cuda_lib, M, N, K):
    """On exact data (small integers: every sum is exact in fp32 and in BF16)
    the checkpoint is the quantizer's rowwise output, byte for byte, scale
    padding included."""
    mx = cuda_lib
    gen = torch.Generator().manual_seed(M)
    x = torch.randint(-1, 2, (M, K), generator=gen).to(torch.bfloat16).cuda()
    w = torch.randint(-1, 2, (N, K), generator=gen).to(torch.bfloat16).cuda()
    ck = mx.MX(M, N)
    ck.scale.fill_(0xAB)
    out = mx.mx_linear_fwd(x, w, None, mx.ACT_RELU, ckpt=ck)
    z = (x.float() @ w.float().T).to(torch.bfloat16)
    ref, _, _ = mx.mx_quantize(z, mx.E4M3, True, False)
    assert torch.equal(out, z.clamp(min=0))
    assert torch.equal(ck.data, ref.data) and torch.equal(ck.scale, ref.scale)


def test_ragged_wgrad_stage_reuse_ends_promptly(cuda_lib):
    """Segments whose last blocks (zeroed past their end) and whole blocks
    alternate in every stage of the ring, ending on either kind: the launch
    ends by itself, far below the bound of a wait (2 s)."""
    mx = cuda_lib
    gen = torch.Generator().manual_seed(12)
    N, K = 264, 264
    for tail in range(1, 14):
        counts = [64 * (i % 5) + (3 if (i + tail) % 2 else 0) for i in range(tail)] + [64 * tail + 5, 64]
        R = sum(counts)
        dy, x = _bf16((R, N), gen), _bf16((R, K), gen)
        off = _offsets(counts)
        mx.mx_ragged_gemm_wgrad(dy, x, len(counts), off)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        mx.mx_ragged_gemm_wgrad(dy, x, len(counts), off)
        b.record()
        assert mx.mx_get_device_status() == "MX_OK"
        assert a.elapsed_time(b) < 500.0


# More tiles than CTA pairs: every pair takes over tiles of other experts, of
# other widths and of another number of contraction steps.

@pytest.mark.parametrize("kn", [False, True], ids=["NK", "KN"])
@pytest.mark.parametrize("N,K", [(1024, 136), (512, 200), (768, 72), (2048, 328)])
def test_ragged_gemm_many_tiles(cuda_lib, N, K, kn):
    mx = cuda_lib
    counts = [(37 * i * i) % 331 for i in range(160)]
    counts[5] = counts[77] = 0
    counts[40] = 1500
    R, G = sum(counts), len(counts)
    gen = torch.Generator().manual_seed(N + K)
    a = _bf16((R + 3, K), gen)
    a[R:] = float("nan")
    w = _bf16((G, K, N) if kn else (G, N, K), gen)
    out = torch.full((R + 3, N), 9.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        mx.mx_ragged_gemm(a, w, _offsets(counts), layout=mx.W_KN if kn else mx.W_NK, out=out)
    assert mx.mx_get_device_status() == "MX_OK"
    ref, mag = _ragged_ref(a[:R], w, counts, kn)
    _check(out[:R], ref, mag, K, 2.0 ** -8)
    assert bool((out[R:] == 9.0).all())


@pytest.mark.parametrize("kind", ["bf16", "f32", "acc"])
@pytest.mark.parametrize("N,K", [(264, 512), (40, 1024), (520, 1000), (136, 2048)])
def test_ragged_wgrad_many_tiles(cuda_lib, N, K, kind):
    mx = cuda_lib
    counts = [(13 * i * i) % 97 for i in range(170)]
    counts[3] = counts[4] = 0
    counts[9] = 4500
    R, G = sum(counts), len(counts)
    gen = torch.Generator().manual_seed(N + K)
    dy, x = _bf16((R + 7, N), gen), _bf16((R + 7, K), gen)
    dy[R:], x[R:] = float("inf"), float("nan")
    off = _offsets(counts)
    if kind == "bf16":
        got = mx.mx_ragged_gemm_wgrad(dy, x, G, off)
        assert torch.equal(got, mx.mx_ragged_gemm_wgrad(dy, x, G, off))
    else:
        got = torch.randn((G, N, K), generator=gen).cuda()
        before = got.clone()
        mx.mx_ragged_gemm_wgrad_f32(dy, x, G, off, got, accumulate=kind == "acc")
    assert mx.mx_get_device_status() == "MX_OK"
    b = 0
    for g, c in enumerate(counts):
        d, e = dy[b:b + c].double(), x[b:b + c].double()
        ref, mag = d.T @ e, d.abs().T @ e.abs()
        if kind == "acc":
            ref = ref + before[g].double()
        _check(got[g], ref, mag, max(c, 1), 2.0 ** -8 if kind == "bf16" else 2.0 ** -23)
        b += c


@pytest.mark.parametrize("G,rows,N,K", [(3, 5, 264, 520), (170, 5, 264, 520), (4, 20000, 136, 264)])
def test_ragged_wgrad_accumulate_leaves_empty_experts_alone(cuda_lib, G, rows, N, K):
    """Bit for bit: negative zeros, subnormals and NaN payloads stay (the last
    case sums its segments in parts)."""
    mx = cuda_lib
    counts = [0 if g % 3 else rows for g in range(G)]
    assert (mx.mx_ragged_gemm_wgrad_workspace_bytes(N, K, sum(counts), G) > 0) == (rows > 5)
    gen = torch.Generator().manual_seed(G)
    dy, x = _bf16((sum(counts), N), gen), _bf16((sum(counts), K), gen)
    before = torch.randint(-2 ** 31, 2 ** 31 - 1, (G, N, K), generator=gen, dtype=torch.int32).cuda()
    before[1, :, ::3] = -2 ** 31
    got = before.clone().view(torch.float32)
    mx.mx_ragged_gemm_wgrad_f32(dy, x, G, _offsets(counts), got, accumulate=True)
    assert mx.mx_get_device_status() == "MX_OK"
    for g, c in enumerate(counts):
        assert torch.equal(got[g].view(torch.int32), before[g]) == (c == 0)


@pytest.mark.parametrize("M,N,K", [(20011, 1024, 72), (9000, 2560, 136)])
def test_linear_many_tiles(cuda_lib, M, N, K):
    """Bias, activation, residual and checkpoint together."""
    mx = cuda_lib
    gen = torch.Generator().manual_seed(M)
    x, w, b, r = _bf16((M, K), gen), _bf16((N, K), gen, K ** -0.5), _bf16((N,), gen), _bf16((M, N), gen)
    ck = mx.MX(M, N)
    out = mx.mx_linear_fwd(x, w, b, mx.ACT_GELU_TANH, r, ckpt=ck)
    assert mx.mx_get_device_status() == "MX_OK"
    z = x.double() @ w.double().T + b.double()
    mag = x.double().abs() @ w.double().abs().T + b.double().abs()
    h = _act(z, mx.ACT_GELU_TANH, mx)
    _check(out, h + r.double(), 1.13 * mag + h.abs() * (2.0 ** 5 / K) + r.double().abs() / K, K, 2.0 ** -8)
    # the checkpoint's values: half a unit of 4 significant bits, or of the block's subnormals
    q, s = ck.data.view(torch.float8_e4m3fn), ck.scale
    rows = torch.arange(M, device="cuda").unsqueeze(1)
    cols = torch.arange(N // 32, device="cuda").unsqueeze(0)
    at = (rows // 128 * (N // 128) + cols // 4) * 512 + rows % 32 * 16 + rows % 128 // 32 * 4 + cols % 4
    scale = torch.exp2(s[at].double() - 127).repeat_interleave(32, 1)
    assert bool(((q.double() * scale - z).abs() <= 2.0 ** -4 * z.abs() + 2.0 ** -10 * scale).all())
    blocks = z.abs().view(M, N // 32, 32).amax(-1)
    assert bool((blocks <= 448 * (1 + 1e-5) * scale[:, ::32]).all())
    assert bool((blocks * (1 + 1e-5) > 224 * scale[:, ::32]).all())
    pad = torch.arange(M, (M + 127) // 128 * 128, device="cuda").unsqueeze(1)
    at = (pad // 128 * (N // 128) + cols // 4) * 512 + pad % 32 * 16 + pad % 128 // 32 * 4 + cols % 4
    assert not bool(s[at].any())


@pytest.mark.parametrize("kind", ["bf16", "f32", "acc"])
@pytest.mark.parametrize("counts,N,K", [([9001], 64, 72), ([5000, 0, 17000, 3], 136, 264), ([5000] * 8, 40, 8),
                                        ([30011], 520, 200)])
def test_ragged_wgrad_few_tiles(cuda_lib, counts, N, K, kind):
    """Few output tiles and long segments: the parts of a segment are summed
    apart and added in order."""
    mx = cuda_lib
    R, G = sum(counts), len(counts)
    assert mx.mx_ragged_gemm_wgrad_workspace_bytes(N, K, R, G) > 0
    gen = torch.Generator().manual_seed(R + N)
    dy, x = _bf16((R + 70, N), gen), _bf16((R + 70, K), gen)
    dy[R:], x[R:] = float("nan"), float("inf")
    off = _offsets(counts)
    if kind == "bf16":
        got = mx.mx_ragged_gemm_wgrad(dy, x, G, off)
        assert torch.equal(got, mx.mx_ragged_gemm_wgrad(dy, x, G, off))
    else:
        got = torch.randn((G, N, K), generator=gen).cuda()
        before = got.clone()
        mx.mx_ragged_gemm_wgrad_f32(dy, x, G, off, got, accumulate=kind == "acc")
    assert mx.mx_get_device_status() == "MX_OK"
    b = 0
    for g, c in enumerate(counts):
        d, e = dy[b:b + c].double(), x[b:b + c].double()
        ref, mag = d.T @ e, d.abs().T @ e.abs()
        if kind == "acc":
            ref = ref + before[g].double()
        _check(got[g], ref, mag, max(c, 1), 2.0 ** -8 if kind == "bf16" else 2.0 ** -22)
        b += c


def test_ragged_wgrad_workspace_refused(cuda_lib):
    mx = cuda_lib
    R, N, K = 20000, 64, 64
    dy = torch.zeros((R, N), dtype=torch.bfloat16, device="cuda")
    n = mx.mx_ragged_gemm_wgrad_workspace_bytes(N, K, R, 1)
    with pytest.raises(mx.MXError, match="WORKSPACE"):
        mx.mx_ragged_gemm_wgrad(dy, dy, 1, None, workspace=torch.empty(n - 4, dtype=torch.uint8, device="cuda"))


# --------------------------------------------- few tiles, long contractions

@pytest.mark.parametrize("act,bias,res,ckpt", [("NONE", False, False, False), ("SILU", True, False, False),
                                               ("GELU_TANH", True, True, True), ("RELU", False, True, False)])
@pytest.mark.parametrize("M,N,K", [(9, 128, 2944), (16, 2048, 1032), (53, 128, 4104), (77, 1056, 1992),
                                   (300, 2048, 1288), (600, 1024, 2056), (777, 2048, 1536), (130, 264, 16384)])
def test_linear_long_contraction(cuda_lib, M, N, K, act, bias, res, ckpt):
    """Tiles whose contraction several pairs share, among them ones with a
    last block of 8 and of 40 steps, and fewer blocks than tokens' blocks."""
    mx = cuda_lib
    act = getattr(mx, "ACT_" + act)
    ckpt = ckpt and N % 32 == 0
    gen = torch.Generator().manual_seed(M + N + K)
    x, w = _bf16((M, K + 8), gen)[:, :K], _bf16((N, K), gen, K ** -0.5)
    b = _bf16((N,), gen) if bias else None
    r = _bf16((M, N), gen) if res else None
    ck = mx.MX(M, N) if ckpt else None
    out = mx.mx_linear_fwd(x, w, b, act, r, ckpt=ck)
    assert mx.mx_get_device_status() == "MX_OK"
    z = x.double() @ w.double().T
    mag = x.double().abs() @ w.double().abs().T
    if bias:
        z, mag = z + b.double(), mag + b.double().abs()
    h = _act(z, act, mx)
    ref = h + r.double() if res else h
    _check(out, ref, 1.13 * mag + h.abs() * (2.0 ** 5 / K) + (r.double().abs() / K if res else 0), K, 2.0 ** -8)
    assert torch.equal(out, mx.mx_linear_fwd(x, w, b, act, r))
    if ckpt:
        rows = torch.arange(M, device="cuda").unsqueeze(1)
        cols = torch.arange(N // 32, device="cuda").unsqueeze(0)
        at = (rows // 128 * ((N + 127) // 128) + cols // 4) * 512 + rows % 32 * 16 + rows % 128 // 32 * 4 + cols % 4
        scale = torch.exp2(ck.scale[at].double() - 127).repeat_interleave(32, 1)
        # half a unit of the code, and the sums' own error
        off = (ck.data.view(torch.float8_e4m3fn).double() * scale - z).abs()
        assert bool((off <= 2.0 ** -4 * z.abs() + 2.0 ** -10 * scale + K * 2.0 ** -22 * mag).all())


@pytest.mark.parametrize("kn", [False, True], ids=["NK", "KN"])
@pytest.mark.parametrize("counts,N,K", [([33], 520, 2056), ([0, 7, 0, 50], 264, 3144), ([200, 1, 129], 136, 1544),
                                        ([16, 16], 2048, 1024), ([700], 1024, 4104)])
def test_ragged_gemm_long_contraction(cuda_lib, counts, N, K, kn):
    """The same for the ragged product, with NaN and Inf in another expert's
    rows and past the last one."""
    mx = cuda_lib
    R, G = sum(counts), len(counts)
    gen = torch.Generator().manual_seed(R + N + K)
    a = _bf16((R + 40, K), gen)
    w = _bf16((G, K, N) if kn else (G, N, K), gen, K ** -0.5)
    out = torch.full((R + 40, N), 9.0, dtype=torch.bfloat16, device="cuda")
    a[R:] = float("nan")
    if G > 1:
        a[:counts[0]] = float("inf")
    mx.mx_ragged_gemm(a, w, _offsets(counts), layout=mx.W_KN if kn else mx.W_NK, out=out)
    assert mx.mx_get_device_status() == "MX_OK"
    first = counts[0] if G > 1 else 0
    ref, mag = _ragged_ref(a[:R], w, counts, kn)
    _check(out[first:R], ref[first:], mag[first:], K, 2.0 ** -8)
    assert bool((out[R:] == 9.0).all())


def test_ragged_gemm_long_contraction_malformed_offsets(cuda_lib):
    """Segments past the rows count nothing and are reported; no cluster waits."""
    mx = cuda_lib
    gen = torch.Generator().manual_seed(5)
    a, w = _bf16((48, 2056), gen), _bf16((3, 264, 2056), gen)
    out = torch.full((48, 264), 9.0, dtype=torch.bfloat16, device="cuda")
    mx.mx_ragged_gemm(a, w, torch.tensor([20, 10, 48], dtype=torch.int32).cuda(), out=out)
    assert mx.mx_get_device_status() == "MX_ERR_OFFSETS"
    ref, mag = _ragged_ref(a[:20], w, [20], False)
    _check(out[:20], ref, mag, 2056, 2.0 ** -8)
    assert bool((out[20:] == 9.0).all())


@pytest.mark.parametrize("act,bias,res,ckpt", [("NONE", False, False, False), ("SILU", True, True, False),
                                               ("GELU_TANH", True, False, True)])
@pytest.mark.parametrize("N,K", [(8, 8), (136, 1000), (544, 328), (96, 4104)])
@pytest.mark.parametrize("M", [7, 8, 9, 15, 16, 17, 23, 24, 31, 32, 33])
def test_linear_few_rows(cuda_lib, M, N, K, act, bias, res, ckpt):
    mx = cuda_lib
    act = getattr(mx, "ACT_" + act)
    gen = torch.Generator().manual_seed(M + N + K)
    buf = _bf16((M + 2, K + 8), gen)
    buf[M:] = float("nan")
    x, w = buf[:M, :K], _bf16((N, K), gen, K ** -0.5)
    b = _bf16((N,), gen) if bias else None
    r = _bf16((M, N), gen) if res else None
    ck = mx.MX(M, N) if ckpt and N % 32 == 0 else None
    out = torch.full((M + 2, N), 9.0, dtype=torch.bfloat16, device="cuda")
    mx.mx_linear_fwd(x, w, b, act, r, out=out[:M], ckpt=ck)
    assert mx.mx_get_device_status() == "MX_OK"
    z = x.double() @ w.double().T
    mag = x.double().abs() @ w.double().abs().T
    if bias:
        z, mag = z + b.double(), mag + b.double().abs()
    h = _act(z, act, mx)
    ref = h + r.double() if res else h
    _check(out[:M], ref, 1.13 * mag + h.abs() * (2.0 ** 5 / K) + (r.double().abs() / K if res else 0), K, 2.0 ** -8)
    assert bool((out[M:] == 9.0).all())
    if ck is not None:
        rows = torch.arange(M, device="cuda").unsqueeze(1)
        cols = torch.arange(N // 32, device="cuda").unsqueeze(0)
        at = (rows // 128 * ((N + 127) // 128) + cols // 4) * 512 + rows % 32 * 16 + rows % 128 // 32 * 4 + cols % 4
        scale = torch.exp2(ck.scale[at].double() - 127).repeat_interleave(32, 1)
        off = (ck.data.view(torch.float8_e4m3fn).double() * scale - z).abs()
        assert bool((off <= 2.0 ** -4 * z.abs() + 2.0 ** -10 * scale + K * 2.0 ** -22 * mag).all())


@pytest.mark.parametrize("counts", [[9, 0, 3, 1], [1] * 8, [0, 17, 0, 0, 0, 0, 0, 3], [4, 4, 4, 4]])
def test_ragged_gemm_few_rows_of_few_experts(cuda_lib, counts):
    mx = cuda_lib
    R, G, N, K = sum(counts), len(counts), 200, 1160
    gen = torch.Generator().manual_seed(R + G)
    a, w = _bf16((R, K), gen), _bf16((G, N, K), gen, K ** -0.5)
    out = mx.mx_ragged_gemm(a, w, _offsets(counts))
    assert mx.mx_get_device_status() == "MX_OK"
    ref, mag = _ragged_ref(a, w, counts, False)
    _check(out, ref, mag, K, 2.0 ** -8)


def test_products_on_two_streams_at_once(cuda_lib):
    """Kernels that hand out their own tiles, share clusters or start early give
    the same bits beside one another as alone."""
    mx = cuda_lib
    gen = torch.Generator().manual_seed(17)
    G, K, N = 24, 520, 776
    counts = [(37 * g * g) % 211 for g in range(G)]
    R, off = sum(counts), _offsets([(37 * g * g) % 211 for g in range(G)])
    a, w, dy = _bf16((R, K), gen), _bf16((G, N, K), gen), _bf16((R, N), gen)
    x, lw = _bf16((120, 4104), gen), _bf16((512, 4104), gen)
    few = _bf16((13, 4104), gen)

    def calls():
        y = mx.mx_ragged_gemm(a, w, off)
        return (y, mx.mx_ragged_gemm(y, w, off, layout=mx.W_KN), mx.mx_ragged_gemm_wgrad(dy, a, G, off),
                mx.mx_ragged_gemm_wgrad_f32(dy, a, G, off, torch.zeros((G, N, K), device="cuda"), accumulate=True),
                mx.mx_linear_fwd(x, lw, act=mx.ACT_SILU), mx.mx_linear_fwd(few, lw))

    want = calls()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(8):
        for s, g in zip(streams, got):
            with torch.cuda.stream(s):
                g.append(calls())
    torch.cuda.synchronize()
    assert mx.mx_get_device_status() == "MX_OK"
    for outs in got[0] + got[1]:
        for u, v in zip(outs, want):
            assert torch.equal(u, v)
