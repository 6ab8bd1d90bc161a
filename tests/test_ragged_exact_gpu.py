"""Weight gradients whose every partial sum is exact: operands in {-1, 0, 1}, so
each sum is a whole number below 2^24 however it is cut, ordered or truncated.
One lost, repeated or foreign row shows: fp32 results equal the whole numbers,
BF16 results their rounding.

Random data: the tensor core's fp32 accumulator truncates, up to 4096 rows at a
time, a drift of at most 2^-26 of the sum for each of 256 steps of 16 rows; the
2-norm error of a long sum stays below the 5e-6 stated for it.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _ternary(shape, gen):
    return torch.randint(-1, 2, shape, generator=gen, dtype=torch.int8).to(torch.bfloat16).cuda()


def _offsets(counts):
    return torch.tensor(np.cumsum(counts), dtype=torch.int32).cuda()


def _whole(dy, x, counts):
    """The gradients as whole numbers, from products in fp64."""
    out = torch.zeros((len(counts), dy.shape[1], x.shape[1]), dtype=torch.float64, device="cuda")
    b = 0
    for g, c in enumerate(counts):
        out[g] = dy[b:b + c].double().T @ x[b:b + c].double()
        b += c
    return out


# (segments, N, K, whether they are cut into parts that a second launch adds)
CASES = [
    ([30011], 520, 200, True), ([5000, 0, 17000, 3], 136, 264, True), ([9001], 64, 72, True),
    ([0, 12345, 0, 0], 264, 520, True), ([4097] * 4, 40, 264, True), ([65536 + 33], 64, 128, True),
    ([4095], 264, 264, True),
    # one pass, or several of 4096 rows over a tile (fp32)
    ([4096, 4097, 1, 8191, 8193, 63], 520, 520, False),
    ([12289, 0, 5000, 77], 1032, 776, False), ([(37 * i * i) % 331 for i in range(160)], 264, 136, False),
    ([1, 2, 3, 15, 16, 17, 31, 33, 47, 48, 49, 63, 64, 65, 127, 129], 136, 264, False),
]


@pytest.mark.parametrize("kind", ["bf16", "f32", "acc"])
@pytest.mark.parametrize("counts,N,K,parts", CASES, ids=lambda v: str(v)[:24])
def test_weight_gradient_is_exact(cuda_lib, counts, N, K, parts, kind):
    mx = cuda_lib
    R, G = sum(counts), len(counts)
    assert (mx.mx_ragged_gemm_wgrad_workspace_bytes(N, K, R, G) > 0) == parts
    gen = torch.Generator().manual_seed(R + N + K)
    dy, x = _ternary((R + 70, N), gen), _ternary((R + 70, K), gen)
    dy[R:], x[R:] = float("nan"), float("inf")
    off, want = _offsets(counts), _whole(dy, x, counts)
    if kind == "bf16":
        got = mx.mx_ragged_gemm_wgrad(dy, x, G, off)
        want = want.float().to(torch.bfloat16)
    else:
        got = torch.randint(-1000, 1000, (G, N, K), generator=gen).float().cuda()
        if kind == "acc":
            want = want + got.double()
        mx.mx_ragged_gemm_wgrad_f32(dy, x, G, off, got, accumulate=kind == "acc")
        want = want.float()
    assert mx.mx_get_device_status() == "MX_OK"
    assert torch.equal(got, want)


@pytest.mark.parametrize("counts,N,K,parts", [([65536], 64, 128, True), ([30011], 520, 200, True),
                                              ([4096], 1544, 1544, False), ([20000, 45000], 1032, 1032, False)],
                         ids=lambda v: str(v)[:24])
def test_long_sums_in_fp32(cuda_lib, counts, N, K, parts):
    mx = cuda_lib
    R, G = sum(counts), len(counts)
    assert (mx.mx_ragged_gemm_wgrad_workspace_bytes(N, K, R, G) > 0) == parts
    gen = torch.Generator().manual_seed(R)
    dy = torch.randn((R, N), generator=gen).to(torch.bfloat16).cuda()
    x = torch.randn((R, K), generator=gen).to(torch.bfloat16).cuda()
    got = mx.mx_ragged_gemm_wgrad_f32(dy, x, G, _offsets(counts), torch.empty((G, N, K), device="cuda")).double()
    want = _whole(dy, x, counts)
    for g in range(G):
        assert float((got[g] - want[g]).norm() / want[g].norm()) < 5e-6


@pytest.mark.parametrize("kn", [False, True], ids=["NK", "KN"])
@pytest.mark.parametrize("counts,N,K", [([33], 520, 2056), ([0, 7, 0, 50], 264, 3144), ([700], 1024, 4104),
                                        ([1, 0, 3], 200, 1160), ([127, 128, 129, 255, 256, 257, 1, 31, 33], 328, 520),
                                        ([(37 * i * i) % 331 for i in range(160)], 520, 136)],
                         ids=lambda v: str(v)[:24])
def test_product_is_exact(cuda_lib, counts, N, K, kn):
    """The products too, shared contractions, few rows and many tiles."""
    mx = cuda_lib
    R, G = sum(counts), len(counts)
    gen = torch.Generator().manual_seed(R + N + K)
    a = _ternary((R + 40, K), gen)
    a[R:] = float("nan")
    w = _ternary((G, K, N) if kn else (G, N, K), gen)
    out = mx.mx_ragged_gemm(a, w, _offsets(counts), layout=mx.W_KN if kn else mx.W_NK)
    assert mx.mx_get_device_status() == "MX_OK"
    b = 0
    for g, c in enumerate(counts):
        want = a[b:b + c].double() @ (w[g].double() if kn else w[g].double().T)
        assert torch.equal(out[b:b + c], want.float().to(torch.bfloat16))
        b += c
