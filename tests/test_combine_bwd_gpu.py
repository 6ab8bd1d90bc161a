"""The gradient of mx_moe_unpermute's weighted sum against the formula in 64 bits:
dropped choices, empty rows, one column piece to many, more choices than are
taken at a time.

Tolerances: din is one fp32 product rounded to BF16, bit for bit that of the
formula in fp32; dweights is a sum of D products, off by at most D / 64 + 16
roundings of 2^-24 of their magnitudes (a thread's values in turn, then trees;
bounded here by D / 8)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _case(mx, T, k, G, D, seed=0, drop=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn((T, G), device="cuda", generator=gen)
    w, ids, _, _ = mx.mx_moe_topk(logits, k)
    offsets, src, row_of = mx.mx_moe_route_index(ids, G)
    R = src.numel()
    if drop:
        src[row_of[::3, 0].long()] = -1
        row_of[::3, 0] = -1
    inp = torch.randn((R, D), device="cuda", generator=gen).to(BF)
    dout = torch.randn((T, D), device="cuda", generator=gen).to(BF)
    return dout, inp, row_of, w, src


def _ref(dout, inp, row_of, w):
    T, k = row_of.shape
    rows = row_of.long()
    there = rows >= 0
    din = torch.zeros(inp.shape, dtype=BF, device="cuda")
    value = (torch.ones_like(rows, dtype=torch.float32) if w is None else w).unsqueeze(2) * dout.float().unsqueeze(1)
    din[rows[there]] = value.to(BF)[there]
    x = inp.double()[rows.clamp(min=0)] * there.unsqueeze(2)
    d = dout.double().unsqueeze(1)
    return din, (d * x).sum(2), (d * x).abs().sum(2)


@pytest.mark.parametrize("drop", [False, True], ids=["all", "dropped"])
@pytest.mark.parametrize("T,k,G,D", [(1, 1, 1, 8), (3, 2, 4, 64), (61, 8, 128, 2048), (37, 6, 8, 1000), (20, 4, 16, 2056),
                                     (9, 8, 8, 8192), (5, 10, 16, 512), (7, 17, 32, 320), (3000, 2, 8, 128)])
def test_formula(cuda_lib, T, k, G, D, drop):
    dout, inp, row_of, w, src = _case(cuda_lib, T, k, G, D, drop=drop)
    for weights in (w, None):
        din, dw = cuda_lib.mx_moe_unpermute_bwd(dout, inp, row_of, weights, src=src)
        want, ref, mag = _ref(dout, inp, row_of, weights)
        assert torch.equal(din, want)
        assert ((dw.double() - ref).abs() <= (D / 8 + 16) * 2.0 ** -24 * mag).all()
        again = cuda_lib.mx_moe_unpermute_bwd(dout, inp, row_of, weights, src=src)
        assert torch.equal(again[0], din) and torch.equal(again[1], dw)
    assert cuda_lib.mx_get_device_status() == "MX_OK"


def test_rows_that_nothing_names_are_left_alone(cuda_lib):
    dout, inp, row_of, w, src = _case(cuda_lib, 10, 2, 4, 256)
    din = torch.full(inp.shape, 7.0, dtype=BF, device="cuda")
    cuda_lib.mx_moe_unpermute_bwd(dout, inp, row_of, w, din=din)
    named = torch.zeros(inp.shape[0], dtype=torch.bool, device="cuda")
    named[row_of.reshape(-1).long()] = True
    assert (din[~named] == 7).all() and torch.equal(din[named], _ref(dout, inp, row_of, w)[0][named])
    cuda_lib.mx_moe_unpermute_bwd(dout, inp, row_of, w, src=src, din=din)
    assert (din[~named] == 0).all()


def test_rows_out_of_range_are_reported(cuda_lib):
    dout, inp, row_of, w, src = _case(cuda_lib, 10, 2, 4, 256)
    row_of[4, 1] = inp.shape[0]
    din, dw = cuda_lib.mx_moe_unpermute_bwd(dout, inp, row_of, w, src=src)
    assert cuda_lib.mx_get_device_status() == "MX_ERR_INVALID_ARG"
    assert dw[4, 1] == 0 and cuda_lib.mx_get_device_status() == "MX_OK"


def test_non_finite_values_of_other_rows(cuda_lib):
    """What stands in rows that no choice names reaches no weight."""
    dout, inp, row_of, w, src = _case(cuda_lib, 10, 2, 4, 256)
    want = cuda_lib.mx_moe_unpermute_bwd(dout, inp, row_of, w, src=src)
    inp[src < 0] = float("nan")
    got = cuda_lib.mx_moe_unpermute_bwd(dout, inp, row_of, w, src=src)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_tokens(cuda_lib):
    inp = torch.zeros((128, 64), dtype=BF, device="cuda")
    din = torch.full((128, 64), 7.0, dtype=BF, device="cuda")
    src = torch.full((128,), -1, dtype=torch.int32, device="cuda")
    src[5] = 0
    _, dw = cuda_lib.mx_moe_unpermute_bwd(torch.empty((0, 64), dtype=BF, device="cuda"), inp,
                                          torch.empty((0, 2), dtype=torch.int32, device="cuda"), src=src, din=din)
    assert dw.shape == (0, 2) and (din[5] == 7).all() and int((din == 7).sum()) == 64


def test_the_combine_moves_by_its_gradient(cuda_lib):
    """mx_moe_unpermute is linear in the rows and in the weights: sum(c out) equals
    <din, in> and <dweights, w> up to the roundings (BF16 of out 2^-9, of din 2^-9 of the magnitudes)."""
    c, inp, row_of, w, src = _case(cuda_lib, 50, 4, 8, 512)
    out = cuda_lib.mx_moe_unpermute(inp, row_of, w)
    din, dw = cuda_lib.mx_moe_unpermute_bwd(c, inp, row_of, w, src=src)
    total = float((c.double() * out.double()).sum())
    size = float((c.double().abs() * cuda_lib.mx_moe_unpermute(inp.abs(), row_of, w).double()).sum())
    assert abs(total - float((din.double() * inp.double()).sum())) <= 2.0 ** -7 * size
    assert abs(total - float((dw.double() * w.double()).sum())) <= 2.0 ** -8 * size
