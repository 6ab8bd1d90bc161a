"""Expert routing against the definition in 64 bits (choices equal to the
index), its gradient against the formula by automatic differentiation in 64 bits
and against differences: both scores, biases, groups, closed experts, values
nearer to each other than fp32 can tell, odd sizes and strides.

Tolerances.  A score is exp of a difference (off by 2 max|x| roundings, exp itself
by 2 units = 4 roundings) over a sum of at most 32 + 5 of them; a weight is a
quotient of two: rel = 2 (2 max|x| + 48) 2^-24.  Sums over T tokens add T roundings.
Gradients: the same relative error of each product of factors."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F, D = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24
INF = math.inf


def _scores(x, sigmoid):
    if sigmoid:
        return torch.sigmoid(x)
    return torch.where(torch.isneginf(x).all(1, keepdim=True), torch.zeros_like(x), torch.softmax(x, 1))


def _first(v, n):
    """Indexes of the n largest of each row, the lowest of equal ones first."""
    return torch.sort(v, dim=1, descending=True, stable=True).indices[:, :n]


def _choose(x, k, sigmoid, bias, groups, topk_groups, group_top):
    """The definition: x the logits in 64 bits."""
    T, G = x.shape
    closed = torch.isneginf(x)
    s = _scores(x, sigmoid)
    v = x if bias is None else torch.where(closed, x, s + bias.to(D))
    if groups > topk_groups:
        u = (x if group_top == 1 else s.masked_fill(closed, -INF)) if bias is None else v
        value = torch.topk(u.view(T, groups, -1), group_top).values.sum(2)
        kept = torch.zeros((T, groups), dtype=torch.bool, device=x.device).scatter_(1, _first(value, topk_groups), True)
        v = v.masked_fill(~kept.repeat_interleave(G // groups, 1), -INF)
    return _first(v, k)


def _weights(x, ids, sigmoid, renorm, scale):
    w = _scores(x, sigmoid).gather(1, ids.long())
    if renorm:
        total = w.sum(1, keepdim=True)
        w = torch.where(total == 0, torch.zeros_like(w), w / total)
    return scale * w


def _rel(x):
    return 2 * (2 * float(x[x.isfinite()].abs().max()) + 48) * U if x.isfinite().any() else 100 * U


def _close(got, ref, bound, what):
    got = got.to(D)
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of the bound" % (
        what, int(bad.sum()), bad.numel(), float(((got - ref).abs() / bound).max()))


def _logits(T, G, dtype, seed, closed=False, pad=0, std=1.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = std * torch.randn((T, G), device="cuda", generator=gen) + 0.5 * torch.randn(G, device="cuda", generator=gen)
    if closed:
        x[torch.rand((T, G), device="cuda", generator=gen) < 0.3] = -INF
        if T > 2:
            x[T // 2] = -INF          # nothing open
            x[T // 3, 1:] = -INF      # one open expert
    buf = torch.full((T, G + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :G] = x.to(dtype)
    return buf[:, :G]


def _check(mx, x, k, sigmoid=False, bias=None, groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0):
    score = mx.SCORE_SIGMOID if sigmoid else mx.SCORE_SOFTMAX
    w, ids, load, total = mx.mx_moe_topk(x, k, score, bias, groups, topk_groups, group_top, renorm, scale, stats=True)
    w2, ids2, none, _ = mx.mx_moe_topk(x, k, score, bias, groups, topk_groups, group_top, renorm, scale)
    assert none is None and torch.equal(w, w2) and torch.equal(ids, ids2)
    d = x.to(D)
    want = _choose(d, k, sigmoid, bias, groups, topk_groups, group_top)
    assert torch.equal(ids.long(), want), "%d of %d choices" % (int((ids != want).sum()), ids.numel())
    ref = _weights(d, want, sigmoid, renorm, scale)
    rel = _rel(d)
    # exp of less than -87 leaves fp32's normal range
    _close(w, ref, rel * ref.abs() + (0 if renorm else 2.0 ** -125), "weights")
    assert torch.equal(load.long(), torch.bincount(want.reshape(-1), minlength=x.shape[1]))
    p = _scores(d, sigmoid)
    if sigmoid:
        n = p.sum(1, keepdim=True)
        p = torch.where(n == 0, torch.zeros_like(p), p / n)
    _close(total, p.sum(0), (rel + x.shape[0] * U) * p.sum(0) + 2.0 ** -120, "score sums")
    return w, ids


SIZES = [(1, 1, 1), (5, 2, 2), (7, 8, 2), (33, 31, 5), (64, 32, 32), (61, 60, 6), (129, 64, 8), (50, 100, 7),
         (1000, 128, 8), (13, 160, 6), (61, 256, 8), (40, 257, 3), (31, 384, 10), (17, 512, 8), (9, 1000, 4),
         (3, 1024, 31), (4, 1024, 32)]


@pytest.mark.parametrize("closed", [False, True], ids=["open", "closed"])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,G,k", SIZES)
def test_choices_and_weights(cuda_lib, T, G, k, dtype, sigmoid, closed):
    x = _logits(T, G, dtype, T + G, closed)
    _check(cuda_lib, x, k, sigmoid, scale=2.5)
    _check(cuda_lib, x, k, sigmoid, renorm=False)
    bias = 0.1 * torch.randn(G, device="cuda", generator=torch.Generator(device="cuda").manual_seed(G))
    _check(cuda_lib, x, k, sigmoid, bias)
    _check(cuda_lib, x, k, sigmoid, torch.zeros(G, device="cuda"))


@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("with_bias", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("T,G,k,groups,kept", [(61, 256, 8, 8, 4), (200, 64, 6, 4, 2), (33, 60, 3, 5, 2), (9, 96, 4, 32, 5),
                                               (17, 1024, 8, 16, 3), (40, 160, 6, 8, 3), (11, 48, 16, 3, 1),
                                               (20, 128, 8, 4, 4)])
def test_groups(cuda_lib, T, G, k, groups, kept, sigmoid, with_bias, group_top):
    for dtype, closed in ((F, False), (F, True), (BF, False)):
        x = _logits(T, G, dtype, G + groups, closed)
        if dtype == BF and not with_bias and group_top == 2 and not sigmoid:
            x = x + 0  # equal logits in different groups: equal values, by index
        bias = 0.1 * torch.randn(G, device="cuda", generator=torch.Generator(device="cuda").manual_seed(G)) if with_bias \
            else None
        _check(cuda_lib, x, k, sigmoid, bias, groups, kept, group_top)


@pytest.mark.parametrize("pad", [1, 4, 8])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_row_strides(cuda_lib, dtype, pad):
    for T, G in ((9, 128), (9, 100), (30, 256)):
        x = _logits(T, G, dtype, G, pad=pad)
        _check(cuda_lib, x, 6)
        w, ids, _, _ = cuda_lib.mx_moe_topk(x, 6)
        dw = torch.randn_like(w)
        out = torch.full((T, G + pad), 7.0, dtype=dtype, device="cuda")
        got = cuda_lib.mx_moe_topk_bwd(x, ids, dw, dlogits=out[:, :G])
        assert torch.equal(got, cuda_lib.mx_moe_topk_bwd(x.contiguous(), ids, dw)) and (out[:, G:] == 7).all()


@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_values_nearer_than_fp32(cuda_lib, sigmoid, groups):
    """Biases that cancel the scores up to a few 2^-27: the fp32 sums are all
    but equal, the order is that of the 64-bit ones."""
    T, G, k = 64, 128, 8
    x = _logits(T, G, F, 3, std=1.0)
    x[1::2] = x[0]                                    # one row's scores for all: its ties under the bias
    s = _scores(x.to(D), sigmoid)[0]
    gen = torch.Generator(device="cuda").manual_seed(11)
    bias = (0.75 - s).to(F) + (torch.randint(-3, 4, (G,), device="cuda", generator=gen) * 2.0 ** -26).to(F)
    _check(cuda_lib, x, k, sigmoid, bias, groups, max(1, groups // 2), 1 if groups == 1 else 2)


@pytest.mark.parametrize("G,groups", [(64, 1), (256, 1), (256, 8), (512, 4), (60, 1), (60, 5)])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_few_values_nearer_than_fp32(cuda_lib, sigmoid, G, groups):
    """Each expert of the first half has one in the second whose sum with its bias is
    equal up to a few 2^-27, the second's logit a little larger: pairs, and with
    groups the groups of a pair, are as near, all others far apart."""
    T, k = 64, 6
    half = G // 2 - (G // 2) % (G // groups) if groups > 1 else G // 2
    x = _logits(1, G, F, 9, std=1.0)
    x[:, half:2 * half] = x[:, :half] + 0.125
    s = _scores(x.to(D), sigmoid)[0]
    gen = torch.Generator(device="cuda").manual_seed(12)
    bias = 0.2 * torch.rand(G, device="cuda", generator=gen)
    bias[half:2 * half] = (bias[:half].to(D) + s[:half] - s[half:2 * half]).to(F)
    step = torch.randint(-3, 4, (T, G), device="cuda", generator=gen) * 2.0 ** -24
    for row in range(0, T, 16):
        b = (bias + step[row] * 0.25).to(F)
        _check(cuda_lib, x.expand(T, G).contiguous() + step, k, sigmoid, b, groups, (groups + 1) // 2, 1 if groups == 1 else 2)


@pytest.mark.parametrize("G", [64, 60])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_biases_that_cancel_in_a_group(cuda_lib, sigmoid, G):
    """Groups of two with biases of 100 and -100: their values are what is left of it."""
    bias = 100.0 - 200.0 * (torch.arange(G, device="cuda") % 2)
    _check(cuda_lib, _logits(2000, G, F, 4, std=0.3), 6, sigmoid, bias, G // 2, 5, 2)


def test_equal_logits_go_by_index(cuda_lib):
    x = torch.zeros((3, 96), dtype=BF, device="cuda")
    x[1, 40:50] = 2.0
    x[2, ::2] = -0.0
    for bias in (None, torch.full((96,), 0.25, device="cuda")):
        for sigmoid in (False, True):
            _, ids = _check(cuda_lib, x, 7, sigmoid, bias)
            assert ids[0].tolist() == list(range(7)) and ids[1].tolist() == list(range(40, 47))
            assert ids[2].tolist() == list(range(7))


def test_saturated_scores(cuda_lib):
    """Sigmoids that round to 1 or underflow: the order is still the logits'."""
    x = torch.linspace(-300, 300, 64, device="cuda").roll(17).repeat(2, 1)
    _, ids, _, _ = cuda_lib.mx_moe_topk(x, 8, cuda_lib.SCORE_SIGMOID)
    assert torch.equal(ids[0].long(), _first(x.to(D), 8)[0])
    x = x - 400                                           # every score 0 in fp32
    w, ids, _, total = cuda_lib.mx_moe_topk(x, 8, cuda_lib.SCORE_SIGMOID, stats=True)
    assert torch.equal(ids[0].long(), _first(x.to(D), 8)[0])
    assert torch.isfinite(w).all() and torch.isfinite(total).all()


@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("bias", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_non_finite_logits(cuda_lib, sigmoid, bias, groups):
    x = _logits(8, 64, F, 5)
    x[1, 7], x[3, 50], x[5] = float("nan"), INF, float("nan")
    b = torch.linspace(0, 0.1, 64, device="cuda") if bias else None
    w, ids, _, _ = cuda_lib.mx_moe_topk(x, 6, cuda_lib.SCORE_SIGMOID if sigmoid else cuda_lib.SCORE_SOFTMAX, b, groups,
                                        max(1, groups // 2), stats=True)
    assert ((ids >= 0) & (ids < 64)).all() and all(len(set(r)) == 6 for r in ids.tolist())
    assert torch.isnan(w[1]).all() and torch.isnan(w[5]).all() and (sigmoid or torch.isnan(w[3]).all())
    assert torch.isfinite(w[[0, 2, 4, 6, 7]]).all()


# ---------------------------------------------------------------- gradients

def _grad(x, ids, a, sigmoid, renorm, scale, v):
    """(gradient of sum(a w) + sum(v score_sum) by differentiation in 64 bits,
    magnitude of its terms); rows whose chosen scores are all 0 give 0."""
    open_ = ~torch.isneginf(x)
    leaf = torch.where(open_, x, torch.zeros_like(x)).requires_grad_(True)
    masked = torch.where(open_, leaf, torch.full_like(x, -INF))
    dead = ~open_.any(1, keepdim=True)
    safe = torch.where(dead, torch.zeros_like(masked), masked)
    p = (torch.sigmoid(safe) if sigmoid else torch.softmax(safe, 1)) * (~dead)
    there = ids >= 0
    c = p.gather(1, ids.clamp(min=0).long()) * there
    if renorm:
        total = c.sum(1, keepdim=True)
        w = c / torch.where(total == 0, torch.ones_like(total), total)
    else:
        w = c
    loss = (scale * w * a.to(D) * there).sum()
    if v is not None:
        n = p.sum(1, keepdim=True)
        loss = loss + (p / torch.where(n == 0, torch.ones_like(n), n) * v.to(D)).sum()
    g = torch.autograd.grad(loss, leaf)[0] * open_
    with torch.no_grad():
        b = (scale * a.to(D)).abs() * there
        mag = torch.zeros_like(p).scatter_add_(1, ids.clamp(min=0).long(), w * (b + ((b * w).sum(1, keepdim=True) if renorm else 0)))
        if not renorm and not sigmoid:
            mag = mag + p * (b * w).sum(1, keepdim=True)
        # With renorm the choices' parts sum to 0 and the other experts' gradient is
        # exactly 0; differentiation leaves its own roundings there, 2^-52 of p_e times
        # the summed parts each: 2^-24 of this.
        mag = mag + 2.0 ** -24 * p * (b * w).sum(1, keepdim=True)
        if v is not None:
            q = p / p.sum(1, keepdim=True).clamp(min=1e-300)
            mag = mag + q * (v.to(D).abs() + (q * v.to(D).abs()).sum(1, keepdim=True))
    return g, mag


@pytest.mark.parametrize("closed", [False, True], ids=["open", "closed"])
@pytest.mark.parametrize("renorm", [False, True], ids=["scores", "renorm"])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,G,k", SIZES)
def test_gradient(cuda_lib, T, G, k, dtype, sigmoid, renorm, closed):
    x = _logits(T, G, dtype, T + G, closed)
    score = cuda_lib.SCORE_SIGMOID if sigmoid else cuda_lib.SCORE_SOFTMAX
    _, ids, _, _ = cuda_lib.mx_moe_topk(x, k, score, renorm=renorm, scale=1.5)
    gen = torch.Generator(device="cuda").manual_seed(1)
    a, v = torch.randn((T, k), device="cuda", generator=gen), torch.randn(G, device="cuda", generator=gen)
    if T > 4:
        ids[1, 0] = -1                # dropped choices
        ids[3] = -1
    for dsum in (None, v):
        got = cuda_lib.mx_moe_topk_bwd(x, ids, a, score, renorm, 1.5, dscore_sum=dsum)
        ref, mag = _grad(x.to(D), ids, a, sigmoid, renorm, 1.5, dsum)
        out = 2.0 ** -8 if dtype == BF else U
        _close(got, ref, out * ref.abs() + (2 * _rel(x.to(D)) + (k + 40) * U) * mag + 2.0 ** -120, "dlogits")
        inplace = x.clone()
        assert torch.equal(cuda_lib.mx_moe_topk_bwd(inplace, ids, a, score, renorm, 1.5, dscore_sum=dsum, dlogits=inplace), got)
    assert cuda_lib.mx_get_device_status() == "MX_OK"


def test_gradient_against_differences(cuda_lib):
    """Weights of an unchanged choice and the score sums move by dlogits along a
    direction: fp32, central differences with a step of 2^-6 (third derivatives of
    order one: 2^-12 of the sum of magnitudes), weights off by 2^-18."""
    for sigmoid in (False, True):
        score = cuda_lib.SCORE_SIGMOID if sigmoid else cuda_lib.SCORE_SOFTMAX
        x = torch.sort(torch.randn((6, 16), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)),
                       1, descending=True).values
        x[:, :4] += 1.0               # a gap behind the four chosen: the step changes no choice
        gen = torch.Generator(device="cuda").manual_seed(3)
        a, v = torch.randn((6, 4), device="cuda", generator=gen), torch.randn(16, device="cuda", generator=gen)
        to = torch.randn((6, 16), device="cuda", generator=gen)
        h = 2.0 ** -6

        def f(x):
            w, ids, _, total = cuda_lib.mx_moe_topk(x, 4, score, stats=True)
            w = torch.zeros((6, 16), dtype=D, device="cuda").scatter_(1, ids.long(), w.to(D))  # by expert: steps may reorder
            return float((w[:, :4] * a.to(D)).sum() + (total.to(D) * v.to(D)).sum())

        _, ids, _, _ = cuda_lib.mx_moe_topk(x, 4, score)
        assert torch.equal(ids.sort(1).values, torch.arange(4, device="cuda", dtype=torch.int32).expand(6, 4))
        dx = cuda_lib.mx_moe_topk_bwd(x, ids, a.gather(1, ids.long()), score, dscore_sum=v)
        moved = (f(x + h * to) - f(x - h * to)) / (2 * h)
        size = float((a.abs().sum() + v.abs().sum() * 6) * to.abs().max() ** 3)
        assert abs(float((dx.to(D) * to.to(D)).sum()) - moved) <= size * (2.0 ** -12 + 2.0 ** -18 / h)


def test_ids_out_of_range_are_reported(cuda_lib):
    x = _logits(4, 32, F, 0)
    _, ids, _, _ = cuda_lib.mx_moe_topk(x, 3)
    a = torch.randn((4, 3), device="cuda")
    bad = ids.clone()
    bad[1, 2], bad[2, 0] = 32, -5
    gone = ids.clone()
    gone[1, 2], gone[2, 0] = -1, -1
    got = cuda_lib.mx_moe_topk_bwd(x, bad, a)
    assert cuda_lib.mx_get_device_status() == "MX_ERR_INVALID_ARG"
    assert torch.equal(got, cuda_lib.mx_moe_topk_bwd(x, gone, a))
    assert cuda_lib.mx_get_device_status() == "MX_OK"


def test_the_same_expert_twice(cuda_lib):
    """Not what the forward pass gives; both parts are added."""
    x = _logits(2, 16, F, 0)
    ids = torch.tensor([[3, 3], [5, 1]], dtype=torch.int32, device="cuda")
    a = torch.randn((2, 2), device="cuda")
    got = cuda_lib.mx_moe_topk_bwd(x, ids, a, renorm=False)
    ref, mag = _grad(x.to(D), ids, a, False, False, 1.0, None)
    _close(got, ref, 100 * U * mag, "dlogits")


def test_no_tokens(cuda_lib):
    x = torch.empty((0, 64), device="cuda")
    w, ids, load, total = cuda_lib.mx_moe_topk(x, 4, stats=True)
    assert w.shape == (0, 4) and (load == 0).all() and (total == 0).all()
    assert cuda_lib.mx_moe_topk_bwd(x, ids, w).shape == (0, 64)


def test_many_tokens_and_graphs(cuda_lib):
    """More tokens than one wave of warps, on two streams, and replayed from a graph."""
    T, G, k = 20011, 128, 8
    xs = [_logits(T, G, BF, i) for i in range(2)]
    bias = 0.05 * torch.randn(G, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0))
    a = torch.randn((T, k), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))

    def call(x, stream=None):
        w, ids, load, total = cuda_lib.mx_moe_topk(x, k, cuda_lib.SCORE_SIGMOID, bias, 8, 4, 2, stats=True, stream=stream)
        return w, ids, load, total, cuda_lib.mx_moe_topk_bwd(x, ids, a, cuda_lib.SCORE_SIGMOID, dscore_sum=bias,
                                                             stream=stream)

    for x in xs:
        _check(cuda_lib, x, k, True, bias, 8, 4, 2)
    want = [call(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(10):
        got = [call(x, s) for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(g, w))
    x = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(x)
    for i in (1, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want[i]))
