"""Sizes whose products pass 64 bits are refused like any others that are too
large: a wrapped product would pass the limit and launch (no GPU: the pointers
are never dereferenced)."""
import pytest

from test_layers_api_cpu import COMBINE, NORM, NORM_BWD, TOPK, TOPK_BWD, _call, mx  # noqa: F401


@pytest.mark.parametrize("k", [1, 4, 32])
@pytest.mark.parametrize("T", [1 << 31, 1 << 59, 1 << 62])
def test_tokens(mx, T, k):  # noqa: F811
    for name, args in (("mx_moe_topk", TOPK), ("mx_moe_topk_bwd", TOPK_BWD), ("mx_moe_unpermute_bwd", COMBINE)):
        st, msg = _call(mx, name, args, dict(T=T, k=k))
        assert st == "MX_ERR_SHAPE" and "T =" in msg, (name, st, msg)


@pytest.mark.parametrize("rows,ld", [(1 << 30, 1 << 34), (1 << 26, (1 << 38) - 64), (1 << 28, 1 << 35), (1 << 27, 1 << 37)])
def test_rows_times_stride(mx, rows, ld):  # noqa: F811
    for name, args, stride, word in (("mx_layernorm_fwd", NORM, "ld_x", "x is too"), ("mx_layernorm_fwd", NORM, "ld_y", "y is too"),
                                     ("mx_layernorm_bwd", NORM_BWD, "ld_dx", "dx is too"),
                                     ("mx_moe_topk", TOPK, "ld", "ld ="), ("mx_moe_topk_bwd", TOPK_BWD, "ld_d", "dlogits")):
        kw = {("R" if "R" in args else "T"): rows, stride: ld}
        if "k" in args:
            kw["k"] = 1
        st, msg = _call(mx, name, args, kw)
        assert st == "MX_ERR_SHAPE" and word in msg, (name, stride, st, msg)


def test_the_largest_that_fit_are_not_refused(mx):  # noqa: F811
    """Up to the first check behind the sizes."""
    st, msg = _call(mx, "mx_moe_topk", TOPK, dict(T=1 << 20, ld=(1 << 26) - 1, logits=0x10004))
    assert st == "MX_ERR_ALIGNMENT" and "logits" in msg
    st, msg = _call(mx, "mx_layernorm_fwd", NORM, dict(R=1 << 20, ld_x=(1 << 26) - 8, x=0x10004))
    assert st == "MX_ERR_ALIGNMENT" and "x must" in msg
