"""Token counts, strides and gradients whose products pass 64 bits are refused by the
routing, the permute and the products (no GPU: the pointers are never dereferenced)."""
import ctypes

import pytest

FAKE = 0x10000


@pytest.fixture(scope="module")
def mx():
    from mlp_gemms_gb300 import build
    build.build()
    import mlp_gemms_gb300 as m
    m.load()
    return m


def _shape(mx, st):
    assert mx.STATUS[st] == "MX_ERR_SHAPE", (mx.STATUS[st], mx.mx_last_error())


def _t(mx, rows, cols):
    return ctypes.byref(mx.MxTensorStruct(FAKE, FAKE, rows, cols, mx.E4M3, 0))


@pytest.mark.parametrize("T,k", [(1 << 31, 1), (1 << 62, 4), (1 << 61, 8), ((1 << 62) + 5, 4)])
def test_routing(mx, T, k):
    L = mx.load()
    _shape(mx, L.mx_moe_route_index_pad(FAKE, T, k, 8, 128, FAKE, FAKE, (1 << 31) - 128, FAKE, FAKE, 1 << 40, None))
    _shape(mx, L.mx_moe_unpermute(FAKE, 128, 64, FAKE, None, T, k, FAKE, None))


@pytest.mark.parametrize("R,D", [(1 << 60, 1 << 10), (1 << 32, 1 << 32)])
def test_unpermuted_rows(mx, R, D):
    _shape(mx, mx.load().mx_moe_unpermute(FAKE, R, D, FAKE, None, 4, 2, FAKE, None))


@pytest.mark.parametrize("T,ld", [(1 << 60, 1 << 10), (1 << 30, 1 << 34), (1 << 20, 1 << 62)])
def test_permuted_tokens(mx, T, ld):
    _shape(mx, mx.load().mx_permute_quantize(FAKE, T, 128, ld, FAKE, 128, None, 0, mx.E4M3, mx.ROWWISE, _t(mx, 128, 128),
                                             None, None))


@pytest.mark.parametrize("ld", [1 << 57, (1 << 62) + 128])
def test_output_strides(mx, ld):
    a, b = _t(mx, 128, 128), _t(mx, 256, 128)
    for call in (mx.load().mx_grouped_gemm, mx.load().mx_grouped_gemm_2sm):
        _shape(mx, call(a, b, 1, None, FAKE, ld, None))


def test_weight_gradients(mx):
    a, b = _t(mx, 1 << 30, 128), _t(mx, 1 << 30, 128)
    _shape(mx, mx.load().mx_grouped_gemm_wgrad(a, b, 16, FAKE, FAKE, None))
