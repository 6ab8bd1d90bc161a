"""Refusals of the layer norm, the expert routing, the combine's gradient and
the 4-bit tensors: malformed calls return a status and a message that names the
argument, before any device work (no GPU: the pointers are never dereferenced)."""
import ctypes

import pytest

FAKE, ODD, WORD = 0x10000, 0x10002, 0x10004


@pytest.fixture(scope="module")
def mx():
    from mlp_gemms_gb300 import build
    build.build()
    import mlp_gemms_gb300 as m
    m.load()
    return m


def _say(mx, st):
    return mx.STATUS[st], mx.mx_last_error()


def _call(mx, name, args, kw):
    bad = set(kw) - set(args)
    assert not bad, bad
    return _say(mx, getattr(mx.load(), name)(*{**args, **kw}.values()))


NORM = dict(x=FAKE, x_type=0, R=10, D=64, ld_x=64, res=None, ld_res=0, sum=None, ld_sum=0, weight=FAKE, bias=FAKE,
            w_type=0, eps=1e-5, rms=0, y=FAKE, ld_y=64, mean=FAKE, rstd=FAKE, stream=None)
NORM_BWD = dict(dy=FAKE, ld_dy=64, x=FAKE, x_type=0, R=10, D=64, ld_x=64, mean=FAKE, rstd=FAKE, weight=FAKE, w_type=0,
                rms=0, dres=None, ld_dres=0, dx=FAKE, ld_dx=64, dweight=FAKE, dbias=FAKE, accumulate=0, ws=FAKE,
                nbytes=1 << 30, stream=None)
TOPK = dict(logits=FAKE, x_type=0, T=10, G=64, ld=64, k=4, score=0, bias=None, groups=1, topk_groups=1, group_top=1,
            renorm=1, scale=1.0, weights=FAKE, ids=FAKE, load=None, score_sum=None, ws=None, nbytes=0, stream=None)
TOPK_BWD = dict(logits=FAKE, x_type=0, T=10, G=64, ld=64, k=4, score=0, renorm=1, scale=1.0, ids=FAKE, dweights=FAKE,
                dsum=None, dlogits=FAKE, ld_d=64, stream=None)
COMBINE = dict(dout=FAKE, T=10, D=64, inp=FAKE, R=128, row_of=FAKE, k=2, weights=FAKE, src=FAKE, din=FAKE + 64,
               dweights=FAKE, stream=None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(x=None), "MX_ERR_INVALID_ARG", "x is NULL"),
    (dict(x=ODD), "MX_ERR_ALIGNMENT", "x must"),
    (dict(y=None), "MX_ERR_INVALID_ARG", "y is NULL"),
    (dict(x_type=2), "MX_ERR_INVALID_ARG", "x_type"),
    (dict(w_type=-1), "MX_ERR_INVALID_ARG", "w_type"),
    (dict(R=-1), "MX_ERR_SHAPE", "R ="),
    (dict(R=1 << 31), "MX_ERR_SHAPE", "R ="),
    (dict(D=0), "MX_ERR_SHAPE", "D ="),
    (dict(D=60), "MX_ERR_SHAPE", "D ="),
    (dict(D=16392, ld_x=16392, ld_y=16392), "MX_ERR_NOT_SUPPORTED", "D ="),
    (dict(ld_x=56), "MX_ERR_ALIGNMENT", "ld of x"),
    (dict(ld_x=68), "MX_ERR_ALIGNMENT", "ld of x"),
    (dict(ld_y=60), "MX_ERR_ALIGNMENT", "ld of y"),
    (dict(weight=ODD), "MX_ERR_ALIGNMENT", "weight"),
    (dict(bias=ODD), "MX_ERR_ALIGNMENT", "bias"),
    (dict(eps=-1.0), "MX_ERR_INVALID_ARG", "eps"),
    (dict(eps=float("nan")), "MX_ERR_INVALID_ARG", "eps"),
    (dict(rms=2), "MX_ERR_INVALID_ARG", "rms"),
    (dict(mean=ODD), "MX_ERR_ALIGNMENT", "mean"),
    (dict(rstd=ODD), "MX_ERR_ALIGNMENT", "rstd"),
    (dict(res=FAKE, ld_res=64), "MX_ERR_ALIGNMENT", "ld of sum"),
    (dict(res=FAKE, ld_res=64, ld_sum=64), "MX_ERR_INVALID_ARG", "sum is NULL"),
    (dict(res=FAKE, ld_res=32, sum=FAKE + 64, ld_sum=64), "MX_ERR_ALIGNMENT", "ld of res"),
    (dict(res=FAKE + 64, ld_res=64, sum=FAKE, ld_sum=72), "MX_ERR_ALIGNMENT", "row stride"),
    (dict(R=(1 << 31) - 1, ld_x=1 << 20), "MX_ERR_SHAPE", "too large"),
], ids=str)
def test_norm(mx, kw, status, word):
    st, msg = _call(mx, "mx_layernorm_fwd", NORM, kw)
    assert st == status and word in msg, (st, msg)


@pytest.mark.parametrize("kw,status,word", [
    (dict(dy=None), "MX_ERR_INVALID_ARG", "dy is NULL"),
    (dict(x=ODD), "MX_ERR_ALIGNMENT", "x must"),
    (dict(dx=None), "MX_ERR_INVALID_ARG", "dx is NULL"),
    (dict(mean=None), "MX_ERR_INVALID_ARG", "mean or rstd"),
    (dict(rstd=None), "MX_ERR_INVALID_ARG", "mean or rstd"),
    (dict(rms=1, rstd=None), "MX_ERR_INVALID_ARG", "rstd"),
    (dict(accumulate=2), "MX_ERR_INVALID_ARG", "accumulate"),
    (dict(dres=FAKE, ld_dres=60), "MX_ERR_ALIGNMENT", "ld of dres"),
    (dict(dres=FAKE, ld_dres=72), "MX_ERR_ALIGNMENT", "row stride"),
    (dict(ld_dy=32), "MX_ERR_ALIGNMENT", "ld of dy"),
    (dict(dweight=ODD), "MX_ERR_ALIGNMENT", "dweight"),
    (dict(dbias=ODD), "MX_ERR_ALIGNMENT", "dbias"),
    (dict(ws=None), "MX_ERR_WORKSPACE", "workspace"),
    (dict(nbytes=16), "MX_ERR_WORKSPACE", "workspace"),
    (dict(ws=FAKE + 8), "MX_ERR_ALIGNMENT", "workspace"),
    (dict(D=16392, ld_x=16392, ld_dy=16392, ld_dx=16392), "MX_ERR_NOT_SUPPORTED", "D ="),
], ids=str)
def test_norm_backward(mx, kw, status, word):
    st, msg = _call(mx, "mx_layernorm_bwd", NORM_BWD, kw)
    assert st == status and word in msg, (st, msg)


ROUTE = [
    (dict(logits=None), "MX_ERR_INVALID_ARG", "logits"),
    (dict(logits=WORD), "MX_ERR_ALIGNMENT", "logits"),
    (dict(x_type=3), "MX_ERR_INVALID_ARG", "x_type"),
    (dict(score=2), "MX_ERR_INVALID_ARG", "score"),
    (dict(renorm=-1), "MX_ERR_INVALID_ARG", "renorm"),
    (dict(scale=float("inf")), "MX_ERR_INVALID_ARG", "scale"),
    (dict(G=0), "MX_ERR_INVALID_ARG", "G ="),
    (dict(G=1025, ld=1025, ld_d=1025), "MX_ERR_NOT_SUPPORTED", "G ="),
    (dict(k=0), "MX_ERR_INVALID_ARG", "k ="),
    (dict(k=65), "MX_ERR_INVALID_ARG", "k ="),
    (dict(k=33), "MX_ERR_NOT_SUPPORTED", "k ="),
    (dict(T=-1), "MX_ERR_SHAPE", "T ="),
    (dict(T=1 << 30), "MX_ERR_SHAPE", "T ="),
    (dict(ld=63), "MX_ERR_SHAPE", "ld ="),
    (dict(ids=None), "MX_ERR_INVALID_ARG", "ids"),
]


@pytest.mark.parametrize("kw,status,word", ROUTE + [
    (dict(weights=None), "MX_ERR_INVALID_ARG", "weights"),
    (dict(bias=ODD), "MX_ERR_ALIGNMENT", "bias"),
    (dict(groups=0), "MX_ERR_INVALID_ARG", "groups"),
    (dict(groups=5), "MX_ERR_INVALID_ARG", "groups"),
    (dict(groups=64), "MX_ERR_INVALID_ARG", "groups"),
    (dict(groups=4, topk_groups=5), "MX_ERR_INVALID_ARG", "topk_groups"),
    (dict(groups=4, topk_groups=0), "MX_ERR_INVALID_ARG", "topk_groups"),
    (dict(groups=32, topk_groups=1), "MX_ERR_INVALID_ARG", "choices from"),
    (dict(groups=4, topk_groups=2, group_top=3), "MX_ERR_INVALID_ARG", "group_top"),
    (dict(G=32, groups=32, topk_groups=8, group_top=2), "MX_ERR_INVALID_ARG", "group_top"),
    (dict(load=FAKE), "MX_ERR_INVALID_ARG", "together"),
    (dict(load=FAKE, score_sum=FAKE), "MX_ERR_WORKSPACE", "workspace"),
    (dict(load=FAKE, score_sum=FAKE, ws=FAKE + 8, nbytes=1 << 30), "MX_ERR_ALIGNMENT", "workspace"),
    (dict(load=ODD, score_sum=FAKE, ws=FAKE, nbytes=1 << 30), "MX_ERR_ALIGNMENT", "load"),
], ids=str)
def test_topk(mx, kw, status, word):
    kw = {n: v for n, v in kw.items() if n != "ld_d"}
    st, msg = _call(mx, "mx_moe_topk", TOPK, kw)
    assert st == status and word in msg, (st, msg)


@pytest.mark.parametrize("kw,status,word", ROUTE + [
    (dict(dweights=None), "MX_ERR_INVALID_ARG", "dweights"),
    (dict(dlogits=None), "MX_ERR_INVALID_ARG", "dlogits"),
    (dict(ld_d=32), "MX_ERR_SHAPE", "dlogits"),
    (dict(ld_d=72), "MX_ERR_ALIGNMENT", "row stride"),
    (dict(dsum=ODD), "MX_ERR_ALIGNMENT", "dscore_sum"),
], ids=str)
def test_topk_backward(mx, kw, status, word):
    st, msg = _call(mx, "mx_moe_topk_bwd", TOPK_BWD, kw)
    assert st == status and word in msg, (st, msg)


@pytest.mark.parametrize("kw,status,word", [
    (dict(dout=None), "MX_ERR_INVALID_ARG", "dout"),
    (dict(inp=None), "MX_ERR_INVALID_ARG", "in is NULL"),
    (dict(din=ODD), "MX_ERR_ALIGNMENT", "din"),
    (dict(din=FAKE), "MX_ERR_INVALID_ARG", "din is in"),
    (dict(row_of=None), "MX_ERR_INVALID_ARG", "row_of"),
    (dict(weights=ODD), "MX_ERR_ALIGNMENT", "weights"),
    (dict(dweights=ODD), "MX_ERR_ALIGNMENT", "dweights"),
    (dict(src=ODD), "MX_ERR_ALIGNMENT", "src"),
    (dict(k=0), "MX_ERR_INVALID_ARG", "k ="),
    (dict(D=60), "MX_ERR_SHAPE", "D ="),
    (dict(T=-1), "MX_ERR_SHAPE", "T ="),
    (dict(R=-1), "MX_ERR_SHAPE", "R ="),
    (dict(T=1 << 30, k=4), "MX_ERR_SHAPE", "T ="),
], ids=str)
def test_combine_backward(mx, kw, status, word):
    st, msg = _call(mx, "mx_moe_unpermute_bwd", COMBINE, kw)
    assert st == status and word in msg, (st, msg)


def _t(mx, rows, cols, data=FAKE, scale=FAKE, row=FAKE):
    return mx.Nvfp4Struct(data, scale, row, rows, cols)


@pytest.mark.parametrize("kw,status,word", [
    (dict(x=None), "MX_ERR_INVALID_ARG", "x is NULL"),
    (dict(K=48, ld=48, cols=48), "MX_ERR_SHAPE", "K ="),
    (dict(K=32800, ld=32800, cols=32800), "MX_ERR_NOT_SUPPORTED", "K ="),
    (dict(ld=32), "MX_ERR_ALIGNMENT", "ld of x"),
    (dict(rows=11), "MX_ERR_SHAPE", "out is"),
    (dict(cols=96), "MX_ERR_SHAPE", "out is"),
    (dict(row=None), "MX_ERR_INVALID_ARG", "out"),
    (dict(data=ODD), "MX_ERR_ALIGNMENT", "out"),
    (dict(src=ODD), "MX_ERR_ALIGNMENT", "src"),
    (dict(offsets=FAKE, G=0), "MX_ERR_INVALID_ARG", "G ="),
    (dict(src=FAKE, rows=1 << 20, ws=FAKE, nbytes=16), "MX_ERR_WORKSPACE", "workspace"),
    (dict(ws=FAKE + 8, nbytes=1 << 30), "MX_ERR_ALIGNMENT", "workspace"),
    (dict(T=-1), "MX_ERR_SHAPE", "T ="),
], ids=str)
def test_nvfp4_quantize(mx, kw, status, word):
    a = dict(x=FAKE, T=10, K=64, ld=64, src=None, offsets=None, G=0, ws=None, nbytes=0, rows=10, cols=64, data=FAKE,
             scale=FAKE, row=FAKE)
    assert set(kw) <= set(a)
    a.update(kw)
    out = _t(mx, a["rows"], a["cols"], a["data"], a["scale"], a["row"])
    st, msg = _say(mx, mx.load().mx_nvfp4_quantize(a["x"], a["T"], a["K"], a["ld"], a["src"], a["offsets"], a["G"],
                                                   ctypes.byref(out), a["ws"], a["nbytes"], None))
    assert st == status and word in msg, (st, msg)


@pytest.mark.parametrize("kw,status,word", [
    (dict(a=(10, 64, None)), "MX_ERR_INVALID_ARG", "a is NULL"),
    (dict(b=(64, 64, FAKE, ODD)), "MX_ERR_ALIGNMENT", "b must"),
    (dict(a=(10, 48)), "MX_ERR_SHAPE", "a has"),
    (dict(a=(10, 96)), "MX_ERR_SHAPE", "a has K"),
    (dict(b=(60, 64)), "MX_ERR_SHAPE", "N ="),
    (dict(b=(130, 64), G=4), "MX_ERR_SHAPE", "multiple of G"),
    (dict(b=(256, 64), G=4, a=(128, 64), offsets=FAKE), "MX_ERR_SHAPE", "N ="),
    (dict(b=(256, 64), G=2), "MX_ERR_INVALID_ARG", "offsets"),
    (dict(offsets=FAKE, ld=64), "MX_ERR_SHAPE", "R ="),
    (dict(G=0), "MX_ERR_INVALID_ARG", "G ="),
    (dict(G=1025), "MX_ERR_NOT_SUPPORTED", "G ="),
    (dict(out=None), "MX_ERR_INVALID_ARG", "out"),
    (dict(ld=60), "MX_ERR_ALIGNMENT", "ld of out"),
], ids=str)
def test_nvfp4_gemm(mx, kw, status, word):
    a = dict(a=(10, 64), b=(64, 64), G=1, offsets=None, out=FAKE, ld=128)
    a.update(kw)
    ta, tb = _t(mx, *a["a"]), _t(mx, *a["b"])
    st, msg = _say(mx, mx.load().mx_nvfp4_gemm(ctypes.byref(ta), ctypes.byref(tb), a["G"], a["offsets"], a["out"], a["ld"],
                                               None))
    assert st == status and word in msg, (st, msg)


def test_row_scales_are_optional_for_operands_only(mx):
    """(A device is needed from here on; without one the call says so.)"""
    ta, tb = _t(mx, 0, 64, None, None, None), _t(mx, 64, 64, row=None)
    assert mx.load().mx_nvfp4_gemm(ctypes.byref(ta), ctypes.byref(tb), 1, None, None, 64, None) == 0  # no rows


def test_nothing_to_do_needs_no_device(mx):
    for name, args, kw in (("mx_layernorm_fwd", NORM, dict(R=0, x=None, y=None)),
                           ("mx_layernorm_bwd", NORM_BWD, dict(R=0, dy=None, x=None, dx=None, accumulate=1)),
                           ("mx_moe_topk", TOPK, dict(T=0, logits=None, weights=None, ids=None)),
                           ("mx_moe_topk_bwd", TOPK_BWD, dict(T=0, logits=None, ids=None, dweights=None, dlogits=None)),
                           ("mx_moe_unpermute_bwd", COMBINE, dict(T=0, R=0, dout=None, inp=None, din=None, row_of=None))):
        assert _call(mx, name, args, kw)[0] == "MX_OK", name


def test_workspace_sizes(mx):
    L = mx.load()
    for R, D in ((1, 8), (333, 8192), (65536, 2048), (100000, 16384)):
        need = L.mx_layernorm_workspace_bytes(R, D)
        assert need >= 8 * D and need <= 152 * 8 * D
        st, msg = _call(mx, "mx_layernorm_bwd", NORM_BWD, dict(R=R, D=D, ld_x=D, ld_dy=D, ld_dx=D, nbytes=need - 1))
        assert st == "MX_ERR_WORKSPACE" and str(need) in msg
    for args in ((0, 8), (-1, 8), (8, 0), (8, 1 << 20)):
        assert L.mx_layernorm_workspace_bytes(*args) == 0
    assert L.mx_moe_topk_workspace_bytes(0, 8) == 0 and L.mx_moe_topk_workspace_bytes(100, 64) >= 64 * 8
    assert L.mx_nvfp4_scale_bytes(1, 32) == 512 and L.mx_nvfp4_scale_bytes(129, 96) == 2 * 2 * 512
    assert L.mx_nvfp4_quantize_workspace_bytes(8192, 2048, 8192) == 0       # each row for itself
    assert L.mx_nvfp4_quantize_workspace_bytes(8192, 2048, 65536) >= 8192 * (1024 + 128 + 4)
