"""Refusals of the BF16 layers' entry points: malformed calls return a status
and a message that names the argument, before any device work (no GPU: the
pointers are never dereferenced)."""
import ctypes

import pytest

FAKE, ODD = 0x10000, 0x10008


@pytest.fixture(scope="module")
def mx():
    from mlp_gemms_gb300 import build
    build.build()
    import mlp_gemms_gb300 as m
    m.load()
    return m


def _t(rows, cols, fmt=0, had=0, data=FAKE, scale=FAKE):
    from mlp_gemms_gb300 import MxTensorStruct
    return MxTensorStruct(data, scale, rows, cols, fmt, had)


def _say(mx, st):
    return mx.STATUS[st], mx.mx_last_error()


def _gemm(mx, a=FAKE, R=10, K=64, ld_a=64, w=FAKE, N=64, G=2, layout=0, offsets=FAKE, out=FAKE, ld_out=64):
    return _say(mx, mx.load().mx_ragged_gemm(a, R, K, ld_a, w, N, G, layout, offsets, out, ld_out, None))


@pytest.mark.parametrize("kw,status,word", [
    (dict(a=None), "MX_ERR_INVALID_ARG", "a is NULL"),
    (dict(a=ODD), "MX_ERR_ALIGNMENT", "a must"),
    (dict(w=None), "MX_ERR_INVALID_ARG", "w is NULL"),
    (dict(w=ODD), "MX_ERR_ALIGNMENT", "w must"),
    (dict(out=None), "MX_ERR_INVALID_ARG", "out is NULL"),
    (dict(out=ODD), "MX_ERR_ALIGNMENT", "out must"),
    (dict(K=60, ld_a=64), "MX_ERR_SHAPE", "K ="),
    (dict(K=0), "MX_ERR_SHAPE", "K ="),
    (dict(N=63), "MX_ERR_SHAPE", "N ="),
    (dict(N=-8), "MX_ERR_SHAPE", "N ="),
    (dict(ld_a=56), "MX_ERR_ALIGNMENT", "ld of a"),
    (dict(ld_a=68), "MX_ERR_ALIGNMENT", "ld of a"),
    (dict(ld_out=56), "MX_ERR_ALIGNMENT", "ld of out"),
    (dict(layout=2), "MX_ERR_INVALID_ARG", "w_layout"),
    (dict(G=0), "MX_ERR_INVALID_ARG", "G ="),
    (dict(G=1025), "MX_ERR_NOT_SUPPORTED", "G ="),
    (dict(R=-1), "MX_ERR_SHAPE", "R ="),
    (dict(R=1 << 31), "MX_ERR_SHAPE", "R ="),
    (dict(offsets=None), "MX_ERR_INVALID_ARG", "offsets"),
    (dict(offsets=FAKE + 2), "MX_ERR_ALIGNMENT", "offsets"),
    (dict(R=(1 << 31) - 8, ld_a=1 << 20), "MX_ERR_SHAPE", "too large"),
    (dict(ld_a=1 << 40), "MX_ERR_SHAPE", "too large"),
    (dict(N=(1 << 31) - 8, ld_out=1 << 31), "MX_ERR_SHAPE", "too large"),
], ids=str)
def test_ragged_gemm_refusals(mx, kw, status, word):
    st, msg = _gemm(mx, **kw)
    assert st == status and word in msg, (st, msg)


def test_no_rows_needs_no_device(mx):
    assert _gemm(mx, R=0, a=None, out=None)[0] == "MX_OK"
    assert mx.load().mx_linear_fwd(None, 0, 64, 64, FAKE, 64, None, 2, None, 0, None, 64, None, None) == 0


def _wgrad(mx, dy=FAKE, N=64, ld_dy=64, x=FAKE, K=64, ld_x=64, R=10, G=2, offsets=FAKE, grad=FAKE, acc=None,
           ws=FAKE, ws_bytes=1 << 40):
    L = mx.load()
    if acc is None:
        st = L.mx_ragged_gemm_wgrad(dy, N, ld_dy, x, K, ld_x, R, G, offsets, grad, ws, ws_bytes, None)
    else:
        st = L.mx_ragged_gemm_wgrad_f32(dy, N, ld_dy, x, K, ld_x, R, G, offsets, grad, acc, ws, ws_bytes, None)
    return _say(mx, st)


@pytest.mark.parametrize("kw,status,word", [
    (dict(dy=None), "MX_ERR_INVALID_ARG", "dy"),
    (dict(x=ODD), "MX_ERR_ALIGNMENT", "x must"),
    (dict(grad=None), "MX_ERR_INVALID_ARG", "grad"),
    (dict(grad=ODD, acc=0), "MX_ERR_ALIGNMENT", "grad"),
    (dict(N=4), "MX_ERR_SHAPE", "N ="),
    (dict(K=12), "MX_ERR_SHAPE", "K ="),
    (dict(ld_dy=32), "MX_ERR_ALIGNMENT", "ld of dy"),
    (dict(ld_x=66), "MX_ERR_ALIGNMENT", "ld of x"),
    (dict(acc=2), "MX_ERR_INVALID_ARG", "accumulate"),
    (dict(G=2, offsets=None), "MX_ERR_INVALID_ARG", "offsets"),
    (dict(G=4096), "MX_ERR_NOT_SUPPORTED", "G ="),
    (dict(ws=ODD), "MX_ERR_ALIGNMENT", "workspace"),
], ids=str)
def test_ragged_wgrad_refusals(mx, kw, status, word):
    st, msg = _wgrad(mx, **kw)
    assert st == status and word in msg, (st, msg)


def test_ragged_wgrad_workspace(mx):
    """A missing or short workspace is refused where one is needed."""
    for N, K, R, G in [(64, 64, 10, 2), (1536, 2048, 65536, 128), (512, 512, 100000, 1)]:
        need = mx.mx_ragged_gemm_wgrad_workspace_bytes(N, K, R, G)
        if need:
            for ws, nb in ((None, 0), (FAKE, need - 1)):
                st, msg = _wgrad(mx, N=N, ld_dy=N, K=K, ld_x=K, R=R, G=G, ws=ws, ws_bytes=nb)
                assert st == "MX_ERR_WORKSPACE" and str(need) in msg


def _linear(mx, x=FAKE, M=10, K=64, ld_x=64, w=FAKE, N=64, bias=None, act=1, res=None, ld_res=0, out=FAKE + 64,
            ld_out=64, ckpt=None):
    st = mx.load().mx_linear_fwd(x, M, K, ld_x, w, N, bias, act, res, ld_res, out, ld_out,
                                 ctypes.byref(ckpt) if ckpt is not None else None, None)
    return _say(mx, st)


@pytest.mark.parametrize("kw,status,word", [
    (dict(x=None), "MX_ERR_INVALID_ARG", "x is NULL"),
    (dict(w=ODD), "MX_ERR_ALIGNMENT", "w must"),
    (dict(bias=ODD), "MX_ERR_ALIGNMENT", "bias"),
    (dict(act=0), "MX_ERR_NOT_SUPPORTED", "SwiGLU"),
    (dict(act=5), "MX_ERR_INVALID_ARG", "activation"),
    (dict(act=-1), "MX_ERR_INVALID_ARG", "activation"),
    (dict(res=FAKE, ld_res=32), "MX_ERR_ALIGNMENT", "ld of res"),
    (dict(res=ODD, ld_res=64), "MX_ERR_ALIGNMENT", "res"),
    (dict(res=FAKE + 64, ld_res=72), "MX_ERR_ALIGNMENT", "row stride"),
    (dict(M=-5), "MX_ERR_SHAPE", "M ="),
    (dict(N=40, ckpt=_t(10, 40)), "MX_ERR_SHAPE", "N ="),
    (dict(ckpt=_t(9, 64)), "MX_ERR_SHAPE", "ckpt"),
    (dict(ckpt=_t(10, 64, fmt=2)), "MX_ERR_INVALID_ARG", "E4M3"),
    (dict(ckpt=_t(10, 64, had=1)), "MX_ERR_INVALID_ARG", "rotation"),
    (dict(ckpt=_t(10, 64, data=None)), "MX_ERR_INVALID_ARG", "ckpt data"),
    (dict(ckpt=_t(10, 64, scale=ODD)), "MX_ERR_ALIGNMENT", "ckpt scale"),
], ids=lambda v: str(v)[:40])
def test_linear_refusals(mx, kw, status, word):
    st, msg = _linear(mx, **kw)
    assert st == status and word in msg, (st, msg)


def _save(mx, z=FAKE, R=10, C=64, ld_z=64, act=1, h=FAKE, ld_h=64, ckpt=None):
    ckpt = ckpt if ckpt is not None else _t(R, C)
    return _say(mx, mx.load().mx_act_ckpt_fwd(z, R, C, ld_z, act, h, ld_h, ctypes.byref(ckpt), None))


def _bwd(mx, ckpt=None, act=1, dh=FAKE, ld_dh=64, dz=FAKE, ld_dz=64, h=None, ld_h=0, db=None, ws=None, nb=0):
    ckpt = ckpt if ckpt is not None else _t(10, 64)
    return _say(mx, mx.load().mx_act_ckpt_bwd(ctypes.byref(ckpt), act, dh, ld_dh, dz, ld_dz, h, ld_h, db, ws, nb,
                                              None))


@pytest.mark.parametrize("kw,status,word", [
    (dict(z=None), "MX_ERR_INVALID_ARG", "z is NULL"),
    (dict(h=ODD), "MX_ERR_ALIGNMENT", "h must"),
    (dict(act=2), "MX_ERR_NOT_SUPPORTED", "identity"),
    (dict(act=9), "MX_ERR_INVALID_ARG", "activation"),
    (dict(C=48, ld_z=48, ld_h=48), "MX_ERR_SHAPE", "C ="),
    (dict(C=96, ld_z=96, ld_h=96, act=0), "MX_ERR_SHAPE", "C ="),
    (dict(ld_z=32), "MX_ERR_ALIGNMENT", "ld of z"),
    (dict(ld_h=60), "MX_ERR_ALIGNMENT", "ld of h"),
    (dict(R=-1), "MX_ERR_SHAPE", "R ="),
    (dict(ckpt=_t(11, 64)), "MX_ERR_SHAPE", "ckpt"),
    (dict(ckpt=_t(10, 64, fmt=1)), "MX_ERR_INVALID_ARG", "E4M3"),
], ids=lambda v: str(v)[:40])
def test_save_refusals(mx, kw, status, word):
    st, msg = _save(mx, **kw)
    assert st == status and word in msg, (st, msg)


@pytest.mark.parametrize("kw,status,word", [
    (dict(dh=None), "MX_ERR_INVALID_ARG", "dh is NULL"),
    (dict(dz=ODD), "MX_ERR_ALIGNMENT", "dz must"),
    (dict(ld_dz=32), "MX_ERR_ALIGNMENT", "ld of dz"),
    (dict(h=ODD, ld_h=64), "MX_ERR_ALIGNMENT", "h must"),
    (dict(h=FAKE, ld_h=8), "MX_ERR_ALIGNMENT", "ld of h"),
    (dict(act=2), "MX_ERR_NOT_SUPPORTED", "identity"),
    (dict(ckpt=_t(10, 32), act=0), "MX_ERR_SHAPE", "C ="),
    (dict(ckpt=_t(10, 64, data=ODD)), "MX_ERR_ALIGNMENT", "ckpt data"),
    (dict(ckpt=_t(5000, 64), db=FAKE), "MX_ERR_WORKSPACE", "workspace"),
    (dict(db=FAKE, ws=ODD, nb=1 << 30), "MX_ERR_ALIGNMENT", "workspace"),
    (dict(db=ODD, ws=FAKE, nb=1 << 30), "MX_ERR_ALIGNMENT", "db"),
], ids=lambda v: str(v)[:40])
def test_backward_refusals(mx, kw, status, word):
    st, msg = _bwd(mx, **kw)
    assert st == status and word in msg, (st, msg)


def test_the_training_step_takes_its_own_activations_only(mx):
    for act in (2, 3, 4):
        a = mx.MlpArgsStruct()
        a.act, a.G, a.R, a.D, a.F = act, 1, 128, 128, 128
        assert _say(mx, mx.load().mx_mlp_fwd_bwd(ctypes.byref(a), None))[0] == "MX_ERR_INVALID_ARG"
