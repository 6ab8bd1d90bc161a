"""What the BF16 layers' bindings refuse before the library sees a pointer: the
C layer cannot tell a strided table from a dense one, nor whose memory a
pointer is (no GPU: launches are stand-ins)."""
import pytest
import torch

from test_binding_streams_cpu import Lib, Tensor


class At(Tensor):
    """A stand-in that says it is on GPU `where` (-1: the host)."""

    def __init__(self, t, where=0):
        super().__init__(t)
        self.where = where

    def get_device(self):
        return self.where


@pytest.fixture
def mx(monkeypatch):
    from mlp_gemms_gb300 import build
    build.build()
    import mlp_gemms_gb300 as m
    lib = Lib(m.load())
    empty = torch.empty
    monkeypatch.setattr(m, "load", lambda: lib)
    monkeypatch.setattr(m, "_current", (lambda d: 0, lambda: 0))
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: At(empty(*a, **{k: v for k, v in kw.items() if k != "device"})))
    return m


def _b(*shape, where=0):
    return At(torch.zeros(shape, dtype=torch.bfloat16), where)


def _f(*shape, where=0):
    return At(torch.zeros(shape), where)


def _i(*v, where=0):
    return At(torch.tensor(v, dtype=torch.int32), where)


def _ckpt(mx, rows, cols, where=0):
    return mx.MX(rows, cols, data=At(torch.zeros((rows, cols), dtype=torch.uint8), where),
                 scale=At(torch.zeros(mx.scale_bytes(rows, cols), dtype=torch.uint8), where))


STRIDED = At(torch.tensor([[8, 0], [40, 0]], dtype=torch.int32)[:, 0])


def _gemm(mx, **kw):
    a = dict(a=_b(40, 64), w=_b(2, 64, 64), offsets=_i(8, 40), out=_b(40, 64))
    return mx.mx_ragged_gemm(**{**a, **kw})


def _wgrad(mx, **kw):
    a = dict(dy=_b(9000, 64), x=_b(9000, 64), G=2, offsets=_i(8, 9000), out=_b(2, 64, 64))
    return mx.mx_ragged_gemm_wgrad(**{**a, **kw})


def _wgrad_f32(mx, **kw):
    a = dict(dy=_b(9000, 64), x=_b(9000, 64), G=2, offsets=_i(8, 9000), grad=_f(2, 64, 64))
    return mx.mx_ragged_gemm_wgrad_f32(**{**a, **kw})


def _linear(mx, **kw):
    a = dict(x=_b(40, 64), w=_b(64, 64), bias=_b(64), residual=_b(40, 64), out=_b(40, 64), ckpt=_ckpt(mx, 40, 64))
    return mx.mx_linear_fwd(**{**a, **kw})


def _save(mx, **kw):
    a = dict(z=_b(40, 64), act=mx.ACT_SILU, h=_b(40, 64), ckpt=_ckpt(mx, 40, 64))
    return mx.mx_act_ckpt_fwd(**{**a, **kw})


def _bwd(mx, **kw):
    a = dict(ckpt=_ckpt(mx, 600, 64), act=mx.ACT_SILU, dh=_b(600, 64), dz=_b(600, 64), h=_b(600, 64), db=_f(64),
             workspace=At(torch.zeros(1 << 20, dtype=torch.uint8)))
    return mx.mx_act_ckpt_bwd(**{**a, **kw})


@pytest.mark.parametrize("call", [_gemm, _wgrad, _wgrad_f32, _linear, _save, _bwd], ids=lambda f: f.__name__[1:])
def test_ordinary_arguments_pass(mx, call):
    call(mx)


@pytest.mark.parametrize("call", [_gemm, _wgrad, _wgrad_f32], ids=lambda f: f.__name__[1:])
def test_strided_offsets(mx, call):
    with pytest.raises(AssertionError):
        call(mx, offsets=STRIDED)


@pytest.mark.parametrize("call", [_wgrad, _wgrad_f32, _bwd], ids=lambda f: f.__name__[1:])
def test_strided_workspace(mx, call):
    with pytest.raises(AssertionError):
        call(mx, workspace=At(torch.zeros((1 << 20, 2), dtype=torch.uint8)[:, 0]))


@pytest.mark.parametrize("where", [-1, 1], ids=["host", "other gpu"])
@pytest.mark.parametrize("call,name,make", [
    (_gemm, "a", lambda w: _b(40, 64, where=w)), (_gemm, "w", lambda w: _b(2, 64, 64, where=w)),
    (_gemm, "offsets", lambda w: _i(8, 40, where=w)), (_gemm, "out", lambda w: _b(40, 64, where=w)),
    (_wgrad, "dy", lambda w: _b(9000, 64, where=w)), (_wgrad, "x", lambda w: _b(9000, 64, where=w)),
    (_wgrad, "offsets", lambda w: _i(8, 9000, where=w)), (_wgrad, "out", lambda w: _b(2, 64, 64, where=w)),
    (_wgrad, "workspace", lambda w: At(torch.zeros(1 << 20, dtype=torch.uint8), w)),
    (_wgrad_f32, "x", lambda w: _b(9000, 64, where=w)), (_wgrad_f32, "grad", lambda w: _f(2, 64, 64, where=w)),
    (_linear, "x", lambda w: _b(40, 64, where=w)), (_linear, "w", lambda w: _b(64, 64, where=w)),
    (_linear, "bias", lambda w: _b(64, where=w)), (_linear, "residual", lambda w: _b(40, 64, where=w)),
    (_linear, "out", lambda w: _b(40, 64, where=w)),
    (_save, "z", lambda w: _b(40, 64, where=w)), (_save, "h", lambda w: _b(40, 64, where=w)),
    (_bwd, "dh", lambda w: _b(600, 64, where=w)), (_bwd, "dz", lambda w: _b(600, 64, where=w)),
    (_bwd, "h", lambda w: _b(600, 64, where=w)), (_bwd, "db", lambda w: _f(64, where=w)),
    (_bwd, "workspace", lambda w: At(torch.zeros(1 << 20, dtype=torch.uint8), w)),
], ids=lambda v: v if isinstance(v, str) else getattr(v, "__name__", "")[1:])
def test_tensors_elsewhere(mx, call, name, make, where):
    with pytest.raises(AssertionError):
        call(mx, **{name: make(where)})


@pytest.mark.parametrize("call", [_gemm, _wgrad, _wgrad_f32], ids=lambda f: f.__name__[1:])
def test_everything_on_the_host(mx, call):
    t = dict(_gemm=dict(a=_b(40, 64, where=-1), w=_b(2, 64, 64, where=-1), offsets=_i(8, 40, where=-1), out=_b(40, 64, where=-1)),
             _wgrad=dict(dy=_b(9000, 64, where=-1), x=_b(9000, 64, where=-1), offsets=_i(8, 9000, where=-1),
                         out=_b(2, 64, 64, where=-1)),
             _wgrad_f32=dict(dy=_b(9000, 64, where=-1), x=_b(9000, 64, where=-1), offsets=_i(8, 9000, where=-1),
                             grad=_f(2, 64, 64, where=-1)))
    with pytest.raises(AssertionError):
        call(mx, **t[call.__name__])


BAD_CKPT = {
    "short payload": lambda d, s: (d[:-1], s),
    "strided payload": lambda d, s: (torch.zeros((d.shape[0], 2 * d.shape[1]), dtype=torch.uint8)[:, ::2], s),
    "short scales": lambda d, s: (d, s[:-1]),
    "strided scales": lambda d, s: (d, torch.zeros((s.numel(), 2), dtype=torch.uint8)[:, 0]),
    "payload on the host": lambda d, s: (At(d, -1), s),
    "scales on another gpu": lambda d, s: (d, At(s, 1)),
}


@pytest.mark.parametrize("bad", list(BAD_CKPT))
@pytest.mark.parametrize("call,rows", [(_linear, 40), (_save, 40), (_bwd, 600)], ids=["linear", "save", "bwd"])
def test_checkpoint_buffers(mx, call, rows, bad):
    """A checkpoint in the caller's own buffers: dense, as large as its shape
    needs, on the call's GPU (the kernels write and read all of it)."""
    data, scale = torch.zeros((rows, 64), dtype=torch.uint8), torch.zeros(mx.scale_bytes(rows, 64), dtype=torch.uint8)
    data, scale = (t if isinstance(t, At) else At(t) for t in BAD_CKPT[bad](data, scale))
    with pytest.raises(AssertionError):
        call(mx, ckpt=mx.MX(rows, 64, data=data, scale=scale))


def test_checkpoint_buffers_of_another_type(mx):
    """Bytes are what counts: a payload held as E4M3 values passes."""
    ck = _ckpt(mx, 40, 64)
    ck.data = At(ck.data.t.view(torch.float8_e4m3fn))
    _linear(mx, ckpt=ck)
