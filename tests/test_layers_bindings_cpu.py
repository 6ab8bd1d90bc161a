"""The bindings of the layers around the expert MLP: what they refuse before the
library sees a pointer, and whose memory their own allocations are (no GPU:
torch's allocator and the launches are stand-ins)."""
import inspect

import pytest
import torch

from test_bf16_bindings_cpu import At, _b, _f, _i, mx  # noqa: F401
from test_binding_streams_cpu import MAIN, SIDE, Stream, Tensor, world  # noqa: F401

BF = torch.bfloat16


def _ints(*shape, where=0):
    return At(torch.zeros(shape, dtype=torch.int32), where)


def _fp4(m, rows, cols, where=0):
    n = m.nvfp4_scale_bytes(rows, cols)
    return m.NVFP4(rows, cols, data=At(torch.zeros((rows, cols // 2), dtype=torch.uint8), where),
                   scale=At(torch.zeros(n, dtype=torch.uint8), where), row_scale=_f(rows, where=where))


def _ws(n=1 << 22, where=0):
    return At(torch.zeros(n, dtype=torch.uint8), where)


# name: (ordinary arguments, as functions of the GPU they are on)
ARGS = {
    "mx_layernorm_fwd": dict(x=lambda w: _b(40, 64, where=w), weight=lambda w: _b(64, where=w), bias=lambda w: _b(64, where=w),
                             residual=lambda w: _b(40, 64, where=w), out=lambda w: _b(40, 64, where=w),
                             sum_out=lambda w: _b(40, 64, where=w), mean=lambda w: _f(40, where=w),
                             rstd=lambda w: _f(40, where=w)),
    "mx_layernorm_bwd": dict(dy=lambda w: _b(40, 64, where=w), x=lambda w: _b(40, 64, where=w), mean=lambda w: _f(40, where=w),
                             rstd=lambda w: _f(40, where=w), weight=lambda w: _b(64, where=w),
                             dres=lambda w: _b(40, 64, where=w), dx=lambda w: _b(40, 64, where=w),
                             dweight=lambda w: _f(64, where=w), dbias=lambda w: _f(64, where=w), workspace=lambda w: _ws(where=w)),
    "mx_moe_topk": dict(logits=lambda w: _b(40, 64, where=w), bias=lambda w: _f(64, where=w), weights=lambda w: _f(40, 4, where=w),
                        ids=lambda w: _ints(40, 4, where=w), load=lambda w: _ints(64, where=w),
                        score_sum=lambda w: _f(64, where=w), workspace=lambda w: _ws(where=w)),
    "mx_moe_topk_bwd": dict(logits=lambda w: _b(40, 64, where=w), ids=lambda w: _ints(40, 4, where=w),
                            dweights=lambda w: _f(40, 4, where=w), dscore_sum=lambda w: _f(64, where=w),
                            dlogits=lambda w: _b(40, 64, where=w)),
    "mx_moe_unpermute_bwd": dict(dout=lambda w: _b(40, 64, where=w), inp=lambda w: _b(256, 64, where=w),
                                 row_of=lambda w: _ints(40, 4, where=w), weights=lambda w: _f(40, 4, where=w),
                                 src=lambda w: _ints(256, where=w), din=lambda w: _b(256, 64, where=w),
                                 dweights=lambda w: _f(40, 4, where=w)),
    "mx_nvfp4_quantize": dict(x=lambda w: _b(40, 64, where=w), src=lambda w: _ints(256, where=w),
                              offsets=lambda w: _i(128, 256, where=w), workspace=lambda w: _ws(where=w)),
    "mx_nvfp4_gemm": dict(offsets=lambda w: _i(128, 256, where=w), out=lambda w: _b(256, 128, where=w)),
}
FIXED = {"mx_moe_topk": dict(k=4), "mx_nvfp4_gemm": dict(G=2)}


def _call(m, name, **kw):
    args = {n: f(0) for n, f in ARGS[name].items()}
    if name == "mx_nvfp4_quantize":
        args["out"] = _fp4(m, 256, 64)
    if name == "mx_nvfp4_gemm":
        args["a"], args["b"] = _fp4(m, 256, 64), _fp4(m, 256, 64)
    return getattr(m, name)(**{**args, **FIXED.get(name, {}), **kw})


@pytest.mark.parametrize("name", list(ARGS))
def test_ordinary_arguments_pass(mx, name):  # noqa: F811
    _call(mx, name)


@pytest.mark.parametrize("where", [-1, 1], ids=["host", "other gpu"])
@pytest.mark.parametrize("name,arg", [(n, a) for n, args in ARGS.items() for a in args])
def test_tensors_elsewhere(mx, name, arg, where):  # noqa: F811
    with pytest.raises(AssertionError):
        _call(mx, name, **{arg: ARGS[name][arg](where)})


@pytest.mark.parametrize("name", list(ARGS))
def test_another_gpu_than_the_current_one(mx, name, monkeypatch):  # noqa: F811
    monkeypatch.setattr(mx, "_current", (lambda d: 0, lambda: 1))
    with pytest.raises(AssertionError):
        _call(mx, name)


def _strided(t):
    return At(torch.stack((t.t, t.t), -1)[..., 0])


@pytest.mark.parametrize("name,arg", [(n, a) for n, args in ARGS.items() for a in args])
def test_strided_tensors(mx, name, arg):  # noqa: F811
    """Every tensor has dense rows, tables and vectors are dense as a whole."""
    with pytest.raises(AssertionError):
        _call(mx, name, **{arg: _strided(ARGS[name][arg](0))})


@pytest.mark.parametrize("name,arg", [(n, a) for n, args in ARGS.items() for a in args if a != "workspace"])
def test_other_types_and_shapes(mx, name, arg):  # noqa: F811
    good = ARGS[name][arg](0)
    main = list(ARGS[name])[0] == arg or arg in ("x", "weight", "bias") and "norm" in name
    if not main:  # the first tensor's type is free (BF16 or fp32), a norm's weights' too
        with pytest.raises(AssertionError):
            _call(mx, name, **{arg: At(good.t.to(torch.float16 if good.t.is_floating_point() else torch.int64))})
    if arg != "src" or name != "mx_nvfp4_quantize":
        with pytest.raises((AssertionError, ValueError)):
            _call(mx, name, **{arg: At(good.t.reshape(-1)[:-8].reshape(1, -1))})


def test_half_precision_is_refused(mx):  # noqa: F811
    h = At(torch.zeros((40, 64), dtype=torch.float16))
    for call in (lambda: mx.mx_layernorm_fwd(h), lambda: mx.mx_moe_topk(h, 4), lambda: mx.mx_nvfp4_quantize(h),
                 lambda: mx.mx_layernorm_fwd(_b(40, 64), At(torch.zeros(64, dtype=torch.float16)))):
        with pytest.raises(AssertionError):
            call()


def test_types_that_go_together(mx):  # noqa: F811
    x32 = _f(40, 64)
    mx.mx_layernorm_fwd(x32, _f(64), _f(64), residual=_f(40, 64))
    with pytest.raises(AssertionError):
        mx.mx_layernorm_fwd(x32, _f(64), _b(64))
    with pytest.raises(AssertionError):
        mx.mx_layernorm_fwd(x32, residual=_b(40, 64))
    with pytest.raises(AssertionError):
        mx.mx_layernorm_fwd(_b(40, 64), sum_out=_b(40, 64))
    with pytest.raises(AssertionError):
        mx.mx_layernorm_fwd(_b(40, 64), rms=True, mean=_f(40))
    with pytest.raises(AssertionError):
        mx.mx_layernorm_bwd(_b(40, 64), x32, _f(40), _f(40), accumulate=True)
    with pytest.raises(AssertionError):
        mx.mx_layernorm_bwd(_b(40, 64), x32, _f(40), _f(40), dres=_b(40, 64))


@pytest.mark.parametrize("bad", ["codes", "strided codes", "scales", "rows", "host"])
def test_four_bit_buffers(mx, bad):  # noqa: F811
    def broken():
        t = _fp4(mx, 256, 64)
        if bad == "codes":
            t.data = At(t.data.t[:-1])
        elif bad == "strided codes":
            t.data = At(torch.zeros((256, 64), dtype=torch.uint8)[:, ::2])
        elif bad == "scales":
            t.scale = At(t.scale.t[:-1])
        elif bad == "rows":
            t.row_scale = At(t.row_scale.t[:-1])
        else:
            t.scale = At(t.scale.t, -1)
        return t

    for call in (lambda: _call(mx, "mx_nvfp4_gemm", a=broken()), lambda: _call(mx, "mx_nvfp4_gemm", b=broken()),
                 lambda: _call(mx, "mx_nvfp4_quantize", out=broken())):
        with pytest.raises(AssertionError):
            call()


def test_the_namespace(mx):  # noqa: F811
    from mlp_gemms_gb300 import layers
    for name, f in vars(layers).items():
        if name.startswith("mx_"):
            assert getattr(mx, name) is f
    assert mx.NVFP4 is layers.NVFP4
    with pytest.raises(AttributeError):
        mx.mx_no_such_call
    with pytest.raises(AttributeError):
        mx.no_such_name


# ---------------------------------------------------------------- allocations

def _t(*shape, dtype=BF):
    return Tensor(torch.zeros(shape, dtype=dtype))


def _w4(m):
    n = m.nvfp4_scale_bytes(64, 64)
    return m.NVFP4(64, 64, data=_t(64, 32, dtype=torch.uint8), scale=_t(n, dtype=torch.uint8), row_scale=_t(64, dtype=torch.float32))


CALLS = {  # name: (its own allocations, the call)
    "mx_layernorm_fwd": (4, lambda m, s: m.mx_layernorm_fwd(_t(40, 64), residual=_t(40, 64), stream=s)),
    "mx_layernorm_bwd": (4, lambda m, s: m.mx_layernorm_bwd(_t(40, 64), _t(40, 64), _t(40, dtype=torch.float32),
                                                            _t(40, dtype=torch.float32), stream=s)),
    "mx_moe_topk": (5, lambda m, s: m.mx_moe_topk(_t(40, 64), 4, stats=True, stream=s)),
    "mx_moe_topk_bwd": (1, lambda m, s: m.mx_moe_topk_bwd(_t(40, 64), _t(40, 4, dtype=torch.int32),
                                                          _t(40, 4, dtype=torch.float32), stream=s)),
    "mx_moe_unpermute_bwd": (2, lambda m, s: m.mx_moe_unpermute_bwd(_t(40, 64), _t(128, 64), _t(40, 2, dtype=torch.int32),
                                                                    stream=s)),
    "mx_nvfp4_quantize": (2, lambda m, s: m.mx_nvfp4_quantize(_t(64, 32768), src=_t(1024, dtype=torch.int32), stream=s)),
    "mx_nvfp4_gemm": (1, lambda m, s: m.mx_nvfp4_gemm(_w4(m), _w4(m), stream=s)),
}


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("stream,owner", [(None, MAIN), (Stream(MAIN), MAIN), (Stream(SIDE), SIDE)],
                         ids=["default", "current", "another"])
def test_whose_memory(world, name, stream, owner):  # noqa: F811
    m, made, _, _ = world
    count, call = CALLS[name]
    call(m, stream)
    assert len(made) == count
    for t in made:
        assert t.owner == owner and t.marks == ([] if owner == MAIN else [MAIN])


def test_every_binding_with_a_stream_is_covered():
    from mlp_gemms_gb300 import layers
    takes = {n for n, f in vars(layers).items() if n.startswith("mx_") and "stream" in inspect.signature(f).parameters}
    assert takes == set(CALLS) == set(ARGS)
