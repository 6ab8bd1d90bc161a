"""Whose memory the bindings' own allocations are (no GPU: torch's allocator
and the launches are stand-ins).  A call on another stream than the current one
takes its workspace and results from that stream's memory and marks them as
used by the current one, so that neither stream's work reuses a block while the
other may still be busy with it."""
import contextlib

import pytest
import torch

MAIN, SIDE = "main", "side"


class Stream:
    def __init__(self, name):
        self.name, self.cuda_stream = name, 0

    def __eq__(self, other):
        return self.name == other.name


class Tensor:
    """A CPU tensor that says it is on a GPU, with its stream and marks."""

    def __init__(self, t, owner=MAIN):
        self.t, self.owner, self.marks = t, owner, []
        self.is_cuda, self.device = True, torch.device("cuda", 0)

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return 0

    def record_stream(self, s):
        self.marks.append(s.name)


class Lib:
    """The library, every launch replaced by a success."""

    def __init__(self, real):
        self.real = real

    def __getattr__(self, name):
        if name.endswith("_bytes") or "route_rows" in name:
            return getattr(self.real, name)
        return lambda *a: 0


@pytest.fixture
def world(monkeypatch):
    from mlp_gemms_gb300 import build
    build.build()
    import mlp_gemms_gb300 as mx
    lib = Lib(mx.load())
    monkeypatch.setattr(mx, "load", lambda: lib)
    monkeypatch.setattr(mx, "_current", (lambda d: 0, lambda: 0))
    current, made, empty = [Stream(MAIN)], [], torch.empty

    def fake_empty(*a, **kw):
        kw.pop("device", None)
        made.append(Tensor(empty(*a, **kw), current[-1].name))
        return made[-1]

    @contextlib.contextmanager
    def use(s):
        current.append(s)
        yield
        current.pop()

    monkeypatch.setattr(torch, "empty", fake_empty)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])

    def bf16(*shape):
        return Tensor(torch.zeros(shape, dtype=torch.bfloat16))

    def q(rows, cols, fmt=None):
        m = mx.MX(rows, cols, mx.E4M3 if fmt is None else fmt)
        m.data, m.scale = Tensor(m.data.t), Tensor(m.scale.t)
        return m

    return mx, made, bf16, q


def _i32(*v):
    return Tensor(torch.tensor(v, dtype=torch.int32))


def _f32(*shape):
    return Tensor(torch.zeros(shape))


CALLS = {
    "mx_ragged_gemm": (1, lambda mx, b, q, s: mx.mx_ragged_gemm(b(40, 64), b(2, 64, 64), _i32(8, 40), stream=s)),
    "mx_ragged_gemm_wgrad": (2, lambda mx, b, q, s: mx.mx_ragged_gemm_wgrad(b(9000, 64), b(9000, 64), 1, None, stream=s)),
    "mx_ragged_gemm_wgrad_f32": (1, lambda mx, b, q, s: mx.mx_ragged_gemm_wgrad_f32(b(9000, 64), b(9000, 64), 1, None,
                                                                          _f32(1, 64, 64), stream=s)),
    "mx_linear_fwd": (1, lambda mx, b, q, s: mx.mx_linear_fwd(b(40, 64), b(64, 64), stream=s)),
    "mx_act_ckpt_fwd": (3, lambda mx, b, q, s: mx.mx_act_ckpt_fwd(b(40, 64), mx.ACT_SILU, stream=s)),
    "mx_act_ckpt_bwd": (4, lambda mx, b, q, s: mx.mx_act_ckpt_bwd(q(600, 64), mx.ACT_SILU, b(600, 64), recompute=True,
                                                           colsum=True, stream=s)),
    "mx_quantize": (6, lambda mx, b, q, s: mx.mx_quantize(b(128, 128), colsum=True, stream=s)),
    "mx_quantize_sr": (4, lambda mx, b, q, s: mx.mx_quantize_sr(b(128, 128), mx.E2M1, 7, stream=s)),
    "mx_quantize_colsum_noalloc": (5, lambda mx, b, q, s: mx.mx_quantize_colsum_noalloc(b(128, 128), stream=s)),
    "mx_moe_route_index": (4, lambda mx, b, q, s: mx.mx_moe_route_index(Tensor(torch.zeros((8, 2), dtype=torch.int32)), 2,
                                                                 stream=s)),
    "mx_permute_quantize": (4, lambda mx, b, q, s: mx.mx_permute_quantize(b(8, 128), _i32(*range(128)), stream=s)),
    "mx_moe_unpermute": (1, lambda mx, b, q, s: mx.mx_moe_unpermute(b(128, 128), Tensor(torch.zeros((8, 2), dtype=torch.int32)),
                                                             stream=s)),
    "mx_grouped_gemm": (1, lambda mx, b, q, s: mx.mx_grouped_gemm(q(128, 128), q(128, 128), 1, _i32(128), stream=s)),
    "mx_grouped_gemm_2sm": (1, lambda mx, b, q, s: mx.mx_grouped_gemm_2sm(q(128, 128), q(128, 128), 1, _i32(128), stream=s)),
    "mx_grouped_gemm_bias": (1, lambda mx, b, q, s: mx.mx_grouped_gemm_bias(q(128, 128), q(128, 128), 1, _i32(128),
                                                                       b(1, 128), stream=s)),
    "mx_grouped_gemm_bias_2sm": (1, lambda mx, b, q, s: mx.mx_grouped_gemm_bias_2sm(q(128, 128), q(128, 128), 1, _i32(128),
                                                                               b(1, 128), stream=s)),
    "mx_grouped_gemm_swiglu_fwd": (5, lambda mx, b, q, s: mx.mx_grouped_gemm_swiglu_fwd(q(128, 128), q(256, 128), 1, _i32(128), stream=s)),
    "mx_grouped_gemm_swiglu_probs_fwd": (5, lambda mx, b, q, s: mx.mx_grouped_gemm_swiglu_probs_fwd(q(128, 128), q(256, 128), 1, _i32(128),
                                                                                  _f32(128), stream=s)),
    "mx_grouped_gemm_dswiglu_probs_bwd": (6, lambda mx, b, q, s: mx.mx_grouped_gemm_dswiglu_probs_bwd(
        q(128, 128), q(128, 128), b(128, 256), _f32(128), 1, _i32(128), stream=s)),
    "mx_grouped_gemm_dswiglu_bwd": (4, lambda mx, b, q, s: mx.mx_grouped_gemm_dswiglu_bwd(q(128, 128), q(128, 128), b(128, 256), 1,
                                                                        _i32(128), stream=s)),
    "mx_grouped_gemm_wgrad": (1, lambda mx, b, q, s: mx.mx_grouped_gemm_wgrad(q(128, 128), q(128, 128), 1, _i32(128), stream=s)),
    "mx_grouped_gemm_wgrad_ws": (2, lambda mx, b, q, s: mx.mx_grouped_gemm_wgrad_ws(q(128, 128), q(128, 128), 1, _i32(128), stream=s)),
    "mx_grouped_gemm_wgrad_f32_ws": (1, lambda mx, b, q, s: mx.mx_grouped_gemm_wgrad_f32_ws(q(128, 128), q(128, 128), 1, _i32(128),
                                                                          _f32(1, 128, 128), stream=s)),
    "mx_gemm_bias": (1, lambda mx, b, q, s: mx.mx_gemm_bias(q(128, 128), q(128, 128), stream=s)),
    "mx_gemm_gelu_fwd": (5, lambda mx, b, q, s: mx.mx_gemm_gelu_fwd(q(128, 128), q(128, 128), stream=s)),
    "mx_gemm_dgelu_bwd": (6, lambda mx, b, q, s: mx.mx_gemm_dgelu_bwd(q(128, 128), q(128, 128), b(128, 128), stream=s)),
}


def _allocations(world, name, stream):
    mx, made, bf16, q = world
    count, call = CALLS[name]
    fixed = {}

    def operand(*a):  # quantized operands are made before the call's own buffers
        m = q(*a)
        fixed.update({id(t): t for t in made})
        return m

    call(mx, bf16, operand, stream)
    own = [t for t in made if id(t) not in fixed]
    assert len(own) == count
    return own


@pytest.mark.parametrize("name", list(CALLS))
def test_another_stream(world, name):
    for t in _allocations(world, name, Stream(SIDE)):
        assert t.owner == SIDE and t.marks == [MAIN]


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("stream", [None, Stream(MAIN)], ids=["default", "current"])
def test_the_current_stream(world, name, stream):
    for t in _allocations(world, name, stream):
        assert t.owner == MAIN and t.marks == []


def test_every_binding_with_a_stream_is_covered():
    import inspect

    import mlp_gemms_gb300 as mx
    nothing = {"mx_grouped_gemm_wgrad_f32", "mx_mlp_fwd_bwd", "mx_get_device_status", "mx_selftest_bounded_wait"}
    takes = {n for n, f in vars(mx).items()
             if n.startswith("mx_") and inspect.isfunction(f) and "stream" in inspect.signature(f).parameters}
    assert takes - nothing == set(CALLS)
