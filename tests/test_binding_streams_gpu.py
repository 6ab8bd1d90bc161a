"""Calls that launch on another stream than the current one while both streams
are busy: neither the workspaces that the bindings allocate nor their results
share a block with the current stream's work."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _bf16(shape, gen):
    return torch.randn(shape, generator=gen).to(torch.bfloat16).cuda()


def _flat(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if isinstance(t, torch.Tensor)]


def _calls(mx):
    gen = torch.Generator().manual_seed(2)
    R, N, K = 30011, 264, 264
    dy, x = _bf16((R, N), gen), _bf16((R, K), gen)
    z = _bf16((2000, 1088), gen)
    _, ck = mx.mx_act_ckpt_fwd(z, mx.ACT_SILU)
    q = _bf16((1024, 512), gen)
    return {
        "wgrad": (mx.mx_ragged_gemm_wgrad_workspace_bytes(N, K, R, 1),
                  lambda s: mx.mx_ragged_gemm_wgrad(dy, x, 1, None, stream=s)),
        "wgrad f32": (mx.mx_ragged_gemm_wgrad_workspace_bytes(N, K, R, 1),
                      lambda s: mx.mx_ragged_gemm_wgrad_f32(dy, x, 1, None, torch.zeros((1, N, K), device="cuda"),
                                                            stream=s)),
        "checkpoint": (mx.mx_act_ckpt_workspace_bytes(2000, 1088),
                       lambda s: mx.mx_act_ckpt_bwd(ck, mx.ACT_SILU, z, recompute=True, colsum=True, stream=s)),
        "quantize": (int(mx.load().mx_quantize_workspace_bytes(1024, 512, mx.ROWWISE | mx.COLWISE | mx.COLSUM)),
                     lambda s: mx.mx_quantize(q, colsum=True, stream=s)[2]),
        "linear": (z.numel() * 2, lambda s: mx.mx_linear_fwd(x[:2000], dy[:1088], stream=s)),
    }


@pytest.mark.parametrize("name", ["wgrad", "wgrad f32", "checkpoint", "quantize", "linear"])
def test_workspace_of_another_stream(cuda_lib, name):
    """The launch waits behind its stream's work; meanwhile the current stream
    allocates and fills blocks of the workspace's size."""
    mx = cuda_lib
    nbytes, call = _calls(mx)[name]
    assert nbytes > 0
    want = _flat(call(None))
    side, busy = torch.cuda.Stream(), torch.empty(1 << 29, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            for _ in range(20):
                busy.zero_()
        got = _flat(call(side))
        junk = [torch.full(((nbytes + 3) // 4,), float("nan"), device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        assert len(got) == len(want) and all(torch.equal(g, w) for g, w in zip(got, want))
        assert all(bool(j.isnan().all()) for j in junk)
        del got, junk
    assert mx.mx_get_device_status() == "MX_OK"


@pytest.mark.parametrize("name", ["wgrad", "checkpoint", "quantize", "linear"])
def test_results_of_another_stream(cuda_lib, name):
    """Blocks that the current stream's pending work still writes, already given
    back to the allocator, hold no result of the other stream."""
    mx = cuda_lib
    _, call = _calls(mx)[name]
    want = _flat(call(None))
    side, busy = torch.cuda.Stream(), torch.empty(1 << 29, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(20):
            busy.zero_()
        for w in want:
            torch.empty_like(w).fill_(float("nan"))
        got = _flat(call(side))
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
        del got
    assert mx.mx_get_device_status() == "MX_OK"


def test_two_streams_at_once(cuda_lib):
    """The same calls on two streams side by side give the bits that they give
    alone (weight gradients in parts, checkpoints with column sums)."""
    mx = cuda_lib
    calls = [call for _, call in _calls(mx).values()]
    want = [_flat(call(None)) for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[_flat(call(s)) for call in calls] for _ in range(6) for s in streams]
    torch.cuda.synchronize()
    assert mx.mx_get_device_status() == "MX_OK"
    for outs in got:
        for g, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
