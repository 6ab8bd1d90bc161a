"""Thin Python binding of the GB300 MX training-MLP library (``include/mx.h``).

Argument marshalling only: every function here computes nothing, checks what
the C layer cannot see of a tensor (types, layouts, devices), and calls exactly
one C-ABI entry point of the same name (``mx_mlp_fwd_bwd`` launches the whole
step).  PyTorch supplies device memory (outputs and workspaces are
``torch.empty`` allocations when the caller passes none, from the memory of the
stream that the call launches on) and the current CUDA stream.

There is no fallback: if the shared library is missing or fails to load,
``load()`` raises and nothing runs.
"""
import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libmxgb300.so")

E4M3, E2M3, E2M1 = 0, 1, 2
ROWWISE, COLWISE, HADAMARD, COLSUM = 1, 2, 4, 8
ACT_SWIGLU, ACT_GELU_TANH, ACT_NONE, ACT_SILU, ACT_RELU = 0, 1, 2, 3, 4
W_NK, W_KN = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
BF16, F32 = 0, 1  # types of the layers around the expert MLP (layers.py)

STATUS = {
    0: "MX_OK", 1: "MX_ERR_INVALID_ARG", 2: "MX_ERR_SHAPE", 3: "MX_ERR_ALIGNMENT", 4: "MX_ERR_OFFSETS",
    5: "MX_ERR_UNSUPPORTED_DEVICE", 6: "MX_ERR_CUDA", 7: "MX_ERR_DEVICE_TIMEOUT", 8: "MX_ERR_WORKSPACE",
    9: "MX_ERR_NOT_SUPPORTED",
}
STATUS_CODE = {v: k for k, v in STATUS.items()}

# Every symbol include/mx.h declares.
ABI_SYMBOLS = (
    "mx_abi_version", "mx_last_error", "mx_status_string", "mx_payload_bytes", "mx_scale_bytes",
    "mx_quantize_workspace_bytes", "mx_quantize", "mx_grouped_gemm", "mx_grouped_gemm_swiglu_fwd",
    "mx_grouped_gemm_dswiglu_bwd", "mx_grouped_gemm_wgrad", "mx_mlp_workspace_bytes", "mx_mlp_fwd_bwd",
    "mx_get_device_status", "mx_selftest_bounded_wait", "mx_gemm_bias", "mx_gemm_gelu_fwd",
    "mx_gemm_dgelu_workspace_bytes", "mx_gemm_dgelu_bwd", "mx_quantize_colsum_noalloc", "mx_debug_tap",
    "mx_mlp_pipeline_create", "mx_mlp_pipeline_run", "mx_mlp_pipeline_sync", "mx_mlp_pipeline_destroy",
    "mx_grouped_gemm_wgrad_f32", "mx_grouped_gemm_swiglu_probs_fwd", "mx_dswiglu_probs_workspace_bytes",
    "mx_grouped_gemm_dswiglu_probs_bwd", "mx_quantize_sr", "mx_moe_route_rows", "mx_moe_route_workspace_bytes",
    "mx_moe_route_index", "mx_permute_quantize", "mx_moe_unpermute", "mx_grouped_gemm_bias", "mx_grouped_gemm_bias_2sm",
    "mx_grouped_gemm_wgrad_workspace_bytes", "mx_grouped_gemm_wgrad_ws", "mx_grouped_gemm_wgrad_f32_ws",
    "mx_mlp_workspace_layout", "mx_moe_route_rows_pad", "mx_moe_route_index_pad", "mx_grouped_gemm_2sm",
    "mx_ragged_gemm", "mx_ragged_gemm_wgrad_workspace_bytes", "mx_ragged_gemm_wgrad", "mx_ragged_gemm_wgrad_f32",
    "mx_linear_fwd", "mx_act_ckpt_fwd", "mx_act_ckpt_workspace_bytes", "mx_act_ckpt_bwd", "mx_layernorm_fwd",
    "mx_layernorm_workspace_bytes", "mx_layernorm_bwd", "mx_moe_topk_workspace_bytes", "mx_moe_topk",
    "mx_moe_topk_bwd", "mx_moe_unpermute_bwd", "mx_nvfp4_scale_bytes",
    "mx_nvfp4_quantize_workspace_bytes", "mx_nvfp4_quantize", "mx_nvfp4_gemm",
)


class MXError(RuntimeError):
    def __init__(self, status, message):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__("%s: %s" % (self.name, message))


class MxTensorStruct(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("fmt", ctypes.c_int32), ("hadamard", ctypes.c_int32)]


class Nvfp4Struct(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("row_scale", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class MlpArgsStruct(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("fmt", ctypes.c_int32), ("hadamard", ctypes.c_int32),
                ("G", ctypes.c_int32), ("R", ctypes.c_int64), ("D", ctypes.c_int64), ("F", ctypes.c_int64),
                ("offsets", ctypes.c_void_p), ("x", ctypes.c_void_p), ("w1", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("dy", ctypes.c_void_p), ("b1", ctypes.c_void_p),
                ("b2", ctypes.c_void_p), ("y", ctypes.c_void_p), ("dx", ctypes.c_void_p),
                ("dw1", ctypes.c_void_p), ("dw2", ctypes.c_void_p), ("db1", ctypes.c_void_p),
                ("db2", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class MlpSlotStruct(ctypes.Structure):
    _fields_ = [("data", ctypes.c_size_t), ("scale", ctypes.c_size_t), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64)]


MLP_SLOTS = ("x_row", "x_col", "w1_row", "w1t_row", "w2_row", "w2t_row", "h_row", "h_col", "dy_row", "dy_col",
             "dz_row", "dz_col")


class MlpLayoutStruct(ctypes.Structure):
    _fields_ = [(n, MlpSlotStruct) for n in MLP_SLOTS] + [("z", ctypes.c_size_t), ("total", ctypes.c_size_t)]


class HostIOStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "w1", "w2", "dy", "b1", "b2", "offsets", "y", "dx", "dw1",
                                               "dw2", "db1", "db2")]


_lib = None


def load(path=None):
    """Load the CUDA library (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError("MX CUDA library not built at %s (run __graft_entry__.build())" % path)
    L = ctypes.CDLL(path)
    vp, i64, i32, u32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t
    f32 = ctypes.c_float
    tp = ctypes.POINTER(MxTensorStruct)
    sig = {
        "mx_abi_version": (ctypes.c_int, []),
        "mx_last_error": (ctypes.c_char_p, []),
        "mx_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "mx_payload_bytes": (sz, [i64, i64, i32]),
        "mx_scale_bytes": (sz, [i64, i64]),
        "mx_quantize_workspace_bytes": (sz, [i64, i64, u32]),
        "mx_quantize": (ctypes.c_int, [vp, i64, i64, i64, i64, i32, u32, tp, tp, vp, vp, sz, vp]),
        "mx_grouped_gemm": (ctypes.c_int, [tp, tp, i32, vp, vp, i64, vp]),
        "mx_grouped_gemm_2sm": (ctypes.c_int, [tp, tp, i32, vp, vp, i64, vp]),
        "mx_grouped_gemm_swiglu_fwd": (ctypes.c_int, [tp, tp, i32, vp, tp, tp, vp, vp]),
        "mx_grouped_gemm_dswiglu_bwd": (ctypes.c_int, [tp, tp, vp, i32, vp, tp, tp, vp]),
        "mx_grouped_gemm_wgrad": (ctypes.c_int, [tp, tp, i32, vp, vp, vp]),
        "mx_grouped_gemm_wgrad_f32": (ctypes.c_int, [tp, tp, i32, vp, vp, i32, vp]),
        "mx_grouped_gemm_swiglu_probs_fwd": (ctypes.c_int, [tp, tp, i32, vp, vp, tp, tp, vp, vp]),
        "mx_dswiglu_probs_workspace_bytes": (sz, [i64, i64]),
        "mx_grouped_gemm_dswiglu_probs_bwd": (ctypes.c_int, [tp, tp, vp, vp, i32, vp, tp, tp, vp, vp, sz, vp]),
        "mx_mlp_workspace_bytes": (sz, [ctypes.POINTER(MlpArgsStruct)]),
        "mx_mlp_workspace_layout": (ctypes.c_int, [ctypes.POINTER(MlpArgsStruct), ctypes.POINTER(MlpLayoutStruct)]),
        "mx_mlp_fwd_bwd": (ctypes.c_int, [ctypes.POINTER(MlpArgsStruct), vp]),
        "mx_get_device_status": (ctypes.c_int, [vp]),
        "mx_selftest_bounded_wait": (ctypes.c_int, [ctypes.c_uint64, vp]),
        "mx_gemm_bias": (ctypes.c_int, [tp, tp, vp, vp, i64, vp]),
        "mx_gemm_gelu_fwd": (ctypes.c_int, [tp, tp, vp, vp, tp, tp, vp]),
        "mx_gemm_dgelu_workspace_bytes": (sz, [i64, i64]),
        "mx_gemm_dgelu_bwd": (ctypes.c_int, [tp, tp, vp, tp, tp, vp, vp, sz, vp]),
        "mx_quantize_colsum_noalloc": (ctypes.c_int, [vp, i64, i64, i64, i32, u32, tp, tp, vp, vp]),
        "mx_quantize_sr": (ctypes.c_int, [vp, i64, i64, i64, i64, i32, u32, ctypes.c_uint64, tp, tp, vp]),
        "mx_moe_route_rows": (i64, [i64, i32, i32]),
        "mx_moe_route_workspace_bytes": (sz, [i64, i32, i32]),
        "mx_moe_route_index": (ctypes.c_int, [vp, i64, i32, i32, vp, vp, i64, vp, vp, sz, vp]),
        "mx_moe_route_rows_pad": (i64, [i64, i32, i32, i32]),
        "mx_moe_route_index_pad": (ctypes.c_int, [vp, i64, i32, i32, i32, vp, vp, i64, vp, vp, sz, vp]),
        "mx_permute_quantize": (ctypes.c_int, [vp, i64, i64, i64, vp, i64, vp, i32, i32, u32, tp, tp, vp]),
        "mx_moe_unpermute": (ctypes.c_int, [vp, i64, i64, vp, vp, i64, i32, vp, vp]),
        "mx_grouped_gemm_bias": (ctypes.c_int, [tp, tp, i32, vp, vp, vp, i64, vp]),
        "mx_grouped_gemm_bias_2sm": (ctypes.c_int, [tp, tp, i32, vp, vp, vp, i64, vp]),
        "mx_grouped_gemm_wgrad_workspace_bytes": (sz, [i64, i64, i64, i32]),
        "mx_grouped_gemm_wgrad_ws": (ctypes.c_int, [tp, tp, i32, vp, vp, vp, sz, vp]),
        "mx_grouped_gemm_wgrad_f32_ws": (ctypes.c_int, [tp, tp, i32, vp, vp, i32, vp, sz, vp]),
        "mx_ragged_gemm": (ctypes.c_int, [vp, i64, i64, i64, vp, i64, i32, i32, vp, vp, i64, vp]),
        "mx_ragged_gemm_wgrad_workspace_bytes": (sz, [i64, i64, i64, i32]),
        "mx_ragged_gemm_wgrad": (ctypes.c_int, [vp, i64, i64, vp, i64, i64, i64, i32, vp, vp, vp, sz, vp]),
        "mx_ragged_gemm_wgrad_f32": (ctypes.c_int, [vp, i64, i64, vp, i64, i64, i64, i32, vp, vp, i32, vp, sz, vp]),
        "mx_linear_fwd": (ctypes.c_int, [vp, i64, i64, i64, vp, i64, vp, i32, vp, i64, vp, i64, tp, vp]),
        "mx_act_ckpt_fwd": (ctypes.c_int, [vp, i64, i64, i64, i32, vp, i64, tp, vp]),
        "mx_act_ckpt_workspace_bytes": (sz, [i64, i64]),
        "mx_act_ckpt_bwd": (ctypes.c_int, [tp, i32, vp, i64, vp, i64, vp, i64, vp, vp, sz, vp]),
        "mx_layernorm_fwd": (ctypes.c_int, [vp, i32, i64, i64, i64, vp, i64, vp, i64, vp, vp, i32, f32, i32, vp, i64,
                                            vp, vp, vp]),
        "mx_layernorm_workspace_bytes": (sz, [i64, i64]),
        "mx_layernorm_bwd": (ctypes.c_int, [vp, i64, vp, i32, i64, i64, i64, vp, vp, vp, i32, i32, vp, i64, vp, i64,
                                            vp, vp, i32, vp, sz, vp]),
        "mx_moe_topk_workspace_bytes": (sz, [i64, i32]),
        "mx_moe_topk": (ctypes.c_int, [vp, i32, i64, i32, i64, i32, i32, vp, i32, i32, i32, i32, f32, vp, vp, vp, vp, vp,
                                       sz, vp]),
        "mx_moe_topk_bwd": (ctypes.c_int, [vp, i32, i64, i32, i64, i32, i32, i32, f32, vp, vp, vp, vp, i64, vp]),
        "mx_moe_unpermute_bwd": (ctypes.c_int, [vp, i64, i64, vp, i64, vp, i32, vp, vp, vp, vp, vp]),
        "mx_nvfp4_scale_bytes": (sz, [i64, i64]),
        "mx_nvfp4_quantize_workspace_bytes": (sz, [i64, i64, i64]),
        "mx_nvfp4_quantize": (ctypes.c_int, [vp, i64, i64, i64, vp, vp, i32, ctypes.POINTER(Nvfp4Struct), vp, sz, vp]),
        "mx_nvfp4_gemm": (ctypes.c_int, [ctypes.POINTER(Nvfp4Struct), ctypes.POINTER(Nvfp4Struct), i32, vp, vp, i64, vp]),
        "mx_debug_tap": (ctypes.c_int, [vp, i64]),
        "mx_mlp_pipeline_create": (ctypes.c_int, [ctypes.POINTER(MlpArgsStruct), vp, ctypes.POINTER(vp)]),
        "mx_mlp_pipeline_run": (ctypes.c_int, [vp, ctypes.POINTER(HostIOStruct)]),
        "mx_mlp_pipeline_sync": (ctypes.c_int, [vp]),
        "mx_mlp_pipeline_destroy": (None, [vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def _check(status):
    if status != 0:
        raise MXError(status, load().mx_last_error().decode())


_current = None  # torch's raw-stream and current-device queries


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    global _current
    if _current is None:
        from torch import _C
        _current = (_C._cuda_getCurrentRawStream, _C._cuda_getDevice)
    return _current[0](_current[1]())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _empty(shape, dtype, device, stream=None):
    """torch.empty for a launch on `stream`.  Memory of the current stream would
    be no other stream's: work still queued here may be using the block,
    and a workspace goes back to the allocator while the launch runs.  So
    another stream's buffers are its own, and kept until both are done."""
    import torch
    here = None if stream is None else torch.cuda.current_stream()
    if here is None or here == stream:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(here)
    return t


# --------------------------------------------------------------------------
# Quantized tensors
# --------------------------------------------------------------------------

@functools.lru_cache(maxsize=256)
def payload_bytes(rows, cols, fmt):
    return int(load().mx_payload_bytes(rows, cols, fmt))


@functools.lru_cache(maxsize=256)
def scale_bytes(rows, cols):
    return int(load().mx_scale_bytes(rows, cols))


class MX:
    """A quantized MX tensor [rows, cols] (blocks along cols) in torch buffers;
    stream: the one that fills them, where that is not the current one."""

    def __init__(self, rows, cols, fmt=E4M3, hadamard=False, device="cuda", data=None, scale=None, stream=None):
        import torch
        self.rows, self.cols, self.fmt, self.hadamard = int(rows), int(cols), int(fmt), bool(hadamard)
        self.data = data if data is not None else _empty((rows, payload_bytes(1, cols, fmt)), torch.uint8, device,
                                                         stream)
        self.scale = scale if scale is not None else _empty(scale_bytes(rows, cols), torch.uint8, device, stream)

    def struct(self):
        return MxTensorStruct(self.data.data_ptr(), self.scale.data_ptr(), self.rows, self.cols, self.fmt,
                              1 if self.hadamard else 0)


def _s(m):
    return None if m is None else ctypes.byref(m.struct())


# --------------------------------------------------------------------------
# Entry points (same names as the C ABI)
# --------------------------------------------------------------------------

def mx_quantize(x, fmt=E4M3, rowwise=True, colwise=True, hadamard=False, colsum=False, out_row=None,
                out_col=None, colsum_out=None, workspace=None, stream=None):
    """x: BF16 [rows, cols] or [batch, rows, cols] on the GPU.  Returns
    (out_row [batch*rows, cols], out_col [batch*cols, rows], colsum [cols])."""
    import torch
    assert x.dtype == torch.bfloat16
    batch = x.shape[0] if x.dim() == 3 else 1
    rows, cols = x.shape[-2], x.shape[-1]
    ld = x.stride(-2)
    flags = (ROWWISE if rowwise else 0) | (COLWISE if colwise else 0) | (HADAMARD if hadamard else 0) | \
            (COLSUM if colsum else 0)
    if rowwise and out_row is None:
        out_row = MX(batch * rows, cols, fmt, hadamard, x.device, stream=stream)
    if colwise and out_col is None:
        out_col = MX(batch * cols, rows, fmt, hadamard, x.device, stream=stream)
    ws_bytes = 0
    if colsum:
        if colsum_out is None:
            colsum_out = _empty(cols, torch.float32, x.device, stream)
        ws_bytes = int(load().mx_quantize_workspace_bytes(rows, cols, flags))
        if workspace is None:
            workspace = _empty(max(ws_bytes, 16), torch.uint8, x.device, stream)
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(load().mx_quantize(_ptr(x), batch, rows, cols, ld, fmt, flags, _s(out_row) if rowwise else None,
                              _s(out_col) if colwise else None, _ptr(colsum_out) if colsum else None,
                              _ptr(workspace) if colsum else None, ws_bytes, _stream(stream)))
    return out_row, out_col, colsum_out


def mx_quantize_sr(x, fmt, seed, rowwise=True, colwise=True, hadamard=False, out_row=None, out_col=None,
                   stream=None):
    """mx_quantize with stochastic rounding of the elements (E2M3 / E2M1);
    returns (out_row, out_col)."""
    import torch
    assert x.dtype == torch.bfloat16
    batch = x.shape[0] if x.dim() == 3 else 1
    rows, cols = x.shape[-2], x.shape[-1]
    ld = x.stride(-2)
    flags = (ROWWISE if rowwise else 0) | (COLWISE if colwise else 0) | (HADAMARD if hadamard else 0)
    if rowwise and out_row is None:
        out_row = MX(batch * rows, cols, fmt, hadamard, x.device, stream=stream)
    if colwise and out_col is None:
        out_col = MX(batch * cols, rows, fmt, hadamard, x.device, stream=stream)
    _check(load().mx_quantize_sr(x.data_ptr(), batch, rows, cols, ld, fmt, flags, int(seed),
                                 _s(out_row) if rowwise else None, _s(out_col) if colwise else None,
                                 _stream(stream)))
    return out_row, out_col


def mx_moe_route_rows(T, k, G):
    return int(load().mx_moe_route_rows(T, k, G))


def mx_moe_route_index(topk, G, R_cap=None, offsets=None, src=None, row_of=None, workspace=None, stream=None,
                       pad=128):
    """topk int32 [T, k] expert ids on the GPU -> (offsets [G], src [R_cap],
    row_of [T, k]) of the token permute; segments padded to `pad` (128 or
    256) rows."""
    import torch
    assert topk.dtype == torch.int32 and topk.is_contiguous()
    T, k = topk.shape
    dev = topk.device
    R_cap = R_cap if R_cap is not None else int(load().mx_moe_route_rows_pad(T, k, G, pad))
    offsets = offsets if offsets is not None else _empty(G, torch.int32, dev, stream)
    src = src if src is not None else _empty(R_cap, torch.int32, dev, stream)
    row_of = row_of if row_of is not None else _empty((T, k), torch.int32, dev, stream)
    nbytes = int(load().mx_moe_route_workspace_bytes(T, k, G))
    if workspace is None:
        workspace = _empty(max(nbytes, 16), torch.uint8, dev, stream)
    _check(load().mx_moe_route_index_pad(_ptr(topk), T, k, G, pad, _ptr(offsets), _ptr(src), R_cap, _ptr(row_of),
                                          _ptr(workspace), workspace.numel(), _stream(stream)))
    return offsets, src, row_of


def mx_permute_quantize(x, src, offsets=None, G=0, fmt=E4M3, rowwise=True, colwise=True, out_row=None,
                        out_col=None, stream=None):
    """The quantizing permute of BF16 tokens x [T, D] by src [R_cap]:
    returns (out_row [R_cap, D], out_col [D, R_cap])."""
    import torch
    assert x.dtype == torch.bfloat16 and src.dtype == torch.int32
    T, D = x.shape
    R_cap = src.numel()
    if offsets is not None and not G:
        G = offsets.numel()
    flags = (ROWWISE if rowwise else 0) | (COLWISE if colwise else 0)
    if rowwise and out_row is None:
        out_row = MX(R_cap, D, fmt, False, x.device, stream=stream)
    if colwise and out_col is None:
        out_col = MX(D, R_cap, fmt, False, x.device, stream=stream)
    _check(load().mx_permute_quantize(_ptr(x), T, D, x.stride(0), _ptr(src), R_cap, _ptr(offsets), int(G), fmt, flags,
                                      _s(out_row) if rowwise else None, _s(out_col) if colwise else None,
                                      _stream(stream)))
    return out_row, out_col


def mx_moe_unpermute(inp, row_of, weights=None, out=None, stream=None):
    """out[t] = sum_j w[t, j] * inp[row_of[t, j]] in BF16 (fp32 sums)."""
    import torch
    assert inp.dtype == torch.bfloat16 and inp.is_contiguous() and row_of.dtype == torch.int32
    R, D = inp.shape
    T, k = row_of.shape
    if out is None:
        out = _empty((T, D), torch.bfloat16, inp.device, stream)
    _check(load().mx_moe_unpermute(_ptr(inp), R, D, _ptr(row_of), _ptr(weights), T, k, _ptr(out), _stream(stream)))
    return out


def mx_quantize_colsum_noalloc(x, fmt=E4M3, rowwise=True, hadamard=False, out_row=None, out_col=None,
                               colsum_out=None, stream=None):
    """Quantize a BF16 [rows, cols] tensor columnwise (and rowwise) with the
    per-column sums, using the library's fixed scratch instead of a
    workspace: for callers that cannot allocate device memory.  Outputs are
    allocated here only when the caller passes none."""
    import torch
    rows, cols = x.shape
    flags = COLWISE | COLSUM | (ROWWISE if rowwise else 0) | (HADAMARD if hadamard else 0)
    if rowwise and out_row is None:
        out_row = MX(rows, cols, fmt, hadamard, x.device, stream=stream)
    if out_col is None:
        out_col = MX(cols, rows, fmt, hadamard, x.device, stream=stream)
    if colsum_out is None:
        colsum_out = _empty(cols, torch.float32, x.device, stream)
    _check(load().mx_quantize_colsum_noalloc(_ptr(x), rows, cols, x.stride(0), fmt, flags,
                                             _s(out_row) if rowwise else None, _s(out_col), _ptr(colsum_out),
                                             _stream(stream)))
    return out_row, out_col, colsum_out


def mx_grouped_gemm(a, b, G, offsets, out=None, ld_out=None, stream=None):
    import torch
    N = b.rows // G if G else 0
    if out is None:
        out = _empty((a.rows, N), torch.bfloat16, a.data.device, stream)
    ld = ld_out if ld_out is not None else out.stride(0)
    _check(load().mx_grouped_gemm(_s(a), _s(b), G, _ptr(offsets), _ptr(out), ld, _stream(stream)))
    return out


def mx_grouped_gemm_2sm(a, b, G, offsets, out=None, ld_out=None, stream=None):
    """mx_grouped_gemm on CTA pairs (256-row tiles; segments multiples of
    128, a 128-row remainder's upper half computed and not stored)."""
    import torch
    N = b.rows // G if G else 0
    if out is None:
        out = _empty((a.rows, N), torch.bfloat16, a.data.device, stream)
    ld = ld_out if ld_out is not None else out.stride(0)
    _check(load().mx_grouped_gemm_2sm(_s(a), _s(b), G, _ptr(offsets), _ptr(out), ld, _stream(stream)))
    return out


def mx_grouped_gemm_bias_2sm(a, b, G, offsets, bias, out=None, ld_out=None, stream=None):
    """mx_grouped_gemm_bias on CTA pairs."""
    import torch
    N = b.rows // G if G else 0
    assert bias.dtype == torch.bfloat16 and bias.is_contiguous()
    if out is None:
        out = _empty((a.rows, N), torch.bfloat16, a.data.device, stream)
    ld = ld_out if ld_out is not None else out.stride(0)
    _check(load().mx_grouped_gemm_bias_2sm(_s(a), _s(b), G, _ptr(offsets), _ptr(bias), _ptr(out), ld,
                                           _stream(stream)))
    return out


def mx_grouped_gemm_bias(a, b, G, offsets, bias, out=None, ld_out=None, stream=None):
    """mx_grouped_gemm with expert g's BF16 bias row bias[g] [G, N] added in
    the fp32 accumulator."""
    import torch
    N = b.rows // G if G else 0
    assert bias.dtype == torch.bfloat16 and bias.is_contiguous()
    if out is None:
        out = _empty((a.rows, N), torch.bfloat16, a.data.device, stream)
    ld = ld_out if ld_out is not None else out.stride(0)
    _check(load().mx_grouped_gemm_bias(_s(a), _s(b), G, _ptr(offsets), _ptr(bias), _ptr(out), ld, _stream(stream)))
    return out


def mx_grouped_gemm_swiglu_fwd(x_row, w1_row, G, offsets, h_row=None, h_col=None, z=None, stream=None):
    import torch
    R = x_row.rows
    F = w1_row.rows // (2 * G)
    dev = x_row.data.device
    if h_row is None:
        h_row = MX(R, F, E4M3, False, dev, stream=stream)
    if h_col is None:
        h_col = MX(F, R, E4M3, False, dev, stream=stream)
    if z is None:
        z = _empty((R, 2 * F), torch.bfloat16, dev, stream)
    _check(load().mx_grouped_gemm_swiglu_fwd(_s(x_row), _s(w1_row), G, _ptr(offsets), _s(h_row), _s(h_col),
                                             _ptr(z), _stream(stream)))
    return z, h_row, h_col


def mx_grouped_gemm_swiglu_probs_fwd(x_row, w1_row, G, offsets, probs, h_row=None, h_col=None, z=None, stream=None):
    """FC1 + SwiGLU with each routed row's activation scaled by probs [R] (fp32)."""
    import torch
    R = x_row.rows
    F = w1_row.rows // (2 * G)
    dev = x_row.data.device
    h_row = h_row if h_row is not None else MX(R, F, E4M3, False, dev, stream=stream)
    h_col = h_col if h_col is not None else MX(F, R, E4M3, False, dev, stream=stream)
    z = z if z is not None else _empty((R, 2 * F), torch.bfloat16, dev, stream)
    _check(load().mx_grouped_gemm_swiglu_probs_fwd(_s(x_row), _s(w1_row), G, _ptr(offsets), _ptr(probs), _s(h_row),
                                                   _s(h_col), _ptr(z), _stream(stream)))
    return z, h_row, h_col


def mx_grouped_gemm_dswiglu_probs_bwd(dy_row, w2t_row, z, probs, G, offsets, dz_row=None, dz_col=None,
                                      dprobs=None, workspace=None, stream=None):
    """The matching backward; returns (dz_row, dz_col, dprobs [R] fp32)."""
    import torch
    R = dy_row.rows
    F = w2t_row.rows // G
    dev = dy_row.data.device
    dz_row = dz_row if dz_row is not None else MX(R, 2 * F, E4M3, False, dev, stream=stream)
    dz_col = dz_col if dz_col is not None else MX(2 * F, R, E4M3, False, dev, stream=stream)
    dprobs = dprobs if dprobs is not None else _empty(R, torch.float32, dev, stream)
    nbytes = int(load().mx_dswiglu_probs_workspace_bytes(R, F))
    if workspace is None:
        workspace = _empty(max(nbytes, 16), torch.uint8, dev, stream)
    _check(load().mx_grouped_gemm_dswiglu_probs_bwd(
        _s(dy_row), _s(w2t_row), _ptr(z), _ptr(probs), G, _ptr(offsets), _s(dz_row), _s(dz_col), _ptr(dprobs),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return dz_row, dz_col, dprobs


def mx_grouped_gemm_dswiglu_bwd(dy_row, w2t_row, z, G, offsets, dz_row=None, dz_col=None, stream=None):
    R = dy_row.rows
    F = w2t_row.rows // G
    dev = dy_row.data.device
    if dz_row is None:
        dz_row = MX(R, 2 * F, E4M3, False, dev, stream=stream)
    if dz_col is None:
        dz_col = MX(2 * F, R, E4M3, False, dev, stream=stream)
    _check(load().mx_grouped_gemm_dswiglu_bwd(_s(dy_row), _s(w2t_row), _ptr(z), G, _ptr(offsets), _s(dz_row),
                                              _s(dz_col), _stream(stream)))
    return dz_row, dz_col


def mx_grouped_gemm_wgrad(a_col, b_col, G, offsets, out=None, stream=None):
    import torch
    if out is None:
        out = _empty((G, a_col.rows, b_col.rows), torch.bfloat16, a_col.data.device, stream)
    _check(load().mx_grouped_gemm_wgrad(_s(a_col), _s(b_col), G, _ptr(offsets), _ptr(out), _stream(stream)))
    return out


def mx_grouped_gemm_wgrad_f32(a_col, b_col, G, offsets, grad, accumulate=False, stream=None):
    """Weight gradient into the caller's fp32 buffer grad [G, N, K]: stored
    (accumulate=False) or added to what it holds (accumulate=True)."""
    import torch
    assert grad.dtype == torch.float32 and grad.is_contiguous()
    _check(load().mx_grouped_gemm_wgrad_f32(_s(a_col), _s(b_col), G, _ptr(offsets), _ptr(grad),
                                            1 if accumulate else 0, _stream(stream)))
    return grad


def mx_grouped_gemm_wgrad_workspace_bytes(N, K, R, G):
    return int(load().mx_grouped_gemm_wgrad_workspace_bytes(N, K, R, G))


def _wgrad_ws(a_col, b_col, G, workspace, stream):
    import torch
    if workspace is None:
        n = mx_grouped_gemm_wgrad_workspace_bytes(a_col.rows, b_col.rows, a_col.cols, G)
        workspace = _empty(max(n, 16), torch.uint8, a_col.data.device, stream)
    return workspace


def mx_grouped_gemm_wgrad_ws(a_col, b_col, G, offsets, out=None, workspace=None, stream=None):
    """mx_grouped_gemm_wgrad with the largest experts' K range split across
    CTAs (workspace from mx_grouped_gemm_wgrad_workspace_bytes)."""
    import torch
    if out is None:
        out = _empty((G, a_col.rows, b_col.rows), torch.bfloat16, a_col.data.device, stream)
    ws = _wgrad_ws(a_col, b_col, G, workspace, stream)
    _check(load().mx_grouped_gemm_wgrad_ws(_s(a_col), _s(b_col), G, _ptr(offsets), _ptr(out), _ptr(ws), ws.numel(),
                                           _stream(stream)))
    return out


def mx_grouped_gemm_wgrad_f32_ws(a_col, b_col, G, offsets, grad, accumulate=False, workspace=None, stream=None):
    import torch
    assert grad.dtype == torch.float32 and grad.is_contiguous()
    ws = _wgrad_ws(a_col, b_col, G, workspace, stream)
    _check(load().mx_grouped_gemm_wgrad_f32_ws(_s(a_col), _s(b_col), G, _ptr(offsets), _ptr(grad),
                                               1 if accumulate else 0, _ptr(ws), ws.numel(), _stream(stream)))
    return grad


def mx_gemm_bias(a, b, bias=None, out=None, ld_out=None, stream=None):
    import torch
    if out is None:
        out = _empty((a.rows, b.rows), torch.bfloat16, a.data.device, stream)
    ld = ld_out if ld_out is not None else out.stride(0)
    _check(load().mx_gemm_bias(_s(a), _s(b), _ptr(bias), _ptr(out), ld, _stream(stream)))
    return out


def mx_gemm_gelu_fwd(x_row, w1_row, b1=None, pre=None, act_row=None, act_col=None, fmt=E2M3, hadamard=True,
                     stream=None):
    import torch
    M, H = x_row.rows, w1_row.rows
    dev = x_row.data.device
    if pre is None:
        pre = _empty((M, H), torch.bfloat16, dev, stream)
    if act_row is None:
        act_row = MX(M, H, fmt, hadamard, dev, stream=stream)
    if act_col is None:
        act_col = MX(H, M, fmt, hadamard, dev, stream=stream)
    _check(load().mx_gemm_gelu_fwd(_s(x_row), _s(w1_row), _ptr(b1), _ptr(pre), _s(act_row), _s(act_col),
                                   _stream(stream)))
    return pre, act_row, act_col


def mx_gemm_dgelu_workspace_bytes(M, H):
    return int(load().mx_gemm_dgelu_workspace_bytes(M, H))


def mx_gemm_dgelu_bwd(dy_row, w2t_row, pre, dpre_row=None, dpre_col=None, db1=None, workspace=None, fmt=E2M3,
                      hadamard=True, stream=None):
    import torch
    M, H = dy_row.rows, w2t_row.rows
    dev = dy_row.data.device
    if dpre_row is None:
        dpre_row = MX(M, H, fmt, hadamard, dev, stream=stream)
    if dpre_col is None:
        dpre_col = MX(H, M, fmt, hadamard, dev, stream=stream)
    if db1 is None:
        db1 = _empty(H, torch.float32, dev, stream)
    if workspace is None:
        workspace = _empty(max(mx_gemm_dgelu_workspace_bytes(M, H), 16), torch.uint8, dev, stream)
    _check(load().mx_gemm_dgelu_bwd(_s(dy_row), _s(w2t_row), _ptr(pre), _s(dpre_row), _s(dpre_col), _ptr(db1),
                                    _ptr(workspace), workspace.numel(), _stream(stream)))
    return dpre_row, dpre_col, db1


# --------------------------------------------------------------------------
# BF16 layers: ragged products, linear layer, 8-bit activation checkpoints
# --------------------------------------------------------------------------

def _one_gpu(first, *others):
    """Refuse host tensors and tensors of several GPUs: the library takes bare
    pointers."""
    dev = first.get_device()
    assert dev >= 0, "a tensor is not on a GPU"
    for t in others:
        assert t is None or t.get_device() == dev, "the tensors are not on one GPU"


def _buffers(t):
    """An MX tensor's (payload, scales), dense and as large as its shape needs."""
    data, scale = t.data, t.scale
    assert data.is_contiguous() and data.nbytes >= payload_bytes(t.rows, t.cols, t.fmt), \
        "the payload is strided or too small"
    assert scale.is_contiguous() and scale.nbytes >= scale_bytes(t.rows, t.cols), "the scales are strided or too small"
    return data, scale


def mx_ragged_gemm(a, w, offsets, layout=W_NK, out=None, stream=None):
    """out[r] = a[r] w[g]^T (W_NK, w [G, N, K]) or a[r] w[g] (W_KN, w [G, K, N])
    for the rows r of expert g's segment, of any length; BF16.  Rows past
    the last segment are not written."""
    import torch
    assert a.dtype == torch.bfloat16 and w.dtype == torch.bfloat16 and w.is_contiguous() and w.dim() == 3
    assert a.stride(1) == 1 and (offsets is None or (offsets.dtype == torch.int32 and offsets.is_contiguous()))
    R, K = a.shape
    G, N = w.shape[0], w.shape[1 if layout == W_NK else 2]
    assert w.shape[2 if layout == W_NK else 1] == K and (offsets is None or offsets.numel() == G)
    if out is None:
        out = _empty((R, N), torch.bfloat16, a.device, stream)
    assert out.shape == (R, N) and out.dtype == torch.bfloat16 and out.stride(1) == 1
    _one_gpu(a, w, offsets, out)
    _check(load().mx_ragged_gemm(a.data_ptr(), R, K, a.stride(0), w.data_ptr(), N, G, layout, _ptr(offsets),
                                 out.data_ptr(), out.stride(0), _stream(stream)))
    return out


def mx_ragged_gemm_wgrad_workspace_bytes(N, K, R, G):
    return int(load().mx_ragged_gemm_wgrad_workspace_bytes(N, K, R, G))


def _ragged_wgrad_args(dy, x, G, offsets, grad, workspace, stream):
    import torch
    assert dy.dtype == torch.bfloat16 and x.dtype == torch.bfloat16 and dy.shape[0] == x.shape[0]
    assert dy.stride(1) == 1 and x.stride(1) == 1
    assert offsets is None or (offsets.dtype == torch.int32 and offsets.numel() == G and offsets.is_contiguous())
    assert workspace is None or workspace.is_contiguous()
    _one_gpu(dy, x, offsets, grad, workspace)
    R, N = dy.shape
    K = x.shape[1]
    if workspace is None:
        n = mx_ragged_gemm_wgrad_workspace_bytes(N, K, R, G)
        workspace = _empty(n, torch.uint8, dy.device, stream) if n else None
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return R, N, K, workspace, nbytes


def mx_ragged_gemm_wgrad(dy, x, G, offsets, out=None, workspace=None, stream=None):
    """Weight gradients [G, N, K] = dy_g^T x_g of ragged segments, BF16."""
    import torch
    R, N, K, workspace, nbytes = _ragged_wgrad_args(dy, x, G, offsets, out, workspace, stream)
    if out is None:
        out = _empty((G, N, K), torch.bfloat16, dy.device, stream)
    assert out.shape == (G, N, K) and out.dtype == torch.bfloat16 and out.is_contiguous()
    _check(load().mx_ragged_gemm_wgrad(dy.data_ptr(), N, dy.stride(0), x.data_ptr(), K, x.stride(0), R, G,
                                       _ptr(offsets), out.data_ptr(), _ptr(workspace), nbytes, _stream(stream)))
    return out


def mx_ragged_gemm_wgrad_f32(dy, x, G, offsets, grad, accumulate=False, workspace=None, stream=None):
    """The weight gradients into the caller's fp32 buffer grad [G, N, K]:
    stored (accumulate=False) or added to what it holds."""
    import torch
    R, N, K, workspace, nbytes = _ragged_wgrad_args(dy, x, G, offsets, grad, workspace, stream)
    assert grad.shape == (G, N, K) and grad.dtype == torch.float32 and grad.is_contiguous()
    _check(load().mx_ragged_gemm_wgrad_f32(dy.data_ptr(), N, dy.stride(0), x.data_ptr(), K, x.stride(0), R, G,
                                           _ptr(offsets), grad.data_ptr(), 1 if accumulate else 0, _ptr(workspace),
                                           nbytes, _stream(stream)))
    return grad


def mx_linear_fwd(x, w, bias=None, act=ACT_NONE, residual=None, out=None, ckpt=None, stream=None):
    """act(x w^T + bias) + residual in BF16 (x [M, K], w [N, K]); ckpt: an
    E4M3 MX tensor [M, N] that receives the pre-activation in 8 bits."""
    import torch
    assert x.dtype == torch.bfloat16 and w.dtype == torch.bfloat16 and w.is_contiguous() and x.stride(1) == 1
    M, K = x.shape
    N = w.shape[0]
    assert w.shape == (N, K)
    assert bias is None or (bias.dtype == torch.bfloat16 and bias.shape == (N,) and bias.is_contiguous())
    if out is None:
        out = _empty((M, N), torch.bfloat16, x.device, stream)
    assert out.shape == (M, N) and out.dtype == torch.bfloat16 and out.stride(1) == 1
    ld_res = 0
    if residual is not None:
        assert residual.shape == (M, N) and residual.dtype == torch.bfloat16 and residual.stride(1) == 1
        ld_res = residual.stride(0)
    _one_gpu(x, w, bias, residual, out, *(_buffers(ckpt) if ckpt is not None else ()))
    _check(load().mx_linear_fwd(x.data_ptr(), M, K, x.stride(0), w.data_ptr(), N, _ptr(bias), act, _ptr(residual),
                                ld_res, out.data_ptr(), out.stride(0), _s(ckpt), _stream(stream)))
    return out


def mx_act_ckpt_fwd(z, act, h=None, ckpt=None, stream=None):
    """h = act(z) (SwiGLU: z [R, 2F] = [gate | up], h [R, F]) and z's 8-bit
    checkpoint, in one pass: returns (h, MX [R, C])."""
    import torch
    assert z.dtype == torch.bfloat16 and z.stride(1) == 1
    R, C = z.shape
    if h is None:
        h = _empty((R, C // 2 if act == ACT_SWIGLU else C), torch.bfloat16, z.device, stream)
    assert h.shape == (R, C // 2 if act == ACT_SWIGLU else C) and h.dtype == torch.bfloat16 and h.stride(1) == 1
    if ckpt is None:
        ckpt = MX(R, C, E4M3, False, z.device, stream=stream)
        _one_gpu(z, h)
    else:
        _one_gpu(z, h, *_buffers(ckpt))
    _check(load().mx_act_ckpt_fwd(z.data_ptr(), R, C, z.stride(0), act, h.data_ptr(), h.stride(0), _s(ckpt),
                                  _stream(stream)))
    return h, ckpt


@functools.lru_cache(maxsize=256)
def mx_act_ckpt_workspace_bytes(R, C):
    return int(load().mx_act_ckpt_workspace_bytes(R, C))


def mx_act_ckpt_bwd(ckpt, act, dh, dz=None, recompute=False, h=None, colsum=False, db=None, workspace=None,
                    stream=None):
    """The activation's backward pass from the 8-bit checkpoint: returns
    (dz [R, C], h or None, db or None): h = act of the checkpoint's values
    when `recompute` or `h`, db = fp32 column sums of dz when `colsum` or `db`."""
    import torch
    R, C = ckpt.rows, ckpt.cols
    H = C // 2 if act == ACT_SWIGLU else C
    dev, bf16 = dh.device, torch.bfloat16
    assert dh.dtype == bf16 and dh.shape == (R, H) and dh.stride(1) == 1
    if dz is None:
        dz = _empty((R, C), bf16, dev, stream)
    else:
        assert dz.shape == (R, C) and dz.dtype == bf16 and dz.stride(1) == 1
    if h is not None:
        assert h.shape == (R, H) and h.dtype == bf16 and h.stride(1) == 1
    elif recompute:
        h = _empty((R, H), bf16, dev, stream)
    if db is not None:
        assert db.shape == (C,) and db.dtype == torch.float32 and db.is_contiguous()
    elif colsum:
        db = _empty(C, torch.float32, dev, stream)
    nbytes = 0
    if db is not None:
        if workspace is None:
            n = mx_act_ckpt_workspace_bytes(R, C)
            workspace = _empty(n, torch.uint8, dev, stream) if n else None
        if workspace is not None:
            assert workspace.is_contiguous()
            nbytes = workspace.numel() * workspace.element_size()
    _one_gpu(dh, dz, h, db, workspace, *_buffers(ckpt))
    _check(load().mx_act_ckpt_bwd(_s(ckpt), act, dh.data_ptr(), dh.stride(0), dz.data_ptr(), dz.stride(0), _ptr(h),
                                  0 if h is None else h.stride(0), _ptr(db), _ptr(workspace), nbytes,
                                  _stream(stream)))
    return dz, h, db


def mlp_args(x, w1, w2, dy, offsets, G, F, y, dx, dw1, dw2, workspace=None, act=ACT_SWIGLU, fmt=E4M3,
             hadamard=False, b1=None, b2=None, db1=None, db2=None):
    R, D = x.shape
    a = MlpArgsStruct()
    a.act, a.fmt, a.hadamard, a.G = act, fmt, 1 if hadamard else 0, G
    a.R, a.D, a.F = R, D, F
    for name, t in (("offsets", offsets), ("x", x), ("w1", w1), ("w2", w2), ("dy", dy), ("b1", b1), ("b2", b2),
                    ("y", y), ("dx", dx), ("dw1", dw1), ("dw2", dw2), ("db1", db1), ("db2", db2)):
        setattr(a, name, None if t is None else t.data_ptr())
    if workspace is not None:
        a.workspace = workspace.data_ptr()
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    return a


def mx_mlp_workspace_bytes(args):
    return int(load().mx_mlp_workspace_bytes(ctypes.byref(args)))


def mx_mlp_workspace_layout(args):
    """{slot: (payload offset, scale offset, rows, cols)} for every quantized
    tensor of the step, plus "z" (offset of the BF16 pre-activation) and
    "total" (workspace bytes)."""
    out = MlpLayoutStruct()
    _check(load().mx_mlp_workspace_layout(ctypes.byref(args), ctypes.byref(out)))
    lay = {n: (int(getattr(out, n).data), int(getattr(out, n).scale), int(getattr(out, n).rows),
               int(getattr(out, n).cols)) for n in MLP_SLOTS}
    lay["z"] = int(out.z)
    lay["total"] = int(out.total)
    return lay


def mlp_workspace_views(args, workspace):
    """The step's intermediates as views into its workspace (uint8 torch
    tensor): {slot: MX} and "z" (BF16 [R, F1])."""
    import torch
    lay = mx_mlp_workspace_layout(args)
    views = {}
    for n in MLP_SLOTS:
        d, sc, rows, cols = lay[n]
        rb = payload_bytes(1, cols, args.fmt)
        data = workspace[d:d + rows * rb].view(rows, rb)
        scale = workspace[sc:sc + scale_bytes(rows, cols)]
        views[n] = MX(rows, cols, args.fmt, bool(args.hadamard), workspace.device, data=data, scale=scale)
    f1 = lay["dz_row"][3]
    views["z"] = workspace[lay["z"]:lay["z"] + args.R * f1 * 2].view(torch.bfloat16).view(args.R, f1)
    return views


def mx_mlp_fwd_bwd(args, stream=None):
    _check(load().mx_mlp_fwd_bwd(ctypes.byref(args), _stream(stream)))


class MlpPipeline:
    """The step with host-memory inputs and outputs (mx_mlp_pipeline_*).

    dev_args: the device argument block (mlp_args with a workspace) whose
    buffers the pipeline stages through; the tensors behind it must outlive
    the pipeline.  run(host) takes CPU tensors (pinned, for overlap) keyed
    x, w1, w2, dy, offsets, y, dx, dw1, dw2 (and b1, b2, db1, db2 for GELU);
    they are read and written asynchronously until sync()."""

    def __init__(self, dev_args, stream=None):
        self._args = dev_args
        h = ctypes.c_void_p()
        _check(load().mx_mlp_pipeline_create(ctypes.byref(dev_args), _stream(stream), ctypes.byref(h)))
        self._h = h
        self._io = []

    def run(self, host):
        io = HostIOStruct()
        for name, _ in HostIOStruct._fields_:
            t = host.get(name)
            setattr(io, name, None if t is None else t.data_ptr())
        self._io.append(io)
        _check(load().mx_mlp_pipeline_run(self._h, ctypes.byref(io)))

    def sync(self):
        _check(load().mx_mlp_pipeline_sync(self._h))
        self._io = []

    def close(self):
        if self._h is not None:
            load().mx_mlp_pipeline_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def mx_get_device_status(stream=None):
    """Synchronise and return the device status name ('MX_OK' or an error)."""
    return STATUS.get(int(load().mx_get_device_status(_stream(stream))), "unknown")


def mx_selftest_bounded_wait(budget_ns, stream=None):
    _check(load().mx_selftest_bounded_wait(int(budget_ns), _stream(stream)))


def mx_debug_tap(tap=None):
    """Attach (fp32 CUDA tensor) or detach (None) the fused epilogues' test
    tap on this host thread: they also write their fp32 pre-quantization
    values into it, row-major [rows, cols] of the requantized output."""
    if tap is None:
        _check(load().mx_debug_tap(None, 0))
        return
    import torch
    assert tap.dtype == torch.float32 and tap.is_cuda and tap.is_contiguous()
    _check(load().mx_debug_tap(tap.data_ptr(), tap.numel()))


def mx_last_error():
    return load().mx_last_error().decode()


# The layers around the expert MLP are part of this namespace and live in
# layers.py, which loads with the first of them.
_LAYERS = ("NVFP4", "mx_layernorm_bwd", "mx_layernorm_fwd", "mx_layernorm_workspace_bytes", "mx_moe_topk",
           "mx_moe_topk_bwd", "mx_moe_topk_workspace_bytes", "mx_moe_unpermute_bwd", "mx_nvfp4_gemm",
           "mx_nvfp4_quantize", "mx_nvfp4_quantize_workspace_bytes", "nvfp4_scale_bytes")
_layers = None


def __getattr__(name):
    global _layers
    if name not in _LAYERS:
        raise AttributeError("module %r has no attribute %r" % (__name__, name))
    if _layers is None:
        import importlib
        _layers = importlib.import_module(__name__ + ".layers").__dict__
    return _layers[name]


def __dir__():
    return sorted({*globals(), *_LAYERS})


__all__ = [n for n in globals() if n[0] != "_"] + list(_LAYERS)
