"""Bindings of the layers around the expert MLP: the layer norm, the expert
routing, the combine's gradient and products of 4-bit tensors.

As in the package's own module, every function checks what the C layer cannot
see and calls the C-ABI entry point of its name.  All of them are reached as
``mlp_gemms_gb300.mx_...``.
"""
import functools

import mlp_gemms_gb300 as _mx


def _here(first, *others):
    """_one_gpu, and that GPU the current one: it is where the call launches."""
    _mx._one_gpu(first, *others)
    _mx._stream()
    assert first.get_device() == _mx._current[1](), "the tensors are not on the current GPU"


def _type(t):
    import torch
    assert t.dtype in (torch.bfloat16, torch.float32), "neither BF16 nor fp32"
    return _mx.F32 if t.dtype == torch.float32 else _mx.BF16


def _rows(t, shape, dtype):
    """A matrix of this shape and type with dense rows; its row stride."""
    assert t.shape == shape and t.dtype == dtype and t.stride(1) == 1, "a matrix of another shape, type or layout"
    return t.stride(0) if shape[0] > 1 else shape[1]


def _vector(t, n, dtype=None):
    assert t is None or (t.shape == (n,) and t.is_contiguous() and dtype in (None, t.dtype)), \
        "a vector of another length, type or layout"


def _norm_weights(weight, bias, D):
    _vector(weight, D)
    _vector(bias, D, weight.dtype if weight is not None else None)
    return _mx.BF16 if weight is None and bias is None else _type(weight if weight is not None else bias)


def mx_layernorm_fwd(x, weight=None, bias=None, eps=1e-5, residual=None, rms=False, stats=True, out=None, sum_out=None,
                     mean=None, rstd=None, stream=None):
    """Layer norm (rms: without the mean) of the rows of s = x + residual (BF16
    or fp32 [R, D]): returns (y BF16, mean, rstd, s), s being x itself
    without a residual and mean None with rms; stats=False: no mean and rstd."""
    import torch
    R, D = x.shape
    xt, wt, dev = _type(x), _norm_weights(weight, bias, D), x.device
    ld_x, ld_res, ld_sum = _rows(x, (R, D), x.dtype), 0, 0
    if out is None:
        out = _mx._empty((R, D), torch.bfloat16, dev, stream)
    if residual is not None:
        ld_res = _rows(residual, (R, D), x.dtype)
        if sum_out is None:
            sum_out = _mx._empty((R, D), x.dtype, dev, stream)
        ld_sum = _rows(sum_out, (R, D), x.dtype)
    else:
        assert sum_out is None, "a sum without a residual"
    if stats and not rms and mean is None:
        mean = _mx._empty(R, torch.float32, dev, stream)
    if stats and rstd is None:
        rstd = _mx._empty(R, torch.float32, dev, stream)
    assert mean is None or not rms, "a mean with rms"
    _vector(mean, R, torch.float32)
    _vector(rstd, R, torch.float32)
    _here(x, weight, bias, residual, out, sum_out, mean, rstd)
    _mx._check(_mx.load().mx_layernorm_fwd(x.data_ptr(), xt, R, D, ld_x, _mx._ptr(residual), ld_res, _mx._ptr(sum_out), ld_sum,
                                   _mx._ptr(weight), _mx._ptr(bias), wt, eps, 1 if rms else 0, out.data_ptr(),
                                   _rows(out, (R, D), torch.bfloat16), _mx._ptr(mean), _mx._ptr(rstd), _mx._stream(stream)))
    return out, mean, rstd, x if residual is None else sum_out


@functools.lru_cache(maxsize=256)
def mx_layernorm_workspace_bytes(R, D):
    return int(_mx.load().mx_layernorm_workspace_bytes(R, D))


def mx_layernorm_bwd(dy, x, mean, rstd, weight=None, dres=None, rms=False, bias=True, wgrad=True, accumulate=False,
                     dx=None, dweight=None, dbias=None, workspace=None, stream=None):
    """The layer norm's backward pass; x: what it normalised (the forward's s).
    Returns (dx, dweight, dbias): dx of x's type with dres added, the others fp32
    [D], dweight None without wgrad, dbias None without bias; accumulate: added
    to the dweight and dbias that the caller brings."""
    import torch
    R, D = x.shape
    xt, wt, dev = _type(x), _norm_weights(weight, None, D), x.device
    ld_x, ld_dy = _rows(x, (R, D), x.dtype), _rows(dy, (R, D), torch.bfloat16)
    ld_dres = 0 if dres is None else _rows(dres, (R, D), x.dtype)
    assert not accumulate or ((dweight is not None or not wgrad) and (dbias is not None or not bias)), \
        "accumulate needs the buffers to add to"
    if dx is None:
        dx = _mx._empty((R, D), x.dtype, dev, stream)
    if wgrad and dweight is None:
        dweight = _mx._empty(D, torch.float32, dev, stream)
    if bias and dbias is None:
        dbias = _mx._empty(D, torch.float32, dev, stream)
    for t, n in ((mean, R), (rstd, R), (dweight, D), (dbias, D)):
        _vector(t, n, torch.float32)
    nbytes = 0
    if dweight is not None or dbias is not None:
        if workspace is None:
            workspace = _mx._empty(max(mx_layernorm_workspace_bytes(R, D), 16), torch.uint8, dev, stream)
        assert workspace.is_contiguous()
        nbytes = workspace.nbytes
    _here(x, dy, mean, rstd, weight, dres, dx, dweight, dbias, workspace)
    _mx._check(_mx.load().mx_layernorm_bwd(dy.data_ptr(), ld_dy, x.data_ptr(), xt, R, D, ld_x, _mx._ptr(mean), _mx._ptr(rstd),
                                   _mx._ptr(weight), wt, 1 if rms else 0, _mx._ptr(dres), ld_dres, dx.data_ptr(),
                                   _rows(dx, (R, D), x.dtype), _mx._ptr(dweight), _mx._ptr(dbias), 1 if accumulate else 0,
                                   _mx._ptr(workspace), nbytes, _mx._stream(stream)))
    return dx, dweight, dbias


# --------------------------------------------------------------------------
# Expert routing and the combine's gradient
# --------------------------------------------------------------------------

def _table(t, shape, dtype):
    """A dense table of this shape and type, or None."""
    assert t is None or (t.shape == shape and t.dtype == dtype and t.is_contiguous()), \
        "a table of another shape, type or layout"


@functools.lru_cache(maxsize=256)
def mx_moe_topk_workspace_bytes(T, G):
    return int(_mx.load().mx_moe_topk_workspace_bytes(T, G))


def mx_moe_topk(logits, k, score=_mx.SCORE_SOFTMAX, bias=None, groups=1, topk_groups=1, group_top=1, renorm=True,
                scale=1.0, stats=False, weights=None, ids=None, load=None, score_sum=None, workspace=None, stream=None):
    """The k experts of each token from its logits (BF16 or fp32 [T, G]) and
    their weights: returns (weights fp32 [T, k], ids int32 [T, k], load, score_sum),
    the last two (choices of each expert, sums of its scores) None without stats."""
    import torch
    T, G = logits.shape
    xt, dev = _type(logits), logits.device
    ld = _rows(logits, (T, G), logits.dtype)
    if weights is None:
        weights = _mx._empty((T, k), torch.float32, dev, stream)
    if ids is None:
        ids = _mx._empty((T, k), torch.int32, dev, stream)
    stats = stats or load is not None or score_sum is not None
    nbytes = 0
    if stats:
        load = load if load is not None else _mx._empty(G, torch.int32, dev, stream)
        score_sum = score_sum if score_sum is not None else _mx._empty(G, torch.float32, dev, stream)
        if workspace is None:
            workspace = _mx._empty(max(mx_moe_topk_workspace_bytes(T, G), 16), torch.uint8, dev, stream)
        assert workspace.is_contiguous()
        nbytes = workspace.nbytes
    _table(weights, (T, k), torch.float32)
    _table(ids, (T, k), torch.int32)
    _vector(bias, G, torch.float32)
    _vector(load, G, torch.int32)
    _vector(score_sum, G, torch.float32)
    _here(logits, bias, weights, ids, load, score_sum, workspace)
    _mx._check(_mx.load().mx_moe_topk(logits.data_ptr(), xt, T, G, ld, k, score, _mx._ptr(bias), groups, topk_groups,
                                      group_top, 1 if renorm else 0, scale, weights.data_ptr(), ids.data_ptr(),
                                      _mx._ptr(load), _mx._ptr(score_sum), _mx._ptr(workspace), nbytes,
                                      _mx._stream(stream)))
    return weights, ids, load, score_sum


def mx_moe_topk_bwd(logits, ids, dweights, score=_mx.SCORE_SOFTMAX, renorm=True, scale=1.0, dscore_sum=None,
                    dlogits=None, stream=None):
    """The logits' gradient (of their type) from that of the weights, and of
    score_sum where dscore_sum is given."""
    import torch
    T, G = logits.shape
    k = ids.shape[1]
    xt, ld = _type(logits), _rows(logits, (T, G), logits.dtype)
    if dlogits is None:
        dlogits = _mx._empty((T, G), logits.dtype, logits.device, stream)
    _table(ids, (T, k), torch.int32)
    _table(dweights, (T, k), torch.float32)
    _vector(dscore_sum, G, torch.float32)
    _here(logits, ids, dweights, dscore_sum, dlogits)
    _mx._check(_mx.load().mx_moe_topk_bwd(logits.data_ptr(), xt, T, G, ld, k, score, 1 if renorm else 0, scale,
                                          ids.data_ptr(), dweights.data_ptr(), _mx._ptr(dscore_sum),
                                          dlogits.data_ptr(), _rows(dlogits, (T, G), logits.dtype),
                                          _mx._stream(stream)))
    return dlogits


def mx_moe_unpermute_bwd(dout, inp, row_of, weights=None, src=None, din=None, dweights=None, stream=None):
    """The gradient of mx_moe_unpermute(inp, row_of, weights): returns (din, dweights),
    din[row_of[t, j]] = weights[t, j] dout[t] and dweights[t, j] = <dout[t], inp[row_of[t, j]]>.
    src (mx_moe_route_index's): the empty rows of din are zeroed; rows that
    neither names are left as they were."""
    import torch
    T, D = dout.shape
    R, k = inp.shape[0], row_of.shape[1]
    if din is None:
        din = _mx._empty((R, D), torch.bfloat16, dout.device, stream)
    if dweights is None:
        dweights = _mx._empty((T, k), torch.float32, dout.device, stream)
    for t, shape, dtype in ((dout, (T, D), torch.bfloat16), (inp, (R, D), torch.bfloat16), (din, (R, D), torch.bfloat16),
                            (row_of, (T, k), torch.int32), (weights, (T, k), torch.float32), (src, (R,), torch.int32),
                            (dweights, (T, k), torch.float32)):
        _table(t, shape, dtype)
    _here(dout, inp, row_of, weights, src, din, dweights)
    _mx._check(_mx.load().mx_moe_unpermute_bwd(dout.data_ptr(), T, D, inp.data_ptr(), R, row_of.data_ptr(), k,
                                               _mx._ptr(weights), _mx._ptr(src), din.data_ptr(), dweights.data_ptr(),
                                               _mx._stream(stream)))
    return din, dweights


# --------------------------------------------------------------------------
# 4-bit tensors with a scale for every 16 values
# --------------------------------------------------------------------------

@functools.lru_cache(maxsize=256)
def nvfp4_scale_bytes(rows, cols):
    return int(_mx.load().mx_nvfp4_scale_bytes(rows, cols))


class NVFP4:
    """A 4-bit tensor [rows, cols] in torch buffers: packed E2M1 codes (uint8
    [rows, cols / 2]), E4M3 scales per 16 values in the blocked layout (uint8),
    fp32 scale of each row (None as an operand: ones); stream: the one that fills
    them, where that is not the current one."""

    def __init__(self, rows, cols, device="cuda", data=None, scale=None, row_scale=None, stream=None):
        import torch
        self.rows, self.cols = int(rows), int(cols)
        if data is None:
            data = _mx._empty((rows, cols // 2), torch.uint8, device, stream)
            row_scale = row_scale if row_scale is not None else _mx._empty(rows, torch.float32, device, stream)
        self.data, self.row_scale = data, row_scale
        self.scale = scale if scale is not None else _mx._empty(nvfp4_scale_bytes(rows, cols), torch.uint8, device, stream)

    def struct(self):
        return _mx.Nvfp4Struct(self.data.data_ptr(), self.scale.data_ptr(), _mx._ptr(self.row_scale), self.rows, self.cols)


def _fp4_buffers(t):
    """A 4-bit tensor's buffers, dense and as large as its shape needs."""
    assert t.data.is_contiguous() and t.data.nbytes >= t.rows * (t.cols // 2), "the codes are strided or too few"
    assert t.scale.is_contiguous() and t.scale.nbytes >= nvfp4_scale_bytes(t.rows, t.cols), \
        "the scales are strided or too few"
    import torch
    _vector(t.row_scale, t.rows, torch.float32)
    return t.data, t.scale, t.row_scale


def mx_nvfp4_quantize(x, src=None, offsets=None, out=None, stream=None):
    """BF16 rows [T, K] as a 4-bit tensor; src int32 [R]: row r is x's row src[r],
    zeros where that is negative; offsets: rows from offsets[-1] on are not produced."""
    import ctypes

    import torch
    T, K = x.shape
    R = T if src is None else src.numel()
    ld = _rows(x, (T, K), torch.bfloat16)
    _vector(src, R, torch.int32)
    G = 0 if offsets is None else offsets.numel()
    _vector(offsets, G, torch.int32)
    if out is None:
        out = NVFP4(R, K, x.device, stream=stream)
    assert out.rows == R and out.cols == K, "a result of another shape"
    _here(x, src, offsets, *_fp4_buffers(out))
    _mx._check(_mx.load().mx_nvfp4_quantize(x.data_ptr(), T, K, ld, _mx._ptr(src), _mx._ptr(offsets), G,
                                            ctypes.byref(out.struct()), _mx._stream(stream)))
    return out


def mx_nvfp4_gemm(a, b, G=1, offsets=None, out=None, stream=None):
    """out[r] = a[r] b[g(r)]^T in BF16 from 4-bit operands a [R, K], b [G * N, K];
    rows past the last segment are not written."""
    import ctypes

    import torch
    N = b.rows // G if G > 0 else 0
    _vector(offsets, G, torch.int32)
    if out is None:
        out = _mx._empty((a.rows, N), torch.bfloat16, a.data.device, stream)
    ld = _rows(out, (a.rows, N), torch.bfloat16)
    data, scale, row_scale = _fp4_buffers(a)
    _here(data, scale, row_scale, offsets, out, *_fp4_buffers(b))
    _mx._check(_mx.load().mx_nvfp4_gemm(ctypes.byref(a.struct()), ctypes.byref(b.struct()), G, _mx._ptr(offsets),
                                        out.data_ptr(), ld, _mx._stream(stream)))
    return out
