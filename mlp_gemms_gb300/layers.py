"""Bindings of the layers around the expert MLP: the layer norm, the expert
routing, the combine's gradient and products of 4-bit tensors.

As in the package's own module, every function checks what the C layer cannot
see and calls the C-ABI entry point of its name.  All of them are reached as
``mlp_gemms_gb300.mx_...``.
"""
import ctypes
import functools

import torch

import mlp_gemms_gb300 as _mx

_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


# Each tensor's attributes are asked for once: the checks are a good part of a
# small call's time.

def _gpu(t):
    """The tensor's GPU, which has to be the current one: the call launches there,
    and the library takes bare pointers."""
    if _mx._current is None:
        _mx._stream()
    dev = t.get_device()
    assert dev >= 0 and dev == _mx._current[1](), "a tensor is not on the current GPU"
    return dev


def _type(t):
    dtype = t.dtype
    assert dtype is _BF16 or dtype is _F32, "neither BF16 nor fp32"
    return _mx.F32 if dtype is _F32 else _mx.BF16


def _rows(t, shape, dtype, dev):
    """Pointer and row stride of a matrix of this shape and type with dense rows."""
    step, one = t.stride()
    assert t.shape == shape and t.dtype is dtype and one == 1 and t.get_device() == dev, \
        "a matrix of another shape, type or layout, or on another GPU"
    return t.data_ptr(), step if shape[0] > 1 else shape[1]


def _dense(t, shape, dtype, dev):
    """Pointer of a dense tensor of this shape and type, or None."""
    if t is None:
        return None
    assert t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.get_device() == dev, \
        "a tensor of another shape, type or layout, or on another GPU"
    return t.data_ptr()


def _new(shape, dtype, like, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    return _mx._empty(shape, dtype, like.device, stream)


def _workspace(workspace, nbytes, like, dev, stream):
    """(workspace, its pointer, its size), allocated where the caller brings none."""
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        workspace = _new(nbytes, _U8, like, stream)
        return workspace, workspace.data_ptr(), nbytes
    assert workspace.is_contiguous() and workspace.get_device() == dev, "a strided workspace, or on another GPU"
    return workspace, workspace.data_ptr(), workspace.nbytes


# --------------------------------------------------------------------------
# Layer norm
# --------------------------------------------------------------------------

def mx_layernorm_fwd(x, weight=None, bias=None, eps=1e-5, residual=None, rms=False, stats=True, out=None, sum_out=None,
                     mean=None, rstd=None, stream=None):
    """Layer norm (rms: without the mean) of the rows of s = x + residual (BF16
    or fp32 [R, D]): returns (y BF16, mean, rstd, s), s being x itself
    without a residual and mean None with rms; stats=False: no mean and rstd."""
    shape, dev, dtype = x.shape, _gpu(x), x.dtype
    R, D = shape
    xt = _type(x)
    xp, ld_x = _rows(x, shape, dtype, dev)
    wt, wp, bp = _mx.BF16, None, None
    if weight is not None:
        wt, wp = _type(weight), _dense(weight, (D,), weight.dtype, dev)
    if bias is not None:
        wt, bp = _type(bias), _dense(bias, (D,), bias.dtype if weight is None else weight.dtype, dev)
    rp, ld_res, sp, ld_sum = None, 0, None, 0
    if residual is not None:
        rp, ld_res = _rows(residual, shape, dtype, dev)
        if sum_out is None:
            sum_out = _new(shape, dtype, x, stream)
            sp, ld_sum = sum_out.data_ptr(), D
        else:
            sp, ld_sum = _rows(sum_out, shape, dtype, dev)
    else:
        assert sum_out is None, "a sum without a residual"
    if out is None:
        out = _new(shape, _BF16, x, stream)
        yp, ld_y = out.data_ptr(), D
    else:
        yp, ld_y = _rows(out, shape, _BF16, dev)
    mp = sdp = None
    assert mean is None or not rms, "a mean with rms"
    if mean is not None:
        mp = _dense(mean, (R,), _F32, dev)
    elif stats and not rms:
        mean = _new(R, _F32, x, stream)
        mp = mean.data_ptr()
    if rstd is not None:
        sdp = _dense(rstd, (R,), _F32, dev)
    elif stats:
        rstd = _new(R, _F32, x, stream)
        sdp = rstd.data_ptr()
    _mx._check(_mx.load().mx_layernorm_fwd(xp, xt, R, D, ld_x, rp, ld_res, sp, ld_sum, wp, bp, wt, eps, 1 if rms else 0,
                                           yp, ld_y, mp, sdp, _mx._stream(stream)))
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
    shape, dev, dtype = x.shape, _gpu(x), x.dtype
    R, D = shape
    xt = _type(x)
    xp, ld_x = _rows(x, shape, dtype, dev)
    dyp, ld_dy = _rows(dy, shape, _BF16, dev)
    wt, wp = (_mx.BF16, None) if weight is None else (_type(weight), _dense(weight, (D,), weight.dtype, dev))
    rp, ld_res = (None, 0) if dres is None else _rows(dres, shape, dtype, dev)
    mp, sdp = _dense(mean, (R,), _F32, dev), _dense(rstd, (R,), _F32, dev)
    assert not accumulate or ((dweight is not None or not wgrad) and (dbias is not None or not bias)), \
        "accumulate needs the buffers to add to"
    if dx is None:
        dx = _new(shape, dtype, x, stream)
        dxp, ld_dx = dx.data_ptr(), D
    else:
        dxp, ld_dx = _rows(dx, shape, dtype, dev)
    dwp = dbp = None
    if dweight is not None:
        dwp = _dense(dweight, (D,), _F32, dev)
    elif wgrad:
        dweight = _new(D, _F32, x, stream)
        dwp = dweight.data_ptr()
    if dbias is not None:
        dbp = _dense(dbias, (D,), _F32, dev)
    elif bias:
        dbias = _new(D, _F32, x, stream)
        dbp = dbias.data_ptr()
    nbytes = 0 if dwp is None and dbp is None else mx_layernorm_workspace_bytes(R, D)
    workspace, wsp, nbytes = _workspace(workspace, nbytes, x, dev, stream)
    _mx._check(_mx.load().mx_layernorm_bwd(dyp, ld_dy, xp, xt, R, D, ld_x, mp, sdp, wp, wt, 1 if rms else 0, rp, ld_res,
                                           dxp, ld_dx, dwp, dbp, 1 if accumulate else 0, wsp, nbytes,
                                           _mx._stream(stream)))
    return dx, dweight, dbias


# --------------------------------------------------------------------------
# Expert routing and the combine's gradient
# --------------------------------------------------------------------------

@functools.lru_cache(maxsize=256)
def mx_moe_topk_workspace_bytes(T, G):
    return int(_mx.load().mx_moe_topk_workspace_bytes(T, G))


def mx_moe_topk(logits, k, score=_mx.SCORE_SOFTMAX, bias=None, groups=1, topk_groups=1, group_top=1, renorm=True,
                scale=1.0, stats=False, weights=None, ids=None, load=None, score_sum=None, workspace=None, stream=None):
    """The k experts of each token from its logits (BF16 or fp32 [T, G]) and
    their weights: returns (weights fp32 [T, k], ids int32 [T, k], load, score_sum),
    the last two (choices of each expert, sums of its scores) None without stats."""
    shape, dev = logits.shape, _gpu(logits)
    T, G = shape
    xt = _type(logits)
    xp, ld = _rows(logits, shape, logits.dtype, dev)
    bp = _dense(bias, (G,), _F32, dev)
    if weights is None:
        weights = _new((T, k), _F32, logits, stream)
        wp = weights.data_ptr()
    else:
        wp = _dense(weights, (T, k), _F32, dev)
    if ids is None:
        ids = _new((T, k), _I32, logits, stream)
        ip = ids.data_ptr()
    else:
        ip = _dense(ids, (T, k), _I32, dev)
    lp = sp = wsp = None
    nbytes = 0
    if stats or load is not None or score_sum is not None:
        load = load if load is not None else _new(G, _I32, logits, stream)
        score_sum = score_sum if score_sum is not None else _new(G, _F32, logits, stream)
        lp, sp = _dense(load, (G,), _I32, dev), _dense(score_sum, (G,), _F32, dev)
        workspace, wsp, nbytes = _workspace(workspace, mx_moe_topk_workspace_bytes(T, G), logits, dev, stream)
    _mx._check(_mx.load().mx_moe_topk(xp, xt, T, G, ld, k, score, bp, groups, topk_groups, group_top, 1 if renorm else 0,
                                      scale, wp, ip, lp, sp, wsp, nbytes, _mx._stream(stream)))
    return weights, ids, load, score_sum


def mx_moe_topk_bwd(logits, ids, dweights, score=_mx.SCORE_SOFTMAX, renorm=True, scale=1.0, dscore_sum=None,
                    dlogits=None, stream=None):
    """The logits' gradient (of their type) from that of the weights, and of
    score_sum where dscore_sum is given."""
    shape, dev, dtype = logits.shape, _gpu(logits), logits.dtype
    T, G = shape
    k = ids.shape[1]
    xt = _type(logits)
    xp, ld = _rows(logits, shape, dtype, dev)
    ip, ap, sp = _dense(ids, (T, k), _I32, dev), _dense(dweights, (T, k), _F32, dev), _dense(dscore_sum, (G,), _F32, dev)
    if dlogits is None:
        dlogits = _new(shape, dtype, logits, stream)
        dp, ld_d = dlogits.data_ptr(), G
    else:
        dp, ld_d = _rows(dlogits, shape, dtype, dev)
    _mx._check(_mx.load().mx_moe_topk_bwd(xp, xt, T, G, ld, k, score, 1 if renorm else 0, scale, ip, ap, sp, dp, ld_d,
                                          _mx._stream(stream)))
    return dlogits


def mx_moe_unpermute_bwd(dout, inp, row_of, weights=None, src=None, din=None, dweights=None, stream=None):
    """The gradient of mx_moe_unpermute(inp, row_of, weights): returns (din, dweights),
    din[row_of[t, j]] = weights[t, j] dout[t] and dweights[t, j] = <dout[t], inp[row_of[t, j]]>.
    src (mx_moe_route_index's): the empty rows of din are zeroed; rows that
    neither names are left as they were."""
    dev = _gpu(dout)
    T, D = dout.shape
    R, k = inp.shape[0], row_of.shape[1]
    op, xp, rp = _dense(dout, (T, D), _BF16, dev), _dense(inp, (R, D), _BF16, dev), _dense(row_of, (T, k), _I32, dev)
    wp, sp = _dense(weights, (T, k), _F32, dev), _dense(src, (R,), _I32, dev)
    if din is None:
        din = _new((R, D), _BF16, dout, stream)
        dp = din.data_ptr()
    else:
        dp = _dense(din, (R, D), _BF16, dev)
    if dweights is None:
        dweights = _new((T, k), _F32, dout, stream)
        gp = dweights.data_ptr()
    else:
        gp = _dense(dweights, (T, k), _F32, dev)
    _mx._check(_mx.load().mx_moe_unpermute_bwd(op, T, D, xp, R, rp, k, wp, sp, dp, gp, _mx._stream(stream)))
    return din, dweights


# --------------------------------------------------------------------------
# 4-bit tensors with a scale for every 16 values
# --------------------------------------------------------------------------

@functools.lru_cache(maxsize=256)
def nvfp4_scale_bytes(rows, cols):
    return int(_mx.load().mx_nvfp4_scale_bytes(rows, cols))


class NVFP4:
    """A 4-bit tensor [rows, cols] in torch buffers: `data`, packed E2M1 codes (uint8
    [rows, cols / 2]), `scale`, E4M3 scales per 16 values in the blocked layout
    (uint8), `row_scale`, fp32 of each row (None as an operand: ones).  Without buffers
    of the caller's the three are views of one allocation, made when they are asked
    for; stream: the one that fills them, where that is not the current one."""

    def __init__(self, rows, cols, device="cuda", data=None, scale=None, row_scale=None, stream=None):
        self.rows, self.cols = rows, cols = int(rows), int(cols)
        self._buffer, self._own = None, None
        if data is None:
            assert scale is None and row_scale is None, "scales without codes"
            self._sizes = rows * cols // 2, nvfp4_scale_bytes(rows, cols), 4 * rows
            at = (self._sizes[0] + 15) // 16 * 16
            self._at = 0, at, at + self._sizes[1]    # the scales are whole blocks of 512 bytes
            nbytes = self._at[2] + self._sizes[2]
            self._buffer = torch.empty(nbytes, dtype=_U8, device=device) if stream is None else \
                _mx._empty(nbytes, _U8, device, stream)
        else:
            if scale is None:
                scale = _mx._empty(nvfp4_scale_bytes(rows, cols), _U8, device, stream)
            self._own = [data, scale, row_scale]

    def _parts(self):
        if self._own is None:
            d, s, r = (self._buffer[a:a + n] for a, n in zip(self._at, self._sizes))
            self._own = [d.view(self.rows, self.cols // 2), s, r.view(_F32)]
        return self._own

    def _set(self, i, value):
        self._parts()[i] = value

    data = property(lambda self: self._parts()[0], lambda self, v: self._set(0, v))
    scale = property(lambda self: self._parts()[1], lambda self, v: self._set(1, v))
    row_scale = property(lambda self: self._parts()[2], lambda self, v: self._set(2, v))

    def struct(self):
        return _fp4(self, self._parts()[0].get_device())


def _fp4_first(t):
    return t._buffer if t._own is None else t._own[0]


def _fp4(t, dev):
    """A 4-bit tensor's structure; its buffers are dense, as large as its shape needs
    and on this GPU."""
    if t._own is None:
        assert t._buffer.get_device() == dev, "a 4-bit tensor on another GPU"
        p, at = t._buffer.data_ptr(), t._at
        return _mx.Nvfp4Struct(p, p + at[1], p + at[2], t.rows, t.cols)
    data, scale, row = t._own
    assert data.is_contiguous() and data.nbytes >= t.rows * (t.cols // 2) and data.get_device() == dev, \
        "the codes are strided, too few or on another GPU"
    assert scale.is_contiguous() and scale.nbytes >= nvfp4_scale_bytes(t.rows, t.cols) and scale.get_device() == dev, \
        "the scales are strided, too few or on another GPU"
    return _mx.Nvfp4Struct(data.data_ptr(), scale.data_ptr(), _dense(row, (t.rows,), _F32, dev), t.rows, t.cols)


@functools.lru_cache(maxsize=256)
def mx_nvfp4_quantize_workspace_bytes(T, K, R):
    return int(_mx.load().mx_nvfp4_quantize_workspace_bytes(T, K, R))


def mx_nvfp4_quantize(x, src=None, offsets=None, out=None, workspace=None, stream=None):
    """BF16 rows [T, K] as a 4-bit tensor; src int32 [R]: row r is x's row src[r],
    zeros where that is negative; offsets: rows from offsets[-1] on are not produced."""
    shape, dev = x.shape, _gpu(x)
    T, K = shape
    xp, ld = _rows(x, shape, _BF16, dev)
    R = T if src is None else src.numel()
    sp = _dense(src, (R,), _I32, dev)
    G = 0 if offsets is None else offsets.numel()
    op = _dense(offsets, (G,), _I32, dev)
    if out is None:
        out = NVFP4(R, K, x.device, stream=stream)
    assert out.rows == R and out.cols == K, "a result of another shape"
    nbytes = 0 if src is None else mx_nvfp4_quantize_workspace_bytes(T, K, R)
    workspace, wsp, nbytes = _workspace(workspace, nbytes, x, dev, stream)
    _mx._check(_mx.load().mx_nvfp4_quantize(xp, T, K, ld, sp, op, G, ctypes.byref(_fp4(out, dev)), wsp, nbytes,
                                            _mx._stream(stream)))
    return out


def mx_nvfp4_gemm(a, b, G=1, offsets=None, out=None, stream=None):
    """out[r] = a[r] b[g(r)]^T in BF16 from 4-bit operands a [R, K], b [G * N, K];
    rows past the last segment are not written."""
    first = _fp4_first(a)
    dev = _gpu(first)
    R, N = a.rows, b.rows // G if G > 0 else 0
    if out is None:
        out = _new((R, N), _BF16, first, stream)
        yp, ld = out.data_ptr(), N
    else:
        yp, ld = _rows(out, (R, N), _BF16, dev)
    op = _dense(offsets, (G,), _I32, dev)
    _mx._check(_mx.load().mx_nvfp4_gemm(ctypes.byref(_fp4(a, dev)), ctypes.byref(_fp4(b, dev)), G, op, yp, ld,
                                        _mx._stream(stream)))
    return out
