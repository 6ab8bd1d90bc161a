"""Cases of the BF16 expert-MLP operators: ragged grouped products and their
weight gradients, the linear layer with bias, activation and residual, and
8-bit activation checkpoints with the backward pass that reads them.

``run`` computes each in its plain form (elementary torch operations in fp32,
rounded once) where ``own`` is false, and calls the library where it is true.
"""
import math

import torch

own = False

BLOCK = 32  # elements that share one E8M0 scale


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # One token through 8 of 128 experts (the FC1 of the 128-expert
        # configuration): latency and the bandwidth of 8 weight matrices.
        {"name": "ragged fwd 1 token", "op": "gemm", "R": 8, "G": 128, "K": 2048, "N": 1536, "layout": "NK",
         "routing": "one"},
        # A decode batch of 61 tokens, 8 choices each: nearly every expert's
        # weights are read for a handful of rows.
        {"name": "ragged fwd 61 tokens", "op": "gemm", "R": 488, "G": 128, "K": 2048, "N": 1536, "layout": "NK",
         "routing": "uniform"},
        # A training batch of 8192 tokens, 8 choices each, skewed routing.
        {"name": "ragged fwd train", "op": "gemm", "R": 65536, "G": 128, "K": 2048, "N": 1536, "layout": "NK",
         "routing": "zipf"},
        # The input gradient of the same layer (its FC1, dX = dZ W1), a
        # batch whose length is no multiple of anything.
        {"name": "ragged dgrad train", "op": "gemm", "R": 65521, "G": 128, "K": 1536, "N": 2048, "layout": "KN",
         "routing": "zipf"},
        # Its weight gradient: long and short experts, some without a token.
        {"name": "ragged wgrad train", "op": "wgrad", "R": 65536, "G": 128, "N": 1536, "K": 2048, "out": "bf16",
         "routing": "zipf"},
        # A microbatch of a small layer, added into an fp32 main gradient.
        {"name": "ragged wgrad accumulate", "op": "wgrad", "R": 2777, "G": 8, "N": 1000, "K": 520, "out": "f32",
         "routing": "uniform"},
        # One token through a dense up projection: a weight matrix is read once.
        {"name": "linear 1 token", "op": "linear", "M": 1, "K": 4096, "N": 16384, "act": "gelu", "bias": True,
         "res": False, "ckpt": False},
        # A short prompt through a down projection with its residual.
        {"name": "linear 777 residual", "op": "linear", "M": 777, "K": 5120, "N": 2048, "act": "none", "bias": True,
         "res": True, "ckpt": False},
        # A training batch through the up projection, the pre-activation
        # saved in 8 bits for the backward pass.
        {"name": "linear train checkpoint", "op": "linear", "M": 16384, "K": 2048, "N": 8192, "act": "gelu",
         "bias": True, "res": False, "ckpt": True},
        # SwiGLU between the expert layer's products, saving its input in 8 bits.
        {"name": "checkpoint save swiglu", "op": "save", "R": 65536, "C": 1536, "act": "swiglu"},
        # Its backward pass from the 8-bit copy, the activation recomputed
        # for the second product's weight gradient.
        {"name": "checkpoint bwd swiglu", "op": "bwd", "R": 65536, "C": 1536, "act": "swiglu", "h": True, "db": False},
        # The dense layer's backward pass with the bias gradient, a short batch.
        {"name": "checkpoint bwd gelu bias", "op": "bwd", "R": 333, "C": 8192, "act": "gelu", "h": False, "db": True},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    kind = rng.choice(["gemm", "gemm", "wgrad", "linear", "linear", "save", "bwd"])
    if kind in ("gemm", "wgrad"):
        R = _log_int(rng, 1 if kind == "gemm" else 64, 65536)
        G = rng.choice([1, 4, 8, 32, 64, 128])
        N, K = _log_int(rng, 64, 2048, 8), _log_int(rng, 64, 2048, 8)
        if kind == "gemm":
            return {"op": "gemm", "R": R, "G": G, "K": K, "N": N, "layout": rng.choice(["NK", "KN"]),
                    "routing": rng.choice(["uniform", "zipf"])}
        return {"op": "wgrad", "R": R, "G": G, "N": N, "K": K, "out": rng.choice(["bf16", "f32"]),
                "routing": rng.choice(["uniform", "zipf"])}
    if kind == "linear":
        return {"op": "linear", "M": _log_int(rng, 1, 16384), "K": _log_int(rng, 64, 4096, 8),
                "N": _log_int(rng, 64, 4096, 32), "act": rng.choice(["none", "gelu", "silu", "relu"]),
                "bias": rng.random() < 0.7, "res": rng.random() < 0.5, "ckpt": rng.random() < 0.4}
    act = rng.choice(["swiglu", "gelu", "silu", "relu"])
    C = _log_int(rng, 64, 8192, 64)
    R = min(_log_int(rng, 1, 65536), (65536 * 1536) // C)
    if kind == "save":
        return {"op": "save", "R": R, "C": C, "act": act}
    return {"op": "bwd", "R": R, "C": C, "act": act, "h": rng.random() < 0.5, "db": rng.random() < 0.5}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _counts(R, G, routing, gen):
    """Rows of each expert, as a list: "one" gives min(R, G) experts one row
    each, "uniform" draws an expert per row, "zipf" draws by rank^-1.1 with
    the last sixteenth of the experts left empty."""
    if routing == "one":
        c = torch.zeros(G, dtype=torch.int64)
        c[torch.randperm(G, generator=gen)[:min(R, G)]] = R // min(R, G)
        c[int(c.argmax())] += R - int(c.sum())
        return c.tolist()
    p = torch.ones(G) if routing == "uniform" else torch.arange(1, G + 1, dtype=torch.float32) ** -1.1
    if routing == "zipf" and G >= 16:
        p[G - G // 16:] = 0
    ids = torch.multinomial(p, R, replacement=True, generator=gen)
    return torch.bincount(torch.randperm(G, generator=gen)[ids], minlength=G).tolist()


def _normal(shape, gen, std=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return x.normal_(0.0, std, generator=gen)


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op in ("gemm", "wgrad"):
        R, G, N, K = case["R"], case["G"], case["N"], case["K"]
        s["counts"] = _counts(R, G, case["routing"], cpu)
        s["offsets"] = torch.tensor(s["counts"], dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
    if op == "gemm":
        s["a"] = _normal((R, K), gen)
        s["w"] = _normal((G, N, K) if case["layout"] == "NK" else (G, K, N), gen, 0.02)
        s["out"] = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    elif op == "wgrad":
        s["x"] = _normal((R, K), gen)
        s["dy"] = _normal((R, N), gen, 1e-3)
        if case["out"] == "f32":
            s["grad"] = torch.empty((G, N, K), device="cuda").normal_(0.0, 1e-2, generator=gen)
        else:
            s["grad"] = torch.empty((G, N, K), dtype=torch.bfloat16, device="cuda")
    elif op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = _normal((M, K), gen)
        s["w"] = _normal((N, K), gen, 0.02)
        s["bias"] = _normal((N,), gen, 0.02) if case["bias"] else None
        s["res"] = _normal((M, N), gen) if case["res"] else None
    elif op == "save":
        s["z"] = _normal((case["R"], case["C"]), gen)
    else:
        z = _normal((case["R"], case["C"]), gen)
        s["ckpt"] = _checkpoint(z.float())
        s["dh"] = _normal((case["R"], case["C"] // 2 if case["act"] == "swiglu" else case["C"]), gen, 1e-3)
    return s


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------

def _to_blocked(m):
    """Scale bytes [rows, cols/32] in the tensor cores' blocked order: chunks
    of 128 rows x 4 scales, padding zero."""
    r, c = m.shape
    m = torch.nn.functional.pad(m, (0, -c % 4, 0, -r % 128))
    m = m.view(m.shape[0] // 128, 4, 32, m.shape[1] // 4, 4)
    return m.permute(0, 3, 2, 1, 4).reshape(-1)


def _from_blocked(b, rows, cols):
    m = b.view((rows + 127) // 128, (cols + 127) // 128, 32, 4, 4).permute(0, 3, 2, 1, 4)
    return m.reshape((rows + 127) // 128 * 128, -1)[:rows, :cols // BLOCK]


def _checkpoint(z):
    """fp32 z -> (E4M3 payload, E8M0 scale bytes in blocked order): each
    block's scale is the smallest power of two with amax <= 448 * scale."""
    r, c = z.shape
    b = z.view(r, c // BLOCK, BLOCK)
    mant, exp = torch.frexp(b.abs().amax(-1))
    e = (exp - 9 + (mant > 0.875).to(exp.dtype)).clamp(-127, 127)
    e = torch.where(mant == 0, torch.full_like(e, -127), e)
    q = torch.ldexp(b, -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.view(r, c), _to_blocked((e + 127).to(torch.uint8))


def _read(ckpt):
    q, s = ckpt
    r, c = q.shape
    e = _from_blocked(s, r, c).to(torch.int32) - 127
    return torch.ldexp(q.float().view(r, c // BLOCK, BLOCK), e.unsqueeze(-1)).view(r, c)


_GELU_A, _GELU_B = math.sqrt(2.0 / math.pi), 0.044715


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "swiglu":
        g, u = z.chunk(2, dim=-1)
        return g / (1.0 + torch.exp(-g)) * u
    return 0.5 * z * (1.0 + torch.tanh(_GELU_A * (z + _GELU_B * z * z * z)))


def _act_bwd(z, dh, act):
    if act == "relu":
        return torch.where(z > 0, dh, torch.zeros_like(dh))
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return dh * s * (1.0 + z * (1.0 - s))
    if act == "swiglu":
        g, u = z.chunk(2, dim=-1)
        s = 1.0 / (1.0 + torch.exp(-g))
        return torch.cat([dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s], dim=-1)
    t = torch.tanh(_GELU_A * (z + _GELU_B * z * z * z))
    return dh * (0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _GELU_A * (1.0 + 3.0 * _GELU_B * z * z))


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "gemm":
        w = s["w"].transpose(1, 2) if case["layout"] == "NK" else s["w"]
        return torch.cat([(a.float() @ b.float()).to(torch.bfloat16)
                          for a, b in zip(s["a"].split(s["counts"]), w.unbind()) if a.shape[0]])
    if op == "wgrad":
        dw = torch.stack([d.float().T @ x.float()
                          for d, x in zip(s["dy"].split(s["counts"]), s["x"].split(s["counts"]))])
        return s["grad"].add_(dw) if case["out"] == "f32" else dw.to(torch.bfloat16)
    if op == "linear":
        z = s["x"].float() @ s["w"].float().T
        z = z if s["bias"] is None else z + s["bias"].float()
        h = _act(z, case["act"])
        out = (h if s["res"] is None else h + s["res"].float()).to(torch.bfloat16)
        if not case["ckpt"]:
            return out
        q, e = _checkpoint(z)
        return out, q, e.view(torch.float8_e8m0fnu)
    if op == "save":
        z = s["z"].float()
        q, e = _checkpoint(z)
        return _act(z, case["act"]).to(torch.bfloat16), q, e
    z = _read(s["ckpt"])
    dz = _act_bwd(z, s["dh"].float(), case["act"])
    return (dz.to(torch.bfloat16), _act(z, case["act"]).to(torch.bfloat16) if case["h"] else None,
            dz.sum(0) if case["db"] else None)


# --------------------------------------------------------------------------
# The library's calls
# --------------------------------------------------------------------------

def _library(s):
    import mlp_gemms_gb300 as mx
    case = s["case"]
    op = case["op"]
    if op == "gemm":
        return mx.mx_ragged_gemm(s["a"], s["w"], s["offsets"], layout=mx.W_NK if case["layout"] == "NK" else mx.W_KN,
                                 out=s["out"])
    if op == "wgrad":
        if case["out"] == "f32":
            return mx.mx_ragged_gemm_wgrad_f32(s["dy"], s["x"], case["G"], s["offsets"], s["grad"], accumulate=True)
        return mx.mx_ragged_gemm_wgrad(s["dy"], s["x"], case["G"], s["offsets"], out=s["grad"])
    act = {"swiglu": mx.ACT_SWIGLU, "gelu": mx.ACT_GELU_TANH, "none": mx.ACT_NONE, "silu": mx.ACT_SILU,
           "relu": mx.ACT_RELU}[case["act"]]
    if op == "linear":
        ck = mx.MX(case["M"], case["N"], mx.E4M3) if case["ckpt"] else None
        out = mx.mx_linear_fwd(s["x"], s["w"], s["bias"], act, s["res"], ckpt=ck)
        if ck is None:
            return out
        return out, ck.data.view(torch.float8_e4m3fn), ck.scale.view(torch.float8_e8m0fnu)
    if op == "save":
        h, ck = mx.mx_act_ckpt_fwd(s["z"], act)
        return h, ck.data.view(torch.float8_e4m3fn), ck.scale
    q, e = s["ckpt"]
    ck = mx.MX(case["R"], case["C"], mx.E4M3, data=q.view(torch.uint8), scale=e)
    return mx.mx_act_ckpt_bwd(ck, act, s["dh"], recompute=case["h"], colsum=case["db"])


def run(state):
    return _library(state) if own else _plain(state)


# --------------------------------------------------------------------------
# Work and definition
# --------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("gemm", "wgrad"):
        R, G, N, K = case["R"], case["G"], case["N"], case["K"]
        used = sum(1 for c in _counts(R, G, case["routing"], torch.Generator().manual_seed(0)) if c)
        if op == "gemm":
            return {"bytes": 2 * (R * K + used * N * K + R * N), "flops": 2 * R * N * K}
        return {"bytes": 2 * R * (N + K) + (8 if case["out"] == "f32" else 2) * G * N * K, "flops": 2 * R * N * K}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        b = 2 * (M * K + N * K + M * N) + (2 * N if case["bias"] else 0) + (2 * M * N if case["res"] else 0)
        return {"bytes": b + (M * N + M * N // BLOCK if case["ckpt"] else 0), "flops": 2 * M * N * K}
    R, C = case["R"], case["C"]
    H = C // 2 if case["act"] == "swiglu" else C
    ck = R * C + R * C // BLOCK
    if op == "save":
        return {"bytes": 2 * R * C + 2 * R * H + ck, "flops": 10 * R * C}
    return {"bytes": ck + 2 * R * H + 2 * R * C + (2 * R * H if case["h"] else 0) + (4 * C if case["db"] else 0),
            "flops": 20 * R * C}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = torch.float64
    if op in ("gemm", "wgrad"):
        R, G, N, K = case["R"], case["G"], case["N"], case["K"]
        if op == "gemm":
            out = torch.zeros((R, N), dtype=d, device="cuda")
        else:
            out = s["grad"].to(d) if case["out"] == "f32" else torch.zeros((G, N, K), dtype=d, device="cuda")
        ends = s["offsets"].tolist()
        begin = 0
        for g, end in enumerate(ends):
            if op == "gemm" and end > begin:
                spec = "rk,nk->rn" if case["layout"] == "NK" else "rk,kn->rn"
                out[begin:end] = torch.einsum(spec, s["a"][begin:end].to(d), s["w"][g].to(d))
            elif op == "wgrad" and end > begin:
                out[g] += torch.einsum("rn,rk->nk", s["dy"][begin:end].to(d), s["x"][begin:end].to(d))
            begin = end
        return out

    def f(z, act):
        if act == "none":
            return z
        if act == "relu":
            return z * (z > 0)
        if act == "silu":
            return z * torch.special.expit(z)
        return z * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))

    def slope(z, act):
        if act == "relu":
            return (z > 0).to(d)
        a = 1.0 if act == "silu" else 2.0 * math.sqrt(2.0 / math.pi)
        b = 0.0 if act == "silu" else 0.044715
        p = torch.special.expit(a * (z + b * z ** 3))
        return p + z * p * (1.0 - p) * a * (1.0 + 3.0 * b * z * z)

    if op == "linear":
        z = torch.einsum("mk,nk->mn", s["x"].to(d), s["w"].to(d))
        if case["bias"]:
            z += s["bias"].to(d)
        out = f(z, case["act"])
        if case["res"]:
            out = out + s["res"].to(d)
        return (out, None, None) if case["ckpt"] else out
    if op == "save":
        z = s["z"].to(d)
        if case["act"] == "swiglu":
            return f(z[:, :case["C"] // 2], "silu") * z[:, case["C"] // 2:], None, None
        return f(z, case["act"]), None, None
    q, b = s["ckpt"]
    rows = torch.arange(case["R"], device="cuda").unsqueeze(1)
    cols = torch.arange(case["C"], device="cuda").unsqueeze(0) // BLOCK
    per = (case["C"] + 127) // 128
    at = (rows // 128 * per + cols // 4) * 512 + rows % 32 * 16 + rows % 128 // 32 * 4 + cols % 4
    z = q.to(d) * torch.exp2(b[at].to(d) - 127.0)
    dh = s["dh"].to(d)
    if case["act"] == "swiglu":
        g, u = z[:, :case["C"] // 2], z[:, case["C"] // 2:]
        dz = torch.cat([dh * u * slope(g, "silu"), dh * f(g, "silu")], 1)
        h = f(g, "silu") * u
    else:
        dz, h = dh * slope(z, case["act"]), f(z, case["act"])
    return dz, h if case["h"] else None, dz.sum(0) if case["db"] else None
