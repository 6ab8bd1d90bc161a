"""Cases of the operators in front of, between and behind the expert MLP's
products: the layer norm, the expert routing, the combine's gradient, and
products of tensors held in 4 bits with a scale for every 16 values.

``run`` computes each in its plain form (elementary torch operations in fp32,
rounded once; the routing's order in 64 bits) where ``own`` is false, and calls
the library where it is true.
"""
import math

import torch

own = False

BLOCK = 16  # elements that share one E4M3 scale
F4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # E2M1 magnitudes


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # One decoded token in front of a layer, the previous layer's output
        # added to the residual stream in the same pass: latency.
        {"name": "norm 1 token residual", "op": "norm", "R": 1, "D": 7168, "x": "bf16", "res": True, "rms": False,
         "bias": True},
        # The norm of a training batch in front of the expert layer.
        {"name": "norm train", "op": "norm", "R": 65536, "D": 2048, "x": "bf16", "res": False, "rms": False,
         "bias": True},
        # Its backward pass for a short batch of a wide layer, the residual
        # stream's own gradient added.
        {"name": "norm bwd 333 rows", "op": "norm_bwd", "R": 333, "D": 8192, "x": "bf16", "res": True, "rms": False,
         "bias": True},
        # The backward pass of a training batch whose residual stream is kept
        # in fp32.
        {"name": "norm bwd train f32", "op": "norm_bwd", "R": 32768, "D": 4096, "x": "f32", "res": True,
         "rms": False, "bias": True},
        # A decode batch routed by sigmoid scores, a balancing bias and groups
        # of experts.
        {"name": "route 61 tokens groups", "op": "route", "T": 61, "G": 256, "k": 8, "score": "sigmoid", "x": "f32",
         "bias": True, "groups": 8, "topk_groups": 4, "group_top": 2, "renorm": True, "stats": False, "masked": False},
        # A training batch over 128 experts, 8 choices, with the sums that a
        # balancing loss takes.
        {"name": "route train", "op": "route", "T": 32768, "G": 128, "k": 8, "score": "softmax", "x": "bf16",
         "bias": False, "groups": 1, "topk_groups": 1, "group_top": 1, "renorm": True, "stats": True, "masked": False},
        # The gradients of both.
        {"name": "route bwd 777 sigmoid", "op": "route_bwd", "T": 777, "G": 256, "k": 8, "score": "sigmoid",
         "x": "f32", "renorm": True, "stats": False, "masked": False},
        {"name": "route bwd train", "op": "route_bwd", "T": 32768, "G": 128, "k": 8, "score": "softmax", "x": "bf16",
         "renorm": True, "stats": True, "masked": False},
        # The gradient of the experts' weighted sum: of the experts' outputs
        # and of the routing weights, a small batch and a training batch.
        {"name": "combine bwd 61 tokens", "op": "combine_bwd", "T": 61, "G": 128, "k": 8, "D": 2048, "pad": 1},
        {"name": "combine bwd train", "op": "combine_bwd", "T": 8192, "G": 128, "k": 8, "D": 2048, "pad": 1},
        # One token through an up projection whose weights are held in 4 bits.
        {"name": "fp4 linear 1 token", "op": "fp4", "T": 1, "G": 1, "k": 1, "K": 4096, "N": 16384},
        # A prompt of 8192 tokens through the first product of 128 experts, 8
        # choices each: tokens gathered and quantized, then the product.
        {"name": "fp4 experts prefill", "op": "fp4", "T": 8192, "G": 128, "k": 8, "K": 2048, "N": 1536},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "norm_bwd", "route", "route", "route_bwd", "combine_bwd", "fp4",
                     "fp4"])
    if op in ("norm", "norm_bwd"):
        D = _log_int(rng, 64, 16384, 8)
        x = rng.choice(["bf16", "bf16", "f32"])
        most = (65536 * 2048) // (D * (2 if x == "f32" else 1))
        return {"op": op, "R": min(_log_int(rng, 1, 65536), most), "D": D, "x": x, "res": rng.random() < 0.5,
                "rms": rng.random() < 0.4, "bias": rng.random() < 0.6}
    if op in ("route", "route_bwd"):
        G = rng.choice([8, 16, 32, 60, 64, 100, 128, 128, 160, 256, 256, 384, 512])
        T = min(_log_int(rng, 1, 32768), (32768 * 128) // G)
        case = {"op": op, "T": T, "G": G, "k": rng.randint(1, min(10, G // 4)), "score": rng.choice(["softmax", "sigmoid"]),
                "x": rng.choice(["bf16", "f32"])}
        if op == "route":
            case["bias"] = rng.random() < 0.5
            groups = rng.choice([1, 4, 8]) if G % 8 == 0 and G >= 64 else 1
            case.update(groups=groups, topk_groups=groups if groups == 1 else groups // 2 + rng.randint(0, 1),
                        group_top=rng.choice([1, 2]))
        case.update(renorm=rng.random() < 0.7, stats=rng.random() < 0.5, masked=rng.random() < 0.3)
        return case
    if op == "combine_bwd":
        D, k = _log_int(rng, 64, 8192, 8), rng.choice([1, 2, 4, 6, 8])
        return {"op": op, "T": min(_log_int(rng, 1, 32768), (8192 * 8 * 2048) // (D * k)),
                "G": rng.choice([8, 32, 64, 128]), "k": k, "D": D, "pad": rng.choice([1, 128])}
    if rng.random() < 0.5:
        return {"op": "fp4", "T": _log_int(rng, 1, 8192), "G": 1, "k": 1, "K": _log_int(rng, 64, 8192, 32),
                "N": _log_int(rng, 64, 8192, 8)}
    return {"op": "fp4", "T": _log_int(rng, 1, 8192), "G": rng.choice([8, 32, 64, 128]), "k": rng.choice([1, 2, 4, 8]),
            "K": _log_int(rng, 128, 2048, 32), "N": _log_int(rng, 128, 1536, 128)}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _normal(shape, gen, std=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _dtype(case):
    return torch.bfloat16 if case["x"] == "bf16" else torch.float32


def _logits(case, gen):
    """Router logits: experts of different popularity, and (masked) an eighth
    of each token's experts closed."""
    T, G = case["T"], case["G"]
    x = _normal((T, G), gen, 1.5, torch.float32) + _normal((G,), gen, 0.5, torch.float32)
    if case["masked"]:
        x.masked_fill_(torch.rand((T, G), device="cuda", generator=gen) < 0.125, -math.inf)
    return x.to(_dtype(case))


def _segments(T, G, k, pad, gen):
    """A routing of T tokens to k of G experts: (row of each choice, source
    token of each row or -1, ends of the experts' rows), each expert's rows
    padded to a multiple of `pad`, in a buffer that every routing fits."""
    if G == 1:
        return None, None, None
    popular = _normal((G,), gen, 0.7, torch.float32)
    ids = torch.topk(popular + _normal((T, G), gen, 1.0, torch.float32), k).indices.reshape(-1)
    counts = torch.bincount(ids, minlength=G)
    padded = (counts + pad - 1) // pad * pad
    ends = padded.cumsum(0)
    order = torch.argsort(ids, stable=True)
    rows = torch.empty_like(ids)
    rows[order] = (ends - padded - counts.cumsum(0) + counts)[ids[order]] + torch.arange(T * k, device="cuda")
    capacity = (T * k + (pad - 1) * G + pad - 1) // pad * pad
    src = torch.full((capacity,), -1, dtype=torch.int32, device="cuda")
    src[rows] = (torch.arange(T * k, device="cuda") // k).to(torch.int32)
    return rows.view(T, k).to(torch.int32), src, ends.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        R, D = case["R"], case["D"]
        # channels of different size around a mean of their own
        s["x"] = (_normal((R, D), gen, 1.0, torch.float32) * (0.5 + torch.rand(D, device="cuda", generator=gen))
                  + _normal((D,), gen, 0.3, torch.float32)).to(_dtype(case))
        s["w"] = (1.0 + _normal((D,), gen, 0.1, torch.float32)).to(torch.bfloat16)
        s["b"] = _normal((D,), gen, 0.1) if case["bias"] else None
        s["res"] = _normal((R, D), gen, 1.0 if op == "norm" else 1e-3, _dtype(case)) if case["res"] else None
        if op == "norm_bwd":
            s["dy"] = _normal((R, D), gen, 1e-3)
            s["mean"], s["rstd"] = _statistics(s["x"].float(), case["rms"])
    elif op in ("route", "route_bwd"):
        T, G, k = case["T"], case["G"], case["k"]
        s["logits"] = _logits(case, gen)
        if op == "route":
            s["bias"] = _normal((G,), gen, 0.05, torch.float32) if case["bias"] else None
        else:
            s["ids"] = _order(s["logits"].double())[:, :k].to(torch.int32).contiguous()
            s["dweights"] = _normal((T, k), gen, 1e-2, torch.float32)
            s["dsum"] = _normal((G,), gen, 1e-3, torch.float32) if case["stats"] else None
    elif op == "combine_bwd":
        T, k, D = case["T"], case["k"], case["D"]
        s["row_of"], s["src"], _ = _segments(T, case["G"], k, case["pad"], gen)
        s["in"] = _normal((s["src"].numel(), D), gen, 0.5)
        s["in"][s["src"] < 0] = 0
        s["w"] = torch.softmax(_normal((T, k), gen, 1.0, torch.float32), -1)
        s["dout"] = _normal((T, D), gen, 1e-3)
    else:
        T, G, K, N = case["T"], case["G"], case["K"], case["N"]
        s["x"] = _normal((T, K), gen)
        _, s["src"], s["ends"] = _segments(T, G, case["k"], 128, gen)
        # the weights as a program keeps them: quantized once, packed
        codes, scale, row = _quantize(_normal((G * N, K), gen, 0.02).float())
        s["w"] = (codes[:, 0::2] | codes[:, 1::2] << 4, _to_blocked(scale.view(torch.uint8)), row)
        s["out"] = torch.zeros((T if G == 1 else s["src"].numel(), N), dtype=torch.bfloat16, device="cuda")
    return s


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------

EPS = 1e-5


def _statistics(x, rms):
    mean = None if rms else x.mean(-1)
    c = x if rms else x - mean.unsqueeze(1)
    return mean, torch.rsqrt((c * c).mean(-1) + EPS)


def _norm(s):
    case = s["case"]
    x = s["x"].float()
    if case["res"]:
        x = (x + s["res"].float()).to(_dtype(case))
        out, x = x, x.float()
    mean, rstd = _statistics(x, case["rms"])
    y = (x if case["rms"] else x - mean.unsqueeze(1)) * rstd.unsqueeze(1) * s["w"].float()
    y = y if s["b"] is None else y + s["b"].float()
    return y.to(torch.bfloat16), mean, rstd, out if case["res"] else None


def _norm_bwd(s):
    case = s["case"]
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"].unsqueeze(1)
    xhat = (x if case["rms"] else x - s["mean"].unsqueeze(1)) * rstd
    g = dy * s["w"].float()
    dx = g - xhat * (g * xhat).mean(-1, keepdim=True)
    dx = dx if case["rms"] else dx - g.mean(-1, keepdim=True)
    dx = dx * rstd if s["res"] is None else dx * rstd + s["res"].float()
    return (dx.to(_dtype(case)), (dy * xhat).sum(0, dtype=torch.float64).float(),
            dy.sum(0, dtype=torch.float64).float() if case["bias"] else None)


def _scores(x, kind):
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.max(-1, keepdim=True).values
    e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _order(v):
    """Indexes of each row's values, largest first, the lowest index first among equals."""
    return torch.sort(v, dim=-1, descending=True, stable=True).indices


def _ratio(a, b):
    return torch.where(b == 0, torch.zeros_like(a), a / torch.where(b == 0, torch.ones_like(b), b))


def _route(s):
    case, x = s["case"], s["logits"].float()
    T, G, k = case["T"], case["G"], case["k"]
    closed = x == -math.inf
    v = x.double() if s["bias"] is None else (_scores(x.double(), case["score"]) + s["bias"].double()).masked_fill(
        closed, -math.inf)
    if case["groups"] > 1:
        n = case["groups"]
        u = (_scores(x.double(), case["score"]).masked_fill(closed, -math.inf) if s["bias"] is None else v).view(T, n, -1)
        value = torch.sort(u, dim=-1, descending=True).values[..., :case["group_top"]].sum(-1)
        kept = torch.zeros((T, n), dtype=torch.bool, device="cuda").scatter_(1, _order(value)[:, :case["topk_groups"]], True)
        v = v.masked_fill(~kept.repeat_interleave(G // n, 1), -math.inf)
    ids = _order(v)[:, :k]
    p = _scores(x, case["score"])
    w = p.gather(1, ids)
    if case["renorm"]:
        w = _ratio(w, w.sum(-1, keepdim=True))
    if not case["stats"]:
        return w * 2.5, ids.to(torch.int32)
    if case["score"] == "sigmoid":
        p = _ratio(p, p.sum(-1, keepdim=True))
    return (w * 2.5, ids.to(torch.int32), torch.bincount(ids.reshape(-1), minlength=G).to(torch.int32),
            p.sum(0, dtype=torch.float64).float())


def _route_bwd(s):
    case, x = s["case"], s["logits"].float()
    p = _scores(x, case["score"])
    ids, a = s["ids"].long(), s["dweights"] * 2.5
    c = p.gather(1, ids)
    if case["renorm"]:
        total = c.sum(-1, keepdim=True)
        da = _ratio(a - (a * _ratio(c, total)).sum(-1, keepdim=True), total)
    else:
        da = a
    dp = torch.zeros_like(p).scatter_(1, ids, da)
    if case["score"] == "softmax":
        dp = dp if s["dsum"] is None else dp + s["dsum"]
        dx = p * (dp - (p * dp).sum(-1, keepdim=True))
    else:
        if case["stats"]:
            total = p.sum(-1, keepdim=True)
            dp = dp + _ratio(s["dsum"] - (s["dsum"] * _ratio(p, total)).sum(-1, keepdim=True), total)
        dx = dp * p / (1.0 + torch.exp(x))
    return dx.to(_dtype(case))


def _combine_bwd(s):
    rows, dout = s["row_of"].reshape(-1).long(), s["dout"].float()
    din = torch.zeros(s["in"].shape, dtype=torch.bfloat16, device="cuda")
    din[rows] = (s["w"].unsqueeze(2) * dout.unsqueeze(1)).to(torch.bfloat16).view(rows.numel(), -1)
    return din, (dout.unsqueeze(1) * s["in"][rows].float().view(*s["w"].shape, -1)).sum(-1)


def _quantize(x):
    """fp32 x [R, K] -> (E2M1 codes [R, K], E4M3 scales [R, K/16], power of two of
    each row): the row's is the smallest 2^e with amax <= 6 * 448 * 2^e, the
    block's the nearest to amax / 6, each value's code the nearest, of two
    equally near ones the even one."""
    b = x.view(x.shape[0], -1, BLOCK)
    amax = b.abs().amax(-1)
    mant, exp = torch.frexp(amax.amax(-1))
    exp = torch.where(mant == 0, -100, (exp - 12 + (mant > 0.65625).int()).clamp(min=-100))
    scale = (torch.ldexp(amax, -exp.unsqueeze(1)) / 6.0).to(torch.float8_e4m3fn)
    step = scale.float().unsqueeze(2)
    v = torch.ldexp(b, -exp.view(-1, 1, 1)) / torch.where(step == 0, torch.full_like(step, math.inf), step)
    a = v.abs()
    codes = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    codes = torch.where((v < 0) & (codes > 0), codes + 8, codes)
    return codes.to(torch.uint8).view(x.shape), scale, torch.ldexp(torch.ones_like(mant), exp)


def _to_blocked(m):
    """Scale bytes [rows, K/16] in the tensor cores' blocked order: chunks of 128
    rows x 4 scales, padding zero."""
    r, c = m.shape
    m = torch.nn.functional.pad(m, (0, -c % 4, 0, -r % 128))
    m = m.view(m.shape[0] // 128, 4, 32, m.shape[1] // 4, 4)
    return m.permute(0, 3, 2, 1, 4).reshape(-1)


def _from_blocked(b, rows, cols):
    m = b.view((rows + 127) // 128, (cols + 3) // 4, 32, 4, 4).permute(0, 3, 2, 1, 4)
    return m.reshape((rows + 127) // 128 * 128, -1)[:rows, :cols]


def _values(codes, scale):
    lut = torch.tensor(F4 + tuple(-v for v in F4), device="cuda")
    v = lut[codes.int()].view(codes.shape[0], -1, BLOCK)
    return (v * scale.float().unsqueeze(2)).view(codes.shape)


def _fp4(s):
    case = s["case"]
    x = s["x"].float()
    if s["src"] is not None:
        x = torch.where((s["src"] < 0).unsqueeze(1), 0.0, x[s["src"].clamp(min=0).long()])
    codes, scale, row = _quantize(x)
    a = _values(codes, scale)
    packed, blocked, wrow = s["w"]
    rows = case["G"] * case["N"]
    w = _values(torch.stack((packed & 15, packed >> 4), -1).view(rows, -1),
                _from_blocked(blocked, rows, case["K"] // BLOCK).contiguous().view(torch.float8_e4m3fn))
    w = w.view(case["G"], case["N"], -1)
    if s["ends"] is None:
        y = a @ w[0].T * wrow
    else:
        counts = s["ends"].diff(prepend=s["ends"].new_zeros(1)).tolist()
        a = a[:sum(counts)]
        y = torch.cat([p @ q.T * r for p, q, r in zip(a.split(counts), w.unbind(), wrow.view(case["G"], -1).unbind())])
    s["out"][:y.shape[0]] = (y * row[:y.shape[0]].unsqueeze(1)).to(torch.bfloat16)
    return s["out"]  # rows past the last expert's stay as they were


_PLAIN = {"norm": _norm, "norm_bwd": _norm_bwd, "route": _route, "route_bwd": _route_bwd,
          "combine_bwd": _combine_bwd, "fp4": _fp4}


# --------------------------------------------------------------------------
# The library's calls
# --------------------------------------------------------------------------

def _library(s):
    import mlp_gemms_gb300 as mx
    case = s["case"]
    op = case["op"]
    if op == "norm":
        y, mean, rstd, out = mx.mx_layernorm_fwd(s["x"], s["w"], s["b"], eps=EPS, residual=s["res"], rms=case["rms"])
        return y, mean, rstd, out if case["res"] else None
    if op == "norm_bwd":
        return mx.mx_layernorm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["w"], dres=s["res"], rms=case["rms"],
                                   bias=case["bias"])
    if op in ("route", "route_bwd"):
        score = mx.SCORE_SIGMOID if case["score"] == "sigmoid" else mx.SCORE_SOFTMAX
    if op == "route":
        w, ids, load, total = mx.mx_moe_topk(s["logits"], case["k"], score, bias=s["bias"], groups=case["groups"],
                                             topk_groups=case["topk_groups"], group_top=case["group_top"],
                                             renorm=case["renorm"], scale=2.5, stats=case["stats"])
        return (w, ids, load, total) if case["stats"] else (w, ids)
    if op == "route_bwd":
        return mx.mx_moe_topk_bwd(s["logits"], s["ids"], s["dweights"], score, renorm=case["renorm"], scale=2.5,
                                  dscore_sum=s["dsum"])
    if op == "combine_bwd":
        return mx.mx_moe_unpermute_bwd(s["dout"], s["in"], s["row_of"], s["w"], src=s["src"])
    data, scale, row = s["w"]
    w = mx.NVFP4(case["G"] * case["N"], case["K"], data=data, scale=scale, row_scale=row)
    a = mx.mx_nvfp4_quantize(s["x"], src=s["src"], offsets=s["ends"])
    return mx.mx_nvfp4_gemm(a, w, case["G"], s["ends"], out=s["out"])


def run(state):
    return _library(state) if own else _PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------
# Work and definition
# --------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        R, D = case["R"], case["D"]
        e = 2 if case["x"] == "bf16" else 4
        if op == "norm":
            return {"bytes": R * D * (e + 2 + (2 * e if case["res"] else 0)) + 2 * D * (1 + case["bias"]) + 8 * R,
                    "flops": 8 * R * D}
        return {"bytes": R * D * (2 * e + 2 + (e if case["res"] else 0)) + D * (2 + 4 * (1 + case["bias"])) + 8 * R,
                "flops": 14 * R * D}
    if op in ("route", "route_bwd"):
        T, G, k = case["T"], case["G"], case["k"]
        e = 2 if case["x"] == "bf16" else 4
        if op == "route":
            return {"bytes": T * G * e + 8 * T * k + (4 * G if case["bias"] else 0) + (8 * G if case["stats"] else 0),
                    "flops": T * G * 8}
        return {"bytes": 2 * T * G * e + 8 * T * k + (4 * G if case["stats"] else 0), "flops": T * G * 8}
    if op == "combine_bwd":
        T, k, D = case["T"], case["k"], case["D"]
        return {"bytes": 2 * T * D + 4 * T * k * D + 12 * T * k, "flops": 3 * T * k * D}
    T, G, k, K, N = case["T"], case["G"], case["k"], case["K"], case["N"]
    used = min(G, T * k)
    return {"bytes": 2 * T * K + used * N * (K // 2 + K // 16 + 4) + 2 * T * k * N, "flops": 2 * T * k * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        x = s["x"].to(d)
        out = None
        if op == "norm" and case["res"]:
            out = x + s["res"].to(d)
            x = out.to(_dtype(case)).to(d)
        mean = torch.zeros(case["R"], 1, dtype=d, device="cuda") if case["rms"] else x.sum(1, keepdim=True) / case["D"]
        if op == "norm":
            rstd = (((x - mean) ** 2).sum(1, keepdim=True) / case["D"] + EPS) ** -0.5
            y = torch.einsum("rd,d->rd", (x - mean) * rstd, s["w"].to(d))
            y = y + s["b"].to(d) if case["bias"] else y
            return y, None if case["rms"] else mean[:, 0], rstd[:, 0], out
        rstd = s["rstd"].to(d).unsqueeze(1)
        mean = mean if case["rms"] else s["mean"].to(d).unsqueeze(1)
        z, dy = (x - mean) * rstd, s["dy"].to(d)
        g = torch.einsum("rd,d->rd", dy, s["w"].to(d))
        along = torch.einsum("rd,rd->r", g, z).unsqueeze(1) / case["D"]
        dx = rstd * (g - z * along - (0.0 if case["rms"] else g.sum(1, keepdim=True) / case["D"]))
        dx = dx + s["res"].to(d) if case["res"] else dx
        return dx, torch.einsum("rd,rd->d", dy, z), dy.sum(0) if case["bias"] else None
    if op == "route":
        x = s["logits"].to(d)
        p = torch.special.expit(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
        bias = torch.zeros(case["G"], dtype=d, device="cuda") if s["bias"] is None else s["bias"].to(d)
        v = torch.where(torch.isinf(x), x, p + bias)
        n, T = case["groups"], case["T"]

        def best(v, count):  # one by one: the largest, of equal ones the lowest index that is left
            index = torch.arange(v.shape[1], device="cuda").expand(T, -1)
            left, chosen = torch.ones_like(v, dtype=torch.bool), []
            for _ in range(count):
                top = torch.where(left, v, -math.inf).amax(1, keepdim=True)
                chosen.append(torch.where((v == top) & left, index, v.shape[1]).amin(1, keepdim=True))
                left = left.scatter(1, chosen[-1], False)
            return torch.cat(chosen, 1)

        if n > 1:
            value = v.view(T, n, -1).topk(case["group_top"], -1).values.sum(-1)
            shut = torch.ones((T, n), dtype=torch.bool, device="cuda").scatter(1, best(value, case["topk_groups"]), False)
            v = v.view(T, n, -1).masked_fill(shut.unsqueeze(2), -math.inf).view(T, -1)
        ids = best(v, case["k"])
        w = torch.gather(p, 1, ids)
        w = 2.5 * (w / w.sum(1, keepdim=True) if case["renorm"] else w)
        if not case["stats"]:
            return w, ids.to(torch.int32)
        share = p / p.sum(1, keepdim=True)
        return w, ids.to(torch.int32), None, share.sum(0)
    if op == "route_bwd":
        x = s["logits"].to(d).requires_grad_(True)
        p = torch.special.expit(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
        w = torch.gather(p, 1, s["ids"].long())
        w = w / w.sum(1, keepdim=True) if case["renorm"] else w
        loss = (2.5 * w * s["dweights"].to(d)).sum()
        if case["stats"]:
            loss = loss + ((p / p.sum(1, keepdim=True)).sum(0) * s["dsum"].to(d)).sum()
        return torch.autograd.grad(loss, x)[0]
    if op == "combine_bwd":
        rows, dout = s["row_of"].long(), s["dout"].to(d)
        din = torch.zeros(s["in"].shape, dtype=d, device="cuda")
        dw = torch.empty(s["w"].shape, dtype=d, device="cuda")
        for j in range(case["k"]):
            din[rows[:, j]] = torch.einsum("t,td->td", s["w"][:, j].to(d), dout)
            dw[:, j] = torch.einsum("td,td->t", dout, s["in"][rows[:, j]].to(d))
        return din, dw
    # 4-bit products: every value by its nearest code, in 64 bits
    def near(x):
        r = x.shape[0]
        amax = x.abs().view(r, -1, BLOCK).amax(2)
        row = torch.exp2(torch.ceil(torch.log2(amax.amax(1, keepdim=True) / 2688)).clamp(min=-100))
        scale = (amax / row / 6).to(torch.float32).to(torch.float8_e4m3fn).to(d)
        step = (scale * row).repeat_interleave(BLOCK, 1)
        q = (x / torch.where(step == 0, math.inf, step)).abs()
        q = torch.where(q < 2, torch.round(2 * q) / 2, torch.where(q < 4, torch.round(q), 2 * torch.round(q / 2))).clamp(max=6)
        return q * step * x.sign()

    x = s["x"].to(d)
    if s["src"] is not None:
        x = torch.cat([x, x.new_zeros(1, case["K"])])[s["src"].long()]
    a = near(x)
    packed, blocked, wrow = s["w"]
    G, N, K = case["G"], case["N"], case["K"]
    grid = torch.tensor(F4, dtype=d, device="cuda")
    signed = torch.cat([grid, -grid])
    w = torch.empty((G * N, K), dtype=d, device="cuda")
    w[:, 0::2], w[:, 1::2] = signed[(packed % 16).long()], signed[(packed // 16).long()]
    r = torch.arange(G * N, device="cuda").unsqueeze(1)
    c = torch.arange(K // BLOCK, device="cuda").unsqueeze(0)
    at = (r // 128 * ((K // BLOCK + 3) // 4) + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4
    w *= (blocked[at].view(torch.float8_e4m3fn).to(d) * wrow.to(d).unsqueeze(1)).repeat_interleave(BLOCK, 1)
    out = torch.zeros((a.shape[0], N), dtype=d, device="cuda")
    begin = 0
    for g, end in enumerate([a.shape[0]] if s["ends"] is None else s["ends"].tolist()):
        out[begin:end] = torch.einsum("rk,nk->rn", a[begin:end], w[g * N:(g + 1) * N])
        begin = end
    return out
