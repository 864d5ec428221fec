"""Timed cases of the operators that stand around the quantized projections of a transformer block:

  * the 8-bit linear: rows quantized to int8 with one scale each, an integer product, and the scales
    of token and channel with the bias in its output;
  * layer norm with a modulation for each sample: forward, backward with the reduction of the weight's
    and the bias's gradient, and the form that writes int8 rows for the 8-bit linear;
  * rotary positions with several axes: the (cos, sin) table, and the rotation of Q and K heads from
    position ids with its inverse, which is also its gradient.

``listed`` gives the cases, ``draw`` more of the same ranges, ``prepare`` a case's inputs, ``run`` one
pass (in plain torch operations, or through the library where ``own`` is true), ``work`` what a pass
cannot do without, ``exact`` the same outputs from the definition in 64 bits.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------- cases
def _linear(name, M, K, N, dtype="bf16", norm=0, smooth=False, bias=True):
    """norm: 0 for plain rows, else the samples whose modulation the layer norm before the product takes."""
    return {"name": name, "op": "linear", "M": M, "K": K, "N": N, "dtype": dtype, "norm": norm, "smooth": smooth,
            "bias": bias}


def _norm(name, M, K, dtype="bf16", params="bf16", groups=1, offset=1.0, backward=False):
    return {"name": name, "op": "norm_backward" if backward else "norm", "M": M, "K": K, "dtype": dtype,
            "params": params, "groups": groups, "offset": offset}


def _rope(name, M, hq, hk, D, pairs, dtype="bf16", halves=False, shared=False, inverse=False, packed=True,
          far=1.0):
    """pairs: the column pairs of each axis, as a text; far: what the grid's positions are multiplied by."""
    return {"name": name, "op": "rope", "M": M, "hq": hq, "hk": hk, "D": D, "pairs": pairs, "dtype": dtype,
            "halves": halves, "shared": shared, "inverse": inverse, "packed": packed, "far": far}


def listed():
    return [
        # one token (a conditioning vector, a decoded token): latency, the weight's bytes
        _linear("linear_token", 1, 4096, 4096),
        # a prompt's tokens, an odd number of them, behind a smoothing of the channels
        _linear("linear_prompt", 333, 2560, 5120, "f16", smooth=True),
        # the fused projection of a large image's tokens
        _linear("linear_image", 4608, 4096, 12288),
        # two samples of one batch: modulated layer norm, int8 rows, product
        _linear("norm_linear", 2202, 1536, 4608, norm=2),
        # a few rows: latency
        _norm("norm_token", 3, 4096, params="f32", offset=0.0),
        # two samples' tokens under their shift and scale
        _norm("norm_image", 9216, 4096, groups=2),
        # the gradient of the same, with the reduction over each sample's tokens
        _norm("norm_image_backward", 9216, 4096, groups=2, backward=True),
        # odd sizes, 32-bit activations, one weight for all rows
        _norm("norm_odd_backward", 1537, 1153, "f32", "f32", offset=0.0, backward=True),
        # Q and K heads of a packed projection, positions of text and of a latent grid
        _rope("rope_image", 16384, 24, 24, 128, "8,28,28"),
        # one decoded token, shared K heads, halves, one ladder over all axes, a far position
        _rope("rope_token", 1, 32, 8, 128, "16,24,24", halves=True, shared=True, packed=False, far=900.0),
        # a gradient: the inverse rotation of 32-bit heads of which a part is turned
        _rope("rope_gradient", 2777, 16, 16, 96, "8,16,16", "f32", inverse=True, packed=False),
        # the table that the fused projection's output stage reads
        {"name": "rope_table", "op": "rope_table", "M": 16384, "pairs": "8,28,28", "shared": False, "far": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "norm", "norm_backward", "rope", "rope", "rope_table"])
    if op == "linear":
        norm = rng.choice([0, 0, 1, 2])
        # 32-bit outputs only of rows that are given: a normalized value next to a border may round either way,
        # which 16-bit outputs do not show
        c = _linear("", _log(rng, 1, 4608), 16 * _log(rng, 16, 256), 16 * _log(rng, 16, 768),
                    rng.choice(["bf16", "bf16", "f16"] if norm else ["bf16", "bf16", "f16", "f32"]), norm,
                    smooth=norm == 0 and rng.random() < 0.5, bias=rng.random() < 0.7)
    elif op in ("norm", "norm_backward"):
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        K = _log(rng, 64, 6144)
        if rng.random() < 0.6:
            K = (K + 7) // 8 * 8
        M = min(_log(rng, 1, 9216), 9216 * 4096 * 2 // (K * BYTES[dtype]))
        c = _norm("", M, K, dtype, rng.choice(["bf16", "f32"]), min(M, rng.choice([1, 1, 2, 5])), rng.choice([0.0, 1.0]),
                  op == "norm_backward")
    elif op == "rope":
        D = rng.choice([64, 80, 96, 128, 256])
        hk = rng.choice([1, 4, 8, 16])
        P = D // 2 if rng.random() < 0.6 else D // 4
        a = rng.randrange(1, P // 3)
        b = rng.randrange(1, (P - a) // 2 + 1)
        pairs = rng.choice(["%d" % P, "%d,%d" % (a, P - a), "%d,%d,%d" % (a, b, P - a - b)])
        M = min(_log(rng, 1, 16384), 16384 * 24 * 128 // (hk * 2 * D))
        c = _rope("", M, hk * rng.choice([1, 2]), hk, D, pairs, rng.choice(["bf16", "bf16", "f16", "f32"]),
                  rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.4, rng.random() < 0.5,
                  rng.choice([1.0, 30.0, 900.0]))
    else:
        P = rng.choice([32, 48, 64, 128])
        a = rng.randrange(1, P // 2)
        c = {"name": "", "op": op, "M": _log(rng, 512, 16384), "pairs": rng.choice(["%d" % P, "%d,%d" % (a, P - a)]),
             "shared": rng.random() < 0.5, "far": rng.choice([1.0, 30.0, 900.0])}
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _pairs(case):
    return [int(p) for p in case["pairs"].split(",")]


def _positions(case, axes, g, dev):
    """Text tokens first, all at their index on the first axis, then a grid of rows and columns on the other axes."""
    M = case["M"]
    text = int(torch.randint(0, M // 8 + 1, (1,), generator=g, device=dev).item()) if M > 8 else 0
    i = torch.arange(M, device=dev)
    j = (i - text).clamp_min(0)
    wide = max(1, math.isqrt(max(1, M - text)))
    cols = [torch.where(i < text, i, torch.full_like(i, text)), j // wide, j % wide][:axes]
    start = torch.randint(0, 50, (axes,), generator=g, device=dev)
    return ((torch.stack(cols, 1) + start) * case["far"]).to(torch.int64)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dtype)

    s = {"case": case}
    op = case["op"]
    if op == "linear":
        M, K, N, dtype = case["M"], case["K"], case["N"], TYPES[case["dtype"]]
        X = normal(M, K)
        hot = torch.randperm(K, generator=g, device=dev)[: max(1, K // 100)]  # outlier channels
        factor = 20 + 30 * torch.rand(hot.numel(), generator=g, device=dev)
        if not case["norm"]:
            X[:, hot] *= factor
        s["X"] = X.to(dtype)
        # the weight as it was quantized at load time: int8 rows and a scale for each
        W = normal(N, K, scale=0.02)
        top = W.abs().amax(1, keepdim=True)
        s["wq"] = (W.double() * 127 / top.double()).round().to(torch.int8)
        s["w_scale"] = (top / 127).reshape(N)
        s["bias"] = normal(N, scale=0.01) if case["bias"] else None
        s["smooth"] = None
        if case["smooth"]:
            s["smooth"] = torch.ones(K, device=dev)
            s["smooth"][hot] = 1 / factor
        if case["norm"]:
            mod = normal(case["norm"], 2 * K, scale=0.2, dtype=torch.bfloat16)  # shift and scale, as a projection wrote them
            s["shift"], s["scale"] = mod[:, :K], mod[:, K:]
    elif op in ("norm", "norm_backward"):
        M, K, dtype, params, G = case["M"], case["K"], TYPES[case["dtype"]], TYPES[case["params"]], case["groups"]
        s["X"] = (normal(M, K) * 1.5 + normal(M, 1, scale=0.5)).to(dtype)
        s["weight"] = (normal(G, K, scale=0.2) + (1.0 - case["offset"])).to(params)
        s["bias"] = normal(G, K, scale=0.2).to(params)
        if op == "norm_backward":
            s["dY"] = normal(M, K, dtype=dtype)
            x = s["X"].double()  # what the forward pass kept
            s["mean"] = x.mean(1)
            s["rstd"] = (x.var(1, unbiased=False) + 1e-6).rsqrt().float()
            s["mean"] = s["mean"].float()
    elif op == "rope":
        M, D, hq, hk, dtype = case["M"], case["D"], case["hq"], case["hk"], TYPES[case["dtype"]]
        if case["packed"]:  # Q and K are sections of the rows that a fused projection wrote
            Y = normal(M, (hq + 2 * hk) * D).to(dtype)
            s["q"] = Y[:, : hq * D].unflatten(1, (hq, D))
            s["k"] = Y[:, hq * D : (hq + hk) * D].unflatten(1, (hk, D))
        else:
            s["q"], s["k"] = normal(M, hq, D).to(dtype), normal(M, hk, D).to(dtype)
        s["pos"] = _positions(case, len(_pairs(case)), g, dev)
    else:
        s["pos"] = _positions(case, len(_pairs(case)), g, dev)
    if op in ("rope", "rope_table"):
        s["theta"] = 10000.0
    return s


# ---------------------------------------------------------------- plain forms
def _rows_per_group(case, groups):
    return -(-case["M"] // groups)


def _per_row(p, rows, M):
    """Row m takes row m // rows of p."""
    return p.float().repeat_interleave(rows, 0)[:M]


def _plain_norm(X, weight, bias, offset, rows, eps=1e-6):
    x = X.float()
    d = x - x.mean(1, keepdim=True)
    xhat = d * ((d * d).mean(1, keepdim=True) + eps).rsqrt()
    M = X.shape[0]
    return xhat * (_per_row(weight, rows, M) + offset) + _per_row(bias, rows, M)


def _plain_quantize(x):
    """int8 values (as 32-bit floats) and the scale of each row; the rounding decided in 64 bits."""
    top = x.abs().amax(1, keepdim=True)
    q = (x.double() * 127 / torch.where(top == 0, 1.0, top).double()).round().float()
    return q, top / 127


def _plain_linear(s):
    c = s["case"]
    if c["norm"]:
        x = _plain_norm(s["X"], s["scale"], s["shift"], 1.0, _rows_per_group(c, c["norm"]))
    else:
        x = s["X"].float()
        if s["smooth"] is not None:
            x = x * s["smooth"]
    q, scale = _plain_quantize(x)
    y = (q @ s["wq"].float().t()) * scale * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["X"].dtype)


def _sum_groups(v, groups, rows):
    """The sum of each group's rows; a group behind the last row has none."""
    v = torch.nn.functional.pad(v, (0, 0, 0, groups * rows - v.shape[0]))
    return v.unflatten(0, (groups, rows)).sum(1)


def _plain_norm_backward(s):
    c = s["case"]
    M, G = c["M"], c["groups"]
    rows = _rows_per_group(c, G)
    dy = s["dY"].float()
    xhat = (s["X"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    gy = dy * (_per_row(s["weight"], rows, M) + c["offset"])
    dx = (gy - gy.mean(1, keepdim=True) - xhat * (gy * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
    return {"dX": dx.to(s["X"].dtype), "dweight": _sum_groups(dy * xhat, G, rows), "dbias": _sum_groups(dy, G, rows)}


def _plain_cos_sin(pos, pairs, theta, shared):
    """Angles in 64 bits: a far position times a frequency has no fraction left in 32."""
    dev, P = pos.device, sum(pairs)
    axis = torch.cat([torch.full((n,), a, dtype=torch.int64, device=dev) for a, n in enumerate(pairs)])
    if shared:
        power = torch.arange(P, dtype=torch.float64, device=dev) / P
    else:
        power = torch.cat([torch.arange(n, dtype=torch.float64, device=dev) / n for n in pairs])
    angle = pos.double()[:, axis] * theta ** -power
    return angle.cos().float(), angle.sin().float()


def _plain_turn(x, cos, sin, halves):
    P = cos.shape[1]
    v = x.float()
    r, rest = v[..., : 2 * P], x[..., 2 * P :]
    a, b = (r[..., :P], r[..., P:]) if halves else (r[..., 0::2], r[..., 1::2])
    cos, sin = cos[:, None, :], sin[:, None, :]
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([u, w], -1) if halves else torch.stack([u, w], -1).flatten(-2)
    return torch.cat([turned.to(x.dtype), rest], -1)


def _plain(s):
    c = s["case"]
    if c["op"] == "linear":
        return _plain_linear(s)
    if c["op"] == "norm":
        return _plain_norm(s["X"], s["weight"], s["bias"], c["offset"], _rows_per_group(c, c["groups"])).to(s["X"].dtype)
    if c["op"] == "norm_backward":
        return _plain_norm_backward(s)
    cos, sin = _plain_cos_sin(s["pos"], _pairs(c), s["theta"], c["shared"])
    if c["op"] == "rope_table":
        return torch.stack([cos, sin], -1)
    if c["inverse"]:
        sin = -sin
    return {"q": _plain_turn(s["q"], cos, sin, c["halves"]), "k": _plain_turn(s["k"], cos, sin, c["halves"])}


# ---------------------------------------------------------------- the library's calls
def _own(s):
    from bit_rank_compensated_b200 import svdq

    c = s["case"]
    if c["op"] == "linear":
        if c["norm"]:
            xq, x_scale = svdq.i8_layer_norm_quantize(s["X"], s["scale"], s["shift"],
                                                      rows_per_group=_rows_per_group(c, c["norm"]), weight_offset=1.0)
            return svdq.i8_gemm(xq, x_scale, s["wq"], s["w_scale"], s["bias"], dtype=s["X"].dtype)
        return svdq.i8_linear_forward(s["X"], s["wq"], s["w_scale"], s["bias"], col_scale=s["smooth"])
    if c["op"] == "norm":
        return svdq.layer_norm(s["X"], s["weight"], s["bias"], rows_per_group=_rows_per_group(c, c["groups"]),
                               weight_offset=c["offset"])
    if c["op"] == "norm_backward":
        dX, dw, db = svdq.layer_norm_backward(s["dY"], s["X"], s["mean"], s["rstd"], s["weight"],
                                              rows_per_group=_rows_per_group(c, c["groups"]), weight_offset=c["offset"])
        return {"dX": dX, "dweight": dw, "dbias": db}
    axes = svdq.RopeAxes(_pairs(c), theta=s["theta"], shared_ladder=c["shared"], halves=c.get("halves", False))
    if c["op"] == "rope_table":
        return svdq.rope_axes_table(s["pos"], axes)
    q, k = svdq.rope_axes_apply(s["q"], s["k"], s["pos"], axes, inverse=c["inverse"])
    return {"q": q, "k": k}


def run(s):
    return _own(s) if own else _plain(s)


# ---------------------------------------------------------------- floors
def work(case):
    op, M = case["op"], case["M"]
    if op == "linear":
        K, N, e = case["K"], case["N"], BYTES[case["dtype"]]
        extra = 4 * K * case["smooth"] + 4 * N * case["bias"] + 4 * K * case["norm"]
        return {"bytes": M * K * e + N * K + 4 * N + M * N * e + extra, "flops": 2 * M * N * K}
    if op in ("norm", "norm_backward"):
        K, e, p, G = case["K"], BYTES[case["dtype"]], BYTES[case["params"]], case["groups"]
        if op == "norm":
            return {"bytes": 2 * M * K * e + 2 * G * K * p, "flops": 8 * M * K}
        return {"bytes": 3 * M * K * e + G * K * (p + 8) + 8 * M, "flops": 14 * M * K}
    P, A = sum(_pairs(case)), len(_pairs(case))
    if op == "rope_table":
        return {"bytes": 8 * M * A + 8 * M * P, "flops": 20 * M * P}
    heads = case["hq"] + case["hk"]
    return {"bytes": 2 * M * heads * case["D"] * BYTES[case["dtype"]] + 8 * M * A, "flops": 6 * M * heads * P + 20 * M * P}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("linear", "norm", "norm_backward"):
        M, K = case["M"], case["K"]
        x = s["X"].double()
        groups = case["norm"] if op == "linear" else case["groups"]
        row = torch.arange(M, device=x.device) // (-(-M // groups)) if groups else None
    if op in ("norm", "linear") and groups:
        w, b = (s["scale"], s["shift"]) if op == "linear" else (s["weight"], s["bias"])
        offset = 1.0 if op == "linear" else case["offset"]
        mean = x.sum(1, keepdim=True) / K
        var = ((x - mean) ** 2).sum(1, keepdim=True) / K
        x = (x - mean) / torch.sqrt(var + 1e-6) * (offset + w.double()[row]) + b.double()[row]
        if op == "norm":
            return x
    if op == "linear":
        if s["smooth"] is not None:
            x = (x * s["smooth"].double()).float().double()  # the smoothed value is defined as rounded to 32 bits
        top = x.abs().max(1).values
        q = torch.round(x / torch.where(top == 0, torch.ones_like(top), top)[:, None] * 127)
        y = torch.einsum("mk,nk->mn", q, s["wq"].double()) * (top / 127)[:, None] * s["w_scale"].double()[None, :]
        return y if s["bias"] is None else y + s["bias"].double()[None, :]
    if op == "norm_backward":
        dy, r = s["dY"].double(), s["rstd"].double()[:, None]
        xhat = (x - s["mean"].double()[:, None]) * r
        g = dy * (case["offset"] + s["weight"].double()[row])
        dx = r * (g - g.sum(1, keepdim=True) / K - xhat * ((g * xhat).sum(1, keepdim=True) / K))
        zero = torch.zeros(groups, K, dtype=torch.float64, device=x.device)
        return {"dX": dx, "dweight": zero.index_add(0, row, dy * xhat), "dbias": zero.index_add(0, row, dy)}
    pairs = _pairs(case)
    P = sum(pairs)
    turns = []
    for a, n in enumerate(pairs):
        for i in range(n):
            p = len(turns)
            f = math.exp(-math.log(s["theta"]) * (p / P if case["shared"] else i / n))
            turns.append(torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["pos"][:, a].double() * f))
    z = torch.stack(turns, 1)
    if op == "rope_table":
        return torch.view_as_real(z)
    if case["inverse"]:
        z = z.conj()
    out = {}
    for name in ("q", "k"):
        v = s[name].double().clone()
        u, w = (slice(0, P), slice(P, 2 * P)) if case["halves"] else (slice(0, 2 * P, 2), slice(1, 2 * P, 2))
        t = torch.complex(v[..., u], v[..., w]) * z[:, None, :]
        v[..., u], v[..., w] = t.real, t.imag
        out[name] = v
    return out
