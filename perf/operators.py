"""The dense path of a transformer block when serving, as cases to measure:

    rmsnorm    root-mean-square norm with the residual's addition, to 16 bits or to e4m3 with a scale a row
    quantize   rows to e4m3 with a scale a row (weights once, activations that no norm produces)
    linear     x w^T with bias, activation, gate and residual in its epilogue (f32, f16, bf16)
    linear_q8  the same on e4m3 rows with their scales

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits; with ``own`` true it calls
the framework.  ``exact`` computes them in 64 bits.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -100  # the least row maximum that a scale is made from
EPS = 1e-6


def _linear(name, M, N, K, dtype, act="none", bias=False, gate=False, residual=False, op="linear"):
    c = {"op": op, "M": M, "N": N, "K": K, "dtype": dtype, "act": act, "bias": bias, "gate": gate, "residual": residual}
    return {"name": name, **c} if name else c


def _rows(name, op, M, D, dtype, out="e4m3", residual=False):
    c = {"op": op, "M": M, "D": D, "dtype": dtype, "out": out, "residual": residual}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one token through an attention block's output projection, added to the residual stream
        _linear("linear_token_bf16", 1, 4096, 4096, "bf16", residual=True),
        # a decode batch of 48 sequences through the gated half of an MLP
        _linear("linear_batch_f16", 48, 8192, 4096, "f16", act="silu", gate=True),
        # a prompt of 4096 tokens through an MLP's first matrix
        _linear("linear_prompt_bf16", 4096, 8192, 4096, "bf16", act="gelu_tanh", bias=True),
        # odd widths (a pruned or concatenated layer): rows that are not 16-byte aligned, partial tiles
        _linear("linear_ragged_f16", 1011, 1500, 2047, "f16", act="gelu", bias=True, residual=True),
        # full precision, as for a checked or numerically delicate layer
        _linear("linear_f32", 640, 2048, 2048, "f32", act="relu", bias=True),
        # one token's norm ahead of an 8-bit product: latency alone
        _rows("rmsnorm_token_q8", "rmsnorm", 1, 4096, "bf16", "e4m3", True),
        # a long prompt's norm in 16 bits: bandwidth alone
        _rows("rmsnorm_prompt_bf16", "rmsnorm", 8192, 8192, "bf16", "bf16", True),
        # odd rows to 8 bits, no residual (the first norm of a block)
        _rows("rmsnorm_ragged_q8", "rmsnorm", 1333, 2561, "f16", "e4m3", False),
        # a decode batch of 8 on 8-bit weights
        _linear("linear_q8_token", 8, 8192, 4096, "bf16", residual=True, op="linear_q8"),
        # a long prompt on 8-bit weights: the matrix rate
        _linear("linear_q8_prompt", 8192, 8192, 8192, "bf16", act="silu", gate=True, op="linear_q8"),
        # a decode batch's MLP activations, ahead of the second matrix
        _rows("quantize_batch", "quantize", 16, 12288, "bf16"),
        # a weight brought to 8 bits when a model is loaded
        _rows("quantize_weight", "quantize", 16384, 8192, "f16"),
    ]


def _size(rng, lo, hi):
    """lo..hi, even over the logarithm; four in ten whole multiples of 64 (16 below 128), the others as they fall."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 64 and rng.random() < 0.4:
        q = 64 if v >= 128 else 16
        v = max(q, v // q * q)
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_q8", "rmsnorm", "quantize"))
    if op in ("linear", "linear_q8"):
        dtype = rng.choice(("f32", "f16", "bf16", "bf16") if op == "linear" else ("f32", "f16", "bf16"))
        most = 2.0 ** 40 if op == "linear_q8" else 2.0 ** 33 if dtype == "f32" else 2.0 ** 38
        while True:
            M, N, K = _size(rng, 1, 8192), _size(rng, 48, 16384), _size(rng, 48, 16384)
            if 2 * M * N * K <= most:
                break
        return _linear(None, M, N, K, dtype, rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")),
                       rng.random() < 0.5, rng.random() < 0.3, rng.random() < 0.5, op)
    while True:
        M, D = _size(rng, 1, 16384), _size(rng, 32, 16384)
        if M * D <= 8192 * 8192:
            break
    dtype = rng.choice(("f32", "f16", "bf16"))
    if op == "quantize":
        return _rows(None, op, M, D, dtype)
    return _rows(None, op, M, D, dtype, rng.choice(("e4m3", dtype)), rng.random() < 0.7)


def _to_e4m3(v):
    """Rows of v (32 bits) as e4m3 and their scales."""
    a = v.abs().amax(dim=1).clamp_min(SCALE_FLOOR)
    s = a / E4M3_MAX
    return (v / s[:, None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    s = {"case": case}
    if case["op"] in ("linear", "linear_q8"):
        M, N, K = case["M"], case["N"], case["K"]
        x = normal(M, K)  # a normed activation: unit size
        w = normal(N, K, std=K ** -0.5)
        if case["op"] == "linear":
            s["x"], s["w"] = x.to(dt), w.to(dt)
        else:
            s["xq"], s["xs"] = _to_e4m3(x)
            s["wq"], s["ws"] = _to_e4m3(w)
        s["bias"] = normal(N, std=0.1) if case["bias"] else None
        s["gate"] = normal(M, N).to(dt) if case["gate"] else None
        s["residual"] = normal(M, N).to(dt) if case["residual"] else None
        return s
    M, D = case["M"], case["D"]
    # a residual stream: rows of different size, a few channels much larger than the rest
    big = 1.0 + 9.0 * (torch.rand(D, generator=g, device="cuda") < 0.01).float()
    s["x"] = (normal(M, D) * big * torch.exp(normal(M, 1, std=0.5))).to(dt)
    if case["op"] == "rmsnorm":
        s["gain"] = 1.0 + normal(D, std=0.1)
        s["residual"] = (normal(M, D) * big).to(dt) if case["residual"] else None
    return s


def _plain_act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _plain(s):
    c = s["case"]
    if c["op"] in ("linear", "linear_q8"):
        if c["op"] == "linear":
            z = torch.mm(s["x"].float(), s["w"].float().t())
        else:
            z = torch.mm(s["xq"].float(), s["wq"].float().t()) * s["xs"][:, None] * s["ws"][None, :]
        if s["bias"] is not None:
            z = z + s["bias"]
        z = _plain_act(z, c["act"])
        if s["gate"] is not None:
            z = z * s["gate"].float()
        if s["residual"] is not None:
            z = z + s["residual"].float()
        return {"y": z.to(DT[c["dtype"]])}
    if c["op"] == "quantize":
        q, scale = _to_e4m3(s["x"].float())
        return {"q": q, "scale": scale}
    h = s["x"].float()
    out = {}
    if s["residual"] is not None:
        h = h + s["residual"].float()
        out["h"] = h.to(DT[c["dtype"]])
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * s["gain"]
    if c["out"] == "e4m3":
        out["q"], out["scale"] = _to_e4m3(y)
    else:
        out["y"] = y.to(DT[c["out"]])
    return out


_ct = None


def _convtile():
    global _ct
    if _ct is None:
        from tensor_compiler_tiling_amd import convtile

        _ct = convtile
    return _ct


def _framework(s):
    ct = _convtile()
    c = s["case"]
    if c["op"] == "linear":
        return {"y": ct.linear(s["x"], s["w"], bias=s["bias"], act=c["act"], gate=s["gate"], residual=s["residual"])}
    if c["op"] == "linear_q8":
        return {"y": ct.linear_q8(s["xq"], s["xs"], s["wq"], s["ws"], bias=s["bias"], act=c["act"], gate=s["gate"],
                                  residual=s["residual"], out_dtype=DT[c["dtype"]])}
    if c["op"] == "quantize":
        q, scale = ct.quantize_rows(s["x"])
        return {"q": q, "scale": scale}
    y, scale, h = ct.rmsnorm(s["x"], s["gain"], residual=s["residual"], eps=EPS, out_dtype=DT[c["out"]])
    out = {} if h is None else {"h": h}
    if c["out"] == "e4m3":
        return {**out, "q": y, "scale": scale}
    return {**out, "y": y}


def run(state):
    return _framework(state) if own else _plain(state)


def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] in ("linear", "linear_q8"):
        M, N, K = case["M"], case["N"], case["K"]
        b = (M * K + N * K) * (e if case["op"] == "linear" else 1)
        b += M * N * e * (1 + case["gate"] + case["residual"]) + 4 * N * case["bias"]
        if case["op"] == "linear_q8":
            b += 4 * (M + N)
        return {"bytes": b, "flops": 2 * M * N * K}
    M, D = case["M"], case["D"]
    o = SIZE[case["out"]]
    b = M * D * (e * (1 + 2 * case["residual"]) + o) + (4 * M if case["out"] == "e4m3" else 0)
    if case["op"] == "rmsnorm":
        return {"bytes": b + 4 * D, "flops": 5 * M * D}
    return {"bytes": b, "flops": 2 * M * D}


def exact(case, seed):
    """The definitions in 64 bits; an 8-bit output's value before its rounding to 8 bits."""
    s = prepare(case, seed)
    f = {k: v.to(torch.float64) for k, v in s.items() if isinstance(v, torch.Tensor)}
    if case["op"] in ("linear", "linear_q8"):
        if case["op"] == "linear":
            y = torch.matmul(f["x"], f["w"].transpose(0, 1).contiguous())
        else:
            # every row's scale inside its own factor
            y = torch.matmul(f["xq"] * f["xs"].unsqueeze(1), (f["wq"] * f["ws"].unsqueeze(1)).transpose(0, 1).contiguous())
        if case["bias"]:
            y += f["bias"].unsqueeze(0)
        a = case["act"]
        if a == "relu":
            y = y.clamp(min=0.0)
        elif a == "gelu":  # z times the normal distribution function
            y = y * torch.special.ndtr(y)
        elif a == "gelu_tanh":  # 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u))
            u = (y + 0.044715 * y.pow(3)) * (8.0 / math.pi) ** 0.5
            y = y * torch.sigmoid(u)
        elif a == "silu":
            y = y * torch.sigmoid(y)
        if case["gate"]:
            y = y * f["gate"]
        if case["residual"]:
            y = y + f["residual"]
        return {"y": y}
    if case["op"] == "quantize":
        y, out = f["x"], {}
    else:
        h, out = f["x"], {}
        if case["residual"]:
            h = h + f["residual"]
            out["h"] = h
        rms = torch.linalg.vector_norm(h, dim=1).pow(2).div(case["D"]).add(EPS).sqrt()
        y = h / rms.unsqueeze(1) * f["gain"].unsqueeze(0)
        if case["out"] != "e4m3":
            return {**out, "y": y}
    top = torch.maximum(y.max(dim=1).values, -y.min(dim=1).values).clamp(min=SCALE_FLOOR)
    return {**out, "q": y * (E4M3_MAX / top).unsqueeze(1), "scale": top / E4M3_MAX}
