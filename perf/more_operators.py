"""FP8 projections and layer norm, as a layer's forward and training step call them.

Each case is one call: the product of FP8 operands with a scale for every 128 values along the summed
axis (a projection of tokens by weights, or a weight's gradient), the quantisation that makes such operands from
activations, gradients and weights (and their transposes, for the backward's products), layer norm as the index
keys and hidden states take it, and its backward.  ``run`` computes a case in elementary torch operations in
fp32, or, where ``own`` is true, through the package's entry points.
"""
import math

import torch

own = False

EPS = 1e-6
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # one decoded token to its latent row and index key (576 + 128 columns): latency
        {"name": "gemm 1 token", "op": "gemm", "m": 1, "n": 704, "k": 4096, "form": "weights", "out": "bf16"},
        # the queries of a decode step: 128 heads of 192 columns
        {"name": "gemm decode", "op": "gemm", "m": 64, "n": 24576, "k": 1536, "form": "weights", "out": "bf16"},
        # a short ragged prompt, odd sizes throughout
        {"name": "gemm ragged", "op": "gemm", "m": 777, "n": 1111, "k": 2050, "form": "weights", "out": "fp32"},
        # a prefill chunk, one token short of a round number
        {"name": "gemm prefill", "op": "gemm", "m": 8191, "n": 8192, "k": 8192, "form": "weights", "out": "bf16"},
        # a weight's gradient: the sum runs over the tokens, both operands scaled row by row
        {"name": "gemm weight grad", "op": "gemm", "m": 4096, "n": 4096, "k": 8191, "form": "rows", "out": "fp32"},
        # a decode step's activations in front of a projection: latency
        {"name": "quantize decode", "op": "quantize", "rows": 64, "cols": 4096, "dtype": "bf16", "block": 1, "plain": True, "turned": False},
        # the gradient that reaches a projection, for both products of its backward
        {"name": "quantize gradient", "op": "quantize", "rows": 8191, "cols": 8192, "dtype": "bf16", "block": 1, "plain": True, "turned": True},
        # fp32 master weights after an optimizer step, for the forward's and the backward's product
        {"name": "quantize weight", "op": "quantize", "rows": 4096, "cols": 7168, "dtype": "fp32", "block": 128, "plain": True, "turned": True},
        # the index keys of one decode step: latency
        {"name": "layernorm decode", "op": "norm", "rows": 64, "cols": 128, "dtype": "bf16", "residual": False, "block": -1},
        # hidden states of a prefill chunk, residual added, FP8 codes per 128 columns for the projection
        {"name": "layernorm prefill", "op": "norm", "rows": 8191, "cols": 8192, "dtype": "bf16", "residual": True, "block": 128},
        # the training step's backward of the same norm
        {"name": "layernorm backward", "op": "norm_bwd", "rows": 8192, "cols": 8192, "dtype": "bf16", "dres": True},
        # ... and of the index keys' norm, whose gradient arrives in fp32
        {"name": "layernorm backward keys", "op": "norm_bwd", "rows": 32767, "cols": 128, "dtype": "fp32", "dres": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm", "quantize", "norm", "norm_bwd"])
    if op == "gemm":
        form = rng.choice(["weights", "weights", "rows"])

        def width():
            v = _log(rng, 64, 16384)
            return v if rng.random() < 0.4 else (v + 63) // 64 * 64

        if form == "weights":
            m, n, k = _log(rng, 1, 8192), width(), width()
        else:
            m, n, k = width(), width(), _log(rng, 1, 8192)
        while m * n * k > 8191 * 8192 * 8192:
            if form == "weights":
                n, k = max(64, n // 2), max(64, k // 2)
            else:
                m, n = max(64, m // 2), max(64, n // 2)
        return {"op": op, "m": m, "n": n, "k": k, "form": form, "out": rng.choice(["bf16", "bf16", "fp32"]) if form == "weights" else "fp32"}
    if op == "quantize":
        cols = _log(rng, 64, 16384)
        cols = cols if rng.random() < 0.4 else (cols + 63) // 64 * 64
        plain, turned = rng.choice([(True, False), (True, True), (True, True), (False, True)])
        return {"op": op, "rows": _log(rng, 1, min(16384, (1 << 26) // cols)), "cols": cols, "dtype": rng.choice(["bf16", "bf16", "fp32"]),
                "block": rng.choice([1, 1, 128]), "plain": plain, "turned": turned}
    cols = _log(rng, 64, 16384)
    cols = cols if rng.random() < 0.5 else (cols + 63) // 64 * 64
    case = {"op": op, "rows": _log(rng, 1, min(32768, (1 << 25) // cols)), "cols": cols, "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "norm":
        return dict(case, residual=rng.random() < 0.5, block=rng.choice([-1, -1, 0, 128]))
    return dict(case, dres=rng.random() < 0.7)


def _pieces(n):
    return -(-n // 128)


def _padded(rows, cols):
    """Codes with rows at multiples of 16 bytes."""
    return torch.empty((rows, (cols + 15) // 16 * 16), dtype=torch.uint8, device=DEV)[:, :cols]


def _operand(v, block_rows):
    """Codes and scales of v, as a program has them from its quantiser."""
    rows, cols = v.shape
    wide = torch.nn.functional.pad(v, (0, -cols % 128, 0, -rows % block_rows))
    cut = wide.view(wide.shape[0] // block_rows, block_rows, -1, 128)
    scale = (cut.abs().amax((1, 3)) / 448.0).clamp_(min=1e-30)
    codes = _padded(rows, cols)
    codes.copy_((cut / scale[:, None, :, None]).to(E4M3).view(torch.uint8).view(wide.shape)[:rows, :cols])
    return codes, scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0):
        return torch.randn(shape, generator=g, device=DEV, dtype=dtype).mul_(std)

    def uneven(rows, cols):
        """Activations: tokens and channels of different size."""
        return normal(rows, cols).mul_(normal(rows, 1, std=0.5).exp_()).mul_(normal(1, cols, std=0.8).exp_())

    op = case["op"]
    s = {"case": case}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["a_scale"] = _operand(uneven(m, k), 1)
        s["b"], s["b_scale"] = _operand(normal(n, k, std=k**-0.5), 128) if case["form"] == "weights" else _operand(uneven(n, k), 1)
        s["out"] = torch.empty((m, n), dtype=TYPES[case["out"]], device=DEV)
    elif op == "quantize":
        rows, cols, r = case["rows"], case["cols"], case["block"]
        s["x"] = uneven(rows, cols).to(TYPES[case["dtype"]])
        s["codes"] = s["scale"] = s["codes_t"] = s["scale_t"] = None
        if case["plain"]:
            s["codes"], s["scale"] = _padded(rows, cols), torch.empty((-(-rows // r), _pieces(cols)), device=DEV)
        if case["turned"]:
            s["codes_t"], s["scale_t"] = _padded(cols, rows), torch.empty((-(-cols // r), _pieces(rows)), device=DEV)
    else:
        rows, cols, t = case["rows"], case["cols"], TYPES[case["dtype"]]
        s["weight"] = normal(cols, std=0.2).add_(1.0).to(t)
        if op == "norm":
            s["bias"] = normal(cols, std=0.2).to(t)
            s["x"] = normal(rows, cols).add_(normal(rows, 1)).to(t)  # rows with means of their own
            s["residual"] = normal(rows, cols, dtype=t, std=2.0) if case["residual"] else None
            s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
            s["out"] = torch.empty_like(s["x"])
            s["codes"] = s["scale"] = None
            if case["block"] >= 0:
                s["codes"] = torch.empty((rows, cols), dtype=torch.uint8, device=DEV)
                s["scale"] = torch.empty((rows, _pieces(cols) if case["block"] else 1), device=DEV)
        else:
            s["dy"] = normal(rows, cols, dtype=t)
            s["h"] = normal(rows, cols, std=2.0).add_(normal(rows, 1)).to(t)
            s["dres"] = normal(rows, cols, dtype=t) if case["dres"] else None
            s["dx"] = torch.empty_like(s["h"])
            s["dweight"], s["dbias"] = (torch.empty(cols, device=DEV) for _ in range(2))
    return s


# ------------------------------------------------------------------ plain forms


def _values(codes, scale, block_rows):
    """What codes and scales stand for."""
    rows, cols = codes.shape
    v = codes.contiguous().view(E4M3).float()
    s = scale.repeat_interleave(block_rows, 0)[:rows] if block_rows > 1 else scale
    return v * s.repeat_interleave(128, 1)[:, :cols]


def _gemm(s):
    block = 128 if s["case"]["form"] == "weights" else 1
    return {"out": (_values(s["a"], s["a_scale"], 1) @ _values(s["b"], s["b_scale"], block).T).to(s["out"].dtype)}


def _fp8(y, axes):
    """E4M3 codes with one scale over the axes, amax / 448 (1 for zeros)."""
    amax = y.abs().amax(axes, keepdim=True)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (y / scale).clamp(-448.0, 448.0).to(E4M3), scale


def _pieces_fp8(x, block_rows):
    rows, cols = x.shape
    wide = torch.nn.functional.pad(x, (0, -cols % 128, 0, -rows % block_rows))
    codes, scale = _fp8(wide.view(wide.shape[0] // block_rows, block_rows, -1, 128), (1, 3))
    return codes.view(wide.shape)[:rows, :cols].contiguous(), scale[:, 0, :, 0]


def _quantize(s):
    c, x = s["case"], s["x"].float()
    out = {"codes": None, "scale": None, "codes_t": None, "scale_t": None}
    if c["plain"]:
        out["codes"], out["scale"] = _pieces_fp8(x, c["block"])
    if c["turned"]:
        out["codes_t"], out["scale_t"] = _pieces_fp8(x.T, c["block"])
    return out


def _norm(s):
    c, x = s["case"], s["x"].float()
    h = x + s["residual"].float() if c["residual"] else x
    d = h - h.mean(-1, keepdim=True)
    y = d * torch.rsqrt(d.square().mean(-1, keepdim=True) + EPS) * s["weight"].float() + s["bias"].float()
    out = {"h": h.to(s["x"].dtype) if c["residual"] else None, "out": y.to(s["x"].dtype), "codes": None, "scale": None}
    if c["block"] > 0:
        out["codes"], out["scale"] = _pieces_fp8(y, 1)
    elif c["block"] == 0:
        out["codes"], out["scale"] = _fp8(y, (1,))
    return out


def _norm_bwd(s):
    dy, h, w = s["dy"].float(), s["h"].float(), s["weight"].float()
    d = h - h.mean(-1, keepdim=True)
    r = torch.rsqrt(d.square().mean(-1, keepdim=True) + EPS)
    xhat, g = d * r, dy * w
    dx = r * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["h"].dtype), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}


def _own(s):
    import sparse_attention_02_gb300 as dsa

    op = s["case"]["op"]

    def e4m3(t):
        return None if t is None else t.view(E4M3)

    if op == "gemm":
        dsa.dsa_gemm_fp8(s["a"], s["a_scale"], s["b"], s["b_scale"], s["out"])
        return {"out": s["out"]}
    if op == "quantize":
        dsa.dsa_quantize_fp8_blocks(s["x"], codes=s["codes"], scale=s["scale"], codes_t=s["codes_t"], scale_t=s["scale_t"],
                                    block_rows=s["case"]["block"])
        return {"codes": e4m3(s["codes"]), "scale": s["scale"], "codes_t": e4m3(s["codes_t"]), "scale_t": s["scale_t"]}
    if op == "norm":
        dsa.dsa_layernorm(s["x"], s["weight"], s["bias"], EPS, out=s["out"], residual=s["residual"], residual_out=s["h"],
                          codes=s["codes"], scale=s["scale"], block=max(s["case"]["block"], 0))
        return {"h": s["h"], "out": s["out"], "codes": e4m3(s["codes"]), "scale": s["scale"]}
    dsa.dsa_layernorm_backward(s["dy"], s["h"], s["weight"], EPS, s["dx"], s["dweight"], dbias=s["dbias"], dres=s["dres"])
    return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}


def run(state):
    if own:
        return _own(state)
    return {"gemm": _gemm, "quantize": _quantize, "norm": _norm, "norm_bwd": _norm_bwd}[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        scales = (m + (_pieces(n) if case["form"] == "weights" else n)) * _pieces(k)
        return {"bytes": (m + n) * k + 4 * scales + m * n * (2 if case["out"] == "bf16" else 4), "flops": 2 * m * n * k}
    rows, cols, e = case["rows"], case["cols"], 2 if case["dtype"] == "bf16" else 4
    n = rows * cols
    if op == "quantize":
        r, forms = case["block"], case["plain"] + case["turned"]
        scales = case["plain"] * -(-rows // r) * _pieces(cols) + case["turned"] * -(-cols // r) * _pieces(rows)
        return {"bytes": n * (e + forms) + 4 * scales, "flops": 4 * n * forms}
    if op == "norm":
        coded = case["block"] >= 0
        scales = rows * (_pieces(cols) if case["block"] > 0 else 1) if coded else 0
        return {"bytes": n * e * (4 if case["residual"] else 2) + (n if coded else 0) + 4 * scales + 2 * cols * e, "flops": 11 * n}
    return {"bytes": n * e * (4 if case["dres"] else 3) + cols * (e + 8), "flops": 20 * n}


# --------------------------------------------- the definitions again, in 64 bits


def _e4m3(v):
    """Nearest E4M3 value (ties to even): three fraction bits, smallest step 2^-9, at most 448."""
    step = torch.exp2(torch.frexp(v.abs().clamp(min=2.0**-6))[1].double() - 4)
    return (v / step).round().mul(step).clamp(-448.0, 448.0)


def _scaled(y, block_rows, width):
    """Codes and scales of pieces of block_rows x width values."""
    parts = [[y[i : i + block_rows, j : j + width] for j in range(0, y.shape[1], width)] for i in range(0, y.shape[0], block_rows)] \
        if block_rows > 1 else [[y[:, j : j + width] for j in range(0, y.shape[1], width)]]
    codes, scales = [], []
    for line in parts:
        top = [torch.linalg.vector_norm(p, ord=math.inf, dim=(0, 1) if block_rows > 1 else 1, keepdim=True) for p in line]
        top = [t / 448 + (t == 0) for t in top]
        codes.append(torch.cat([_e4m3(p / t) for p, t in zip(line, top)], 1))
        scales.append(torch.cat(top, 1))
    return torch.cat(codes), torch.cat(scales)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        total = torch.zeros((m, n), dtype=torch.float64, device=DEV)
        width = 128 * max(1, 16384 // 128 // max(1, (m * n) >> 22))  # pieces of the sum at once
        table = torch.arange(256, dtype=torch.uint8).view(E4M3).double().to(DEV)
        rows_of = torch.arange(n, device=DEV) // (128 if case["form"] == "weights" else 1)
        for k0 in range(0, k, width):
            piece = torch.div(torch.arange(k0, min(k, k0 + width), device=DEV), 128, rounding_mode="floor")
            a = table[s["a"][:, k0 : k0 + width].int()] * s["a_scale"].double()[:, piece]
            b = table[s["b"][:, k0 : k0 + width].int()] * s["b_scale"].double()[rows_of][:, piece]
            total.addmm_(a, b.t())
        return {"out": total}
    if op == "quantize":
        x, r = s["x"].double(), case["block"]
        codes, scale = _scaled(x, r, 128) if case["plain"] else (None, None)
        turned, scale_t = _scaled(x.t(), r, 128) if case["turned"] else (None, None)
        return {"codes": codes, "scale": scale, "codes_t": turned, "scale_t": scale_t}
    if op == "norm":
        h = s["x"].double() + (s["residual"].double() if case["residual"] else 0)
        var, mean = torch.var_mean(h, dim=1, correction=0, keepdim=True)
        y = torch.addcmul(s["bias"].double(), (h - mean) / torch.sqrt(var + EPS), s["weight"].double())
        codes, scale = (None, None) if case["block"] < 0 else _scaled(y, 1, case["block"] or case["cols"])
        return {"h": h if case["residual"] else None, "out": y, "codes": codes, "scale": scale}
    with torch.enable_grad():  # the gradient of the definition itself
        h, w = s["h"].double().requires_grad_(True), s["weight"].double().requires_grad_(True)
        b = torch.zeros_like(w).requires_grad_(True)
        var, mean = torch.var_mean(h, dim=1, correction=0, keepdim=True)
        y = torch.addcmul(b, (h - mean) / torch.sqrt(var + EPS), w)
        dh, dw, db = torch.autograd.grad(y, (h, w, b), s["dy"].double())
    return {"dx": dh + (s["dres"].double() if case["dres"] else 0), "dweight": dw, "dbias": db}
