"""The steps around sparse and dense MLA decoding, as one layer of a served or trained model calls them.

Each case is one call: the residual add with RMS norm and FP8 output in front of the projections (and
its backward), the write of new tokens into the paged latent and index-key caches with the position
rotation, the rotation (and FP8 codes) of the queries (and its backward), and dense MLA attention of
single tokens over the paged latent cache.  ``run`` computes a case in elementary torch operations
in fp32, or, where ``own`` is true, through the package's entry points.
"""
import math

import torch

own = False

EPS = 1e-6
D, DV, DR, DI = 576, 512, 64, 128  # latent row, its value part, rotated columns, index-key width
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one decoded token in front of the projections: latency
        {"name": "norm 1 token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "residual": True, "block": 0},
        # a prefill chunk, FP8 scales per 128 columns, one row short of a round number
        {"name": "norm prefill", "op": "norm", "rows": 8191, "cols": 8192, "dtype": "bf16", "residual": True, "block": 128},
        # the training step's backward of the same norm
        {"name": "norm backward", "op": "norm_bwd", "rows": 8192, "cols": 8192, "dtype": "bf16", "dres": True},
        # a small odd-sized norm in fp32 (per-head or latent norms of a small model)
        {"name": "norm backward odd", "op": "norm_bwd", "rows": 517, "cols": 1111, "dtype": "fp32", "dres": False},
        # one decode step: a new token for each of 64 sequences, far positions, both caches
        {"name": "append decode", "op": "append", "tokens": 64, "seqs": 64, "start": 60000, "page": 64, "norm": True},
        # a prefill's tokens, five ragged sequences
        {"name": "append prefill", "op": "append", "tokens": 32768, "seqs": 5, "start": 0, "page": 64, "norm": True},
        # the queries of one decode step
        {"name": "queries decode", "op": "queries", "tokens": 64, "heads": 128, "index_heads": 64, "start": 60000},
        # the queries of a prefill chunk
        {"name": "queries prefill", "op": "queries", "tokens": 4096, "heads": 128, "index_heads": 64, "start": 28672},
        # the warm-up's gradient of the index queries, back through the rotation
        {"name": "queries backward", "op": "queries_bwd", "tokens": 4096, "index_heads": 64, "start": 28672},
        # one short conversation on a rank that holds 16 heads: latency
        {"name": "mla 1 x 1000", "op": "mla", "seqs": 1, "heads": 16, "lo": 1000, "hi": 1000, "page": 64},
        # a full decode batch of long contexts
        {"name": "mla 64 long", "op": "mla", "seqs": 64, "heads": 128, "lo": 8192, "hi": 65536, "page": 64},
        # a few sequences from one token to very long ones, 16 heads, small pages
        {"name": "mla 9 ragged", "op": "mla", "seqs": 9, "heads": 16, "lo": 1, "hi": 131072, "page": 32},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "append", "queries", "queries_bwd", "mla", "mla"])
    if op in ("norm", "norm_bwd"):
        cols = _log(rng, 64, 16384)
        cols = cols if rng.random() < 0.5 else (cols + 63) // 64 * 64
        case = {"op": op, "rows": _log(rng, 1, min(32768, (1 << 25) // cols)), "cols": cols, "dtype": rng.choice(["bf16", "bf16", "fp32"])}
        if op == "norm":
            return dict(case, residual=rng.random() < 0.7, block=rng.choice([0, 128]))
        return dict(case, dres=rng.random() < 0.7)
    if op == "append":
        tokens = _log(rng, 1, 32768)
        return {"op": op, "tokens": tokens, "seqs": _log(rng, 1, min(tokens, 128)), "start": _log(rng, 1, 131072) - 1,
                "page": rng.choice([32, 64, 128]), "norm": rng.random() < 0.7}
    if op == "queries":
        return {"op": op, "tokens": _log(rng, 1, 4096), "heads": rng.choice([8, 16, 64, 128]), "index_heads": rng.choice([32, 64]),
                "start": _log(rng, 1, 131072) - 1}
    if op == "queries_bwd":
        return {"op": op, "tokens": _log(rng, 1, 4096), "index_heads": rng.choice([1, 32, 64]), "start": _log(rng, 1, 131072) - 1}
    seqs = _log(rng, 1, 256)
    hi = _log(rng, 1, min(131072, (1 << 21) // seqs))
    return {"op": op, "seqs": seqs, "heads": rng.choice([8, 16, 16, 32, 64, 128, 128, 7, 100]), "lo": _log(rng, 1, hi), "hi": hi,
            "page": rng.choice([32, 64, 64, 128])}


def _shares(total, parts):
    """Ragged lengths of ``parts`` sequences, every one at least 1, that sum to ``total``."""
    rest = total - parts
    w = [(i * 7 + 3) % 11 + 1 for i in range(parts)]
    ends = [rest * sum(w[: i + 1]) // sum(w) for i in range(parts)]
    return [1 + e - (ends[i - 1] if i else 0) for i, e in enumerate(ends)]


def _contexts(case):
    """Context lengths spread evenly over [lo, hi], in a mixed order."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    if n == 1:
        return [hi]
    step = next(s for s in (37, 41, 43, 47) if math.gcd(s, n) == 1)
    return [lo + (hi - lo) * ((i * step) % n) // (n - 1) for i in range(n)]


def _freqs():
    return (10000.0 ** (-torch.arange(0, DR, 2, dtype=torch.float64) / DR)).to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0):
        return torch.randn(shape, generator=g, device=DEV, dtype=dtype).mul_(std)

    op, bf16, u8, f32 = case["op"], torch.bfloat16, torch.uint8, torch.float32
    s = {"case": case}
    if op in ("norm", "norm_bwd"):
        rows, cols, t = case["rows"], case["cols"], TYPES[case["dtype"]]
        s["weight"] = normal(cols, std=0.2).add_(1.0).to(t)
        if op == "norm":
            s["x"] = normal(rows, cols, dtype=t)
            s["residual"] = normal(rows, cols, dtype=t, std=2.0) if case["residual"] else None
            s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
            s["out"] = torch.empty_like(s["x"])
            s["codes"] = torch.empty((rows, cols), dtype=u8, device=DEV)
            s["scale"] = torch.empty((rows, -(-cols // case["block"]) if case["block"] else 1), device=DEV)
        else:
            s["dy"] = normal(rows, cols, dtype=t)
            s["h"] = normal(rows, cols, dtype=t, std=2.0)
            s["dres"] = normal(rows, cols, dtype=t) if case["dres"] else None
            s["dx"] = torch.empty_like(s["h"])
            s["dweight"] = torch.empty(cols, device=DEV)
    elif op == "append":
        n, ps, start = case["tokens"], case["page"], case["start"]
        lens = _shares(n, case["seqs"])
        first = [start + (i * 131) % 977 if start else 0 for i in range(len(lens))]  # where each sequence goes on
        s["pos"] = torch.cat([torch.arange(p, p + m) for p, m in zip(first, lens)]).to(torch.int32).to(DEV)
        s["seq"] = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).to(torch.int32).to(DEV)
        need = [((p + m - 1) // ps + 1) - p // ps for p, m in zip(first, lens)]  # only pages that are written are in hand
        pages = torch.randperm(sum(need), generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        table = torch.full((len(lens), max((p + m - 1) // ps + 1 for p, m in zip(first, lens))), -1, dtype=torch.int32)
        at = 0
        for i, (p, k) in enumerate(zip(first, need)):
            table[i, p // ps : p // ps + k] = pages[at : at + k]
            at += k
        s["table"], s["freq"] = table.to(DEV), _freqs()
        s["kv"] = normal(n, D, dtype=bf16)
        s["kI"] = normal(n, DI, dtype=bf16)
        s["kv_weight"] = normal(DV, std=0.2).add_(1.0).to(bf16) if case["norm"] else None
        s["kv_pool"] = normal(at, ps, D, dtype=bf16)  # what the other slots hold stays
        s["k8_pool"] = torch.randint(0, 120, (at, ps, DI), dtype=u8, generator=g, device=DEV)
        s["ks_pool"] = normal(at, ps).abs_()
    elif op == "queries":
        n, h, hi = case["tokens"], case["heads"], case["index_heads"]
        s["pos"] = (torch.arange(n) + case["start"]).to(torch.int32).to(DEV)
        s["freq"] = _freqs()
        s["q_rope"] = normal(n, h, 192, dtype=bf16)[..., 128:]  # the rotated part of the projection's output
        s["q"] = normal(n, h, D, dtype=bf16)  # its other 512 columns are there already
        s["qI"] = normal(n, hi, DI, dtype=bf16)
        s["q8"] = torch.empty((n, hi, DI), dtype=u8, device=DEV)
        s["q_scale"] = torch.empty(n, device=DEV)
    elif op == "queries_bwd":
        n, hi = case["tokens"], case["index_heads"]
        s["pos"] = (torch.arange(n) + case["start"]).to(torch.int32).to(DEV)
        s["freq"] = _freqs()
        s["dq"] = normal(n, hi, DI)
        s["dx"] = torch.empty((n, hi, DI), dtype=bf16, device=DEV)
    else:
        ctx, ps, h = _contexts(case), case["page"], case["heads"]
        need = [-(-c // ps) for c in ctx]
        pages = torch.randperm(sum(need), generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        table = torch.full((len(ctx), max(need)), -1, dtype=torch.int32)
        at = 0
        s["kv_pool"] = normal(sum(need), ps, D, dtype=bf16)
        for i, k in enumerate(need):
            table[i, :k] = pages[at : at + k]
            at += k
            if ctx[i] % ps:
                s["kv_pool"][int(table[i, k - 1]), ctx[i] % ps :] = float("nan")  # slots behind the end are never read
        s["table"] = table.to(DEV)
        s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        s["q"] = normal(len(ctx), h, D, dtype=bf16)
        s["out"] = torch.empty((len(ctx), h, DV), dtype=bf16, device=DEV)
        s["lse"] = torch.empty((len(ctx), h), device=DEV)
    return s


# ------------------------------------------------------------------ plain forms


def _fp8(y):
    """E4M3 codes of the last axis with one scale, amax / 448 (1 for zeros)."""
    amax = y.abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (y / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale.squeeze(-1)


def _angles(s):
    a = s["pos"].double()[:, None] * s["freq"]  # far positions lose their angle in fp32
    return a.cos().float(), a.sin().float()


def _rot_pairs(x, c, n):
    """Rotates the pairs (2i, 2i + 1)."""
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * c - b * n, a * n + b * c), -1).flatten(-2)


def _rot_halves(x, c, n):
    """Rotates the pairs (i, i + 32) of the first 64 columns."""
    a, b = x[..., :32], x[..., 32:64]
    return torch.cat((a * c - b * n, a * n + b * c, x[..., 64:]), -1)


def _norm(s):
    c, x = s["case"], s["x"].float()
    h = x + s["residual"].float() if c["residual"] else x
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    rows, cols = y.shape
    width = c["block"] or cols
    blocks = torch.nn.functional.pad(y, (0, -cols % width)).view(rows, -1, width)
    codes, scale = _fp8(blocks)
    return {"h": h.to(s["x"].dtype) if c["residual"] else None, "out": y.to(s["x"].dtype),
            "codes": codes.view(rows, -1)[:, :cols].contiguous(), "scale": scale}


def _norm_bwd(s):
    dy, h, w = s["dy"].float(), s["h"].float(), s["weight"].float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    xhat, g = h * r, dy * w
    dx = r * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["h"].dtype), "dweight": (dy * xhat).sum(0)}


def _append(s):
    ps, pos = s["case"]["page"], s["pos"].long()
    slot = s["table"][s["seq"].long(), pos // ps].long() * ps + pos % ps
    cos, sin = _angles(s)
    kv = s["kv"].float()
    lat = kv[:, :DV]
    if s["kv_weight"] is not None:
        lat = lat * torch.rsqrt(lat.square().mean(-1, keepdim=True) + EPS) * s["kv_weight"].float()
    s["kv_pool"].view(-1, D)[slot] = torch.cat((lat, _rot_pairs(kv[:, DV:], cos, sin)), -1).to(torch.bfloat16)
    codes, scale = _fp8(_rot_halves(s["kI"].float(), cos, sin))
    s["k8_pool"].view(-1, DI)[slot] = codes.view(torch.uint8)
    s["ks_pool"].view(-1)[slot] = scale
    return {"kv": s["kv_pool"], "k8": s["k8_pool"].view(torch.float8_e4m3fn), "ks": s["ks_pool"]}


def _queries(s):
    cos, sin = (v[:, None] for v in _angles(s))
    s["q"][..., DV:] = _rot_pairs(s["q_rope"].float(), cos, sin).to(torch.bfloat16)
    y = _rot_halves(s["qI"].float(), cos, sin)
    codes, scale = _fp8(y.flatten(1))
    return {"q": s["q"], "q8": codes.view(y.shape), "q_scale": scale}


def _queries_bwd(s):
    cos, sin = (v[:, None] for v in _angles(s))
    return {"dx": _rot_halves(s["dq"], cos, -sin).to(torch.bfloat16)}


def _mla(s):
    table, ctx, q = s["table"], s["ctx"], s["q"].float()
    b, n = table.shape[0], table.shape[1] * s["case"]["page"]
    seen = torch.arange(n, device=DEV)[None] < ctx[:, None]
    kv = s["kv_pool"][table.clamp(min=0).long()].view(b, n, D).float()
    kv = kv.masked_fill_(~seen[..., None], 0.0)
    scores = (q @ kv.transpose(1, 2)).mul_(1.0 / math.sqrt(D)).masked_fill_(~seen[:, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return {"out": ((p @ kv[..., :DV]) / total).to(torch.bfloat16), "lse": (top + total.log()).squeeze(-1)}


def _own(s):
    import sparse_attention_02_gb300 as dsa

    op, e4m3 = s["case"]["op"], torch.float8_e4m3fn
    if op == "norm":
        dsa.dsa_rmsnorm(s["x"], s["weight"], EPS, out=s["out"], residual=s["residual"], residual_out=s["h"], codes=s["codes"],
                        scale=s["scale"], block=s["case"]["block"])
        return {"h": s["h"], "out": s["out"], "codes": s["codes"].view(e4m3), "scale": s["scale"]}
    if op == "norm_bwd":
        dsa.dsa_rmsnorm_backward(s["dy"], s["h"], s["weight"], EPS, s["dx"], s["dweight"], dres=s["dres"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    if op == "append":
        dsa.dsa_cache_append(s["pos"], s["table"], s["freq"], kv=s["kv"], kv_pool=s["kv_pool"], kI=s["kI"], k8_pool=s["k8_pool"],
                             ks_pool=s["ks_pool"], seq=s["seq"], kv_weight=s["kv_weight"], eps=EPS)
        return {"kv": s["kv_pool"], "k8": s["k8_pool"].view(e4m3), "ks": s["ks_pool"]}
    if op == "queries":
        dsa.dsa_rope_queries(s["pos"], s["freq"], q_rope=s["q_rope"], q=s["q"], qI=s["qI"], q8=s["q8"], q_scale=s["q_scale"])
        return {"q": s["q"], "q8": s["q8"].view(e4m3), "q_scale": s["q_scale"]}
    if op == "queries_bwd":
        dsa.dsa_index_rope_backward(s["dq"], s["pos"], s["freq"], s["dx"])
        return {"dx": s["dx"]}
    dsa.dsa_mla_decode_paged(s["q"], s["kv_pool"], s["table"], s["ctx"], 1.0 / math.sqrt(D), s["out"], s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    plain = {"norm": _norm, "norm_bwd": _norm_bwd, "append": _append, "queries": _queries, "queries_bwd": _queries_bwd, "mla": _mla}
    return plain[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        n, e = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        if op == "norm":
            scales = case["rows"] * (-(-case["cols"] // case["block"]) if case["block"] else 1)
            return {"bytes": n * e * (4 if case["residual"] else 2) + n + 4 * scales + case["cols"] * e, "flops": 8 * n}
        return {"bytes": n * e * (4 if case["dres"] else 3) + case["cols"] * (e + 4), "flops": 14 * n}
    t = case.get("tokens", 0)
    if op == "append":
        return {"bytes": t * (2 * D * 2 + DI * 2 + DI + 4 + 12), "flops": t * (4 * DV + 6 * DR + 8 * DI)}
    if op == "queries":
        return {"bytes": t * (case["heads"] * DR * 4 + case["index_heads"] * DI * 3 + 8), "flops": t * (case["heads"] * DR * 3 + case["index_heads"] * DI * 5)}
    if op == "queries_bwd":
        return {"bytes": t * (case["index_heads"] * DI * 6 + 4), "flops": t * case["index_heads"] * DR * 3}
    keys, rows = sum(_contexts(case)), case["seqs"] * case["heads"]
    return {"bytes": keys * D * 2 + rows * (D * 2 + DV * 2 + 4) + 4 * sum(-(-c // case["page"]) for c in _contexts(case)),
            "flops": 2 * keys * case["heads"] * (D + DV)}


# --------------------------------------------- the definitions again, in 64 bits


def _e4m3(v):
    """Nearest E4M3 value (ties to even): three fraction bits, smallest step 2^-9, at most 448."""
    step = torch.exp2(torch.frexp(v.abs().clamp(min=2.0**-6))[1].double() - 4)
    return (v / step).round().mul(step).clamp(-448.0, 448.0)


def _scaled(y):
    big = torch.linalg.vector_norm(y, ord=math.inf, dim=-1, keepdim=True)
    scale = big / 448 + (big == 0)
    return _e4m3(y / scale), scale[..., 0]


def _turn(a, b, pos, freq, back=False):
    """(a + ib) e^{i pos f}, or its inverse."""
    phase = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), torch.outer(pos.double(), freq))
    phase = phase.conj() if back else phase
    phase = phase.view(phase.shape[:1] + (1,) * (a.dim() - 2) + phase.shape[1:])
    z = torch.complex(a.double().contiguous(), b.double().contiguous()) * phase
    return z.real, z.imag


def _turn_index(x, s, back=False):
    re, im = _turn(x[..., :32], x[..., 32:64], s["pos"], s["freq"], back)
    return torch.cat([re, im, x[..., 64:].double()], dim=-1)


def _turn_main(x, s):
    re, im = _turn(x[..., ::2], x[..., 1::2], s["pos"], s["freq"])
    out = torch.empty(x.shape, dtype=torch.float64, device=DEV)
    out[..., ::2], out[..., 1::2] = re, im
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        h = s["x"].double() + (s["residual"].double() if case["residual"] else 0)
        y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / h.shape[1] + EPS) * s["weight"].double()
        w = case["block"] or case["cols"]
        parts = [_scaled(y[:, c : c + w]) for c in range(0, case["cols"], w)]
        return {"h": h if case["residual"] else None, "out": y, "codes": torch.cat([p[0] for p in parts], 1),
                "scale": torch.stack([p[1] for p in parts], 1)}
    if op == "norm_bwd":
        with torch.enable_grad():  # the gradient of the definition itself
            h = s["h"].double().requires_grad_(True)
            w = s["weight"].double().requires_grad_(True)
            y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / h.shape[1] + EPS) * w
            dh, dw = torch.autograd.grad(y, (h, w), s["dy"].double())
        return {"dx": dh + (s["dres"].double() if case["dres"] else 0), "dweight": dw}
    if op == "append":
        lat = s["kv"][:, :DV].double()
        if case["norm"]:
            lat = lat / torch.sqrt((lat * lat).sum(-1, keepdim=True) / DV + EPS) * s["kv_weight"].double()
        row = torch.cat([lat, _turn_main(s["kv"][:, DV:], s)], 1)
        codes, scale = _scaled(_turn_index(s["kI"], s))
        page = s["table"][s["seq"].long(), torch.div(s["pos"], case["page"], rounding_mode="floor").long()].long()
        at = (page, torch.remainder(s["pos"], case["page"]).long())
        kv, k8, ks = s["kv_pool"].double(), s["k8_pool"].view(torch.float8_e4m3fn).double(), s["ks_pool"].double()
        kv[at], k8[at], ks[at] = row, codes, scale
        return {"kv": kv, "k8": k8, "ks": ks}
    if op == "queries":
        q = s["q"].double()
        q[..., DV:] = _turn_main(s["q_rope"], s)
        y = _turn_index(s["qI"], s)
        codes, scale = _scaled(y.reshape(y.shape[0], -1))
        return {"q": q, "q8": codes.view(y.shape), "q_scale": scale}
    if op == "queries_bwd":
        return {"dx": _turn_index(s["dq"], s, back=True)}
    if 4 * sum(_contexts(case)) * case["heads"] * D > 4e12:  # over a few seconds in 64 bits
        return None
    outs, lses = [], []
    for b, c in enumerate(_contexts(case)):
        pages = s["table"][b, : -(-c // case["page"])].long()
        kv = s["kv_pool"][pages].reshape(-1, D)[:c].double()
        z = torch.einsum("hd,sd->hs", s["q"][b].double(), kv) / math.sqrt(D)
        lse = torch.logsumexp(z, -1)
        outs.append(torch.einsum("hs,sv->hv", torch.exp(z - lse[:, None]), kv[:, :DV]))
        lses.append(lse)
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
