"""The norm, rotation, FP8 and dense-attention definitions in fp64 on the CPU, for the operator tests.

Error bounds are stated in half steps of the types' rounding (bf16 2^-8, fp32 2^-24, E4M3 2^-4 relative
or 2^-10 for its subnormals) times the operations that can each be off by one.
"""
import math

import torch

BF16, FP32, E4M3 = 2.0 ** -8, 2.0 ** -24, 2.0 ** -4


def half_step(dtype):
    return BF16 if dtype == torch.bfloat16 else FP32


def d(t):
    return None if t is None else t.detach().cpu().double()


def inv_freq(base=10000.0):
    return base ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)


def rmsnorm(x, residual, weight, eps):
    h = d(x) if residual is None else d(x) + d(residual)
    return h, h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps) * d(weight)


def rmsnorm_backward(dy, h, weight, dres, eps):
    """dx, dweight and the magnitudes that their rounding errors scale with."""
    dy, h, w = d(dy), d(h), d(weight)
    r = 1.0 / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    xhat, g = h * r, dy * w
    dx = r * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    mag = r * (g.abs() + xhat.abs() * (g * xhat).abs().mean(-1, keepdim=True))
    if dres is not None:
        dx, mag = dx + d(dres), mag + d(dres).abs()
    return dx, (dy * xhat).sum(0), mag, (dy * xhat).abs().sum(0)


def rotate(a, b, pos, freq):
    t = pos.double()[:, None] * freq[None]
    t = t.view(t.shape[:1] + (1,) * (a.dim() - 2) + t.shape[1:])
    return a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos()


def rotate_main(x, pos, freq):
    """[T, ..., 64], pairs (2i, 2i + 1)."""
    a, b = rotate(x[..., 0::2], x[..., 1::2], pos, freq)
    return torch.stack([a, b], -1).flatten(-2)


def rotate_index(x, pos, freq):
    """[T, ..., 128], pairs (i, i + 32) of the first 64."""
    a, b = rotate(x[..., :32], x[..., 32:64], pos, freq)
    return torch.cat([a, b, x[..., 64:]], -1)


def check_close(got, ref, bound, what):
    err = (d(got) - ref).abs()
    assert torch.isfinite(d(got)).all(), f"{what}: non-finite"
    over = err - bound
    assert (over <= 0).all(), f"{what}: off by {err.flatten()[over.argmax()]:.3g}, {over.max():.3g} over the bound"


def e4m3_values():
    return torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def check_fp8(codes, scale, y, rel, mode, what):
    """codes [n, c] uint8 and scale [n] of the fp64 rows y, whose fp32 forms are off by at most rel (relative, plus
    the row's own amax times rel)."""
    codes, scale = codes.cpu(), d(scale)
    amax = y.abs().amax(-1)
    ratio = amax / 448.0
    nz = ratio > 0
    assert (scale[~nz] == 1).all() and (codes[~nz] & 0x7F == 0).all(), f"{what}: zero rows"
    if mode == 0:
        assert ((scale - ratio)[nz].abs() <= (rel + 2 * FP32) * ratio[nz]).all(), f"{what}: scale"
    else:
        assert (torch.frexp(scale)[0] == 0.5).all(), f"{what}: scale is no power of two"
        s, r = scale[nz], ratio[nz]
        assert (s >= r * (1 - rel - 2 * FP32)).all() and (s <= 2 * r * (1 + rel + 2 * FP32)).all(), f"{what}: scale"
    got = e4m3_values()[codes.long()]
    assert torch.isfinite(got).all(), f"{what}: NaN codes"
    v = y / scale[:, None]
    bound = torch.maximum(v.abs() * E4M3, torch.tensor(2.0 ** -10, dtype=torch.float64)) + \
        (rel + 2 * FP32) * (v.abs() + (amax / scale)[:, None])
    err = (got - v).abs()
    assert (err <= bound).all(), f"{what}: code off by {err.max():.3g}"


def dense_mla(q, rows, sm_scale):
    """q [H, 576], rows [n, 576] -> out [H, 512], lse [H], sum p |v| [H, 512], largest sum |q||k| scale."""
    q, kv = d(q), d(rows)
    if kv.shape[0] == 0:
        z = torch.zeros((q.shape[0], 512), dtype=torch.float64)
        return z, torch.full((q.shape[0],), -math.inf, dtype=torch.float64), z, 0.0
    s = q @ kv.T * sm_scale
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None])
    return p @ kv[:, :512], lse, p @ kv[:, :512].abs(), float((q.abs() @ kv.abs().T).max()) * sm_scale
