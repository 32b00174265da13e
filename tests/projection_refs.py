"""The FP8 product, block quantisation and layer norm in fp64, for the operator tests.

Error bounds count half steps of the types' rounding (bf16 2^-8, fp32 2^-24), as in operator_refs.
"""
import torch

from tests import operator_refs as R

U8, F32, BF, F64 = torch.uint8, torch.float32, torch.bfloat16, torch.float64


def pieces(n):
    return -(-n // 128)


def values(codes):
    """What E4M3 codes stand for, in fp64 where the codes are."""
    return R.e4m3_values().to(codes.device)[codes.int()]


def spread(scale, rows, cols, block_rows):
    """scale [ceil(rows / block_rows), ceil(cols / 128)] for every value."""
    return scale.double().repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def padded(rows, cols, device, fill=0x7F):
    """uint8 [rows, cols] with rows at multiples of 16 bytes; between them `fill` (NaN codes: never to be used)."""
    return torch.full((rows, (cols + 15) // 16 * 16), fill, dtype=U8, device=device)[:, :cols]


def codes_like(rows, cols, g, device):
    """Finite codes of every size, in rows at multiples of 16 bytes."""
    c = padded(rows, cols, device)
    v = torch.randint(0, 256, (rows, cols), generator=g, device=device, dtype=torch.int32)
    c.copy_(torch.where((v & 0x7F) == 0x7F, v - 1, v).to(U8))
    return c


def scales_like(shape, g, device):
    """Scales of either sign's neighbourhood of 2^-8, four octaves wide."""
    return torch.exp2(torch.rand(shape, generator=g, device=device) * 4 - 10)


def gemm(a, a_scale, b, b_scale):
    """out [M, N] and sum |a| |b|, which its rounding errors scale with."""
    M, K = a.shape
    N = b.shape[0]
    block = 128 if b_scale.shape[0] == pieces(N) else 1
    va = values(a) * spread(a_scale, M, K, 1)
    vb = values(b) * spread(b_scale, N, K, block)
    return va @ vb.T, va.abs() @ vb.abs().T


def gemm_bound(ref, mag, K, out_dtype):
    """A piece: up to 127 additions in fp32 of exact products, each off by at most a whole step 2^-23 of the sum's size (the
    tensor cores may cut instead of rounding).  Then a scale's product, and one rounding for each piece and CTA added."""
    return (127 * 2 * R.FP32 + (pieces(K) + 12) * R.FP32) * mag + R.half_step(out_dtype) * ref.abs() + 1e-30


def layernorm(x, residual, weight, bias, eps):
    """h, y, and the magnitude that y's fp32 errors scale with."""
    h = R.d(x) if residual is None else R.d(x) + R.d(residual)
    mean = h.mean(-1, keepdim=True)
    c = h - mean
    r = 1.0 / torch.sqrt(c.square().mean(-1, keepdim=True) + eps)
    y = c * r * R.d(weight)
    # h and its difference from the mean are each rounded once; the mean is off by the roundings of its sum
    mag = y.abs() + (h.abs() + h.abs().mean(-1, keepdim=True)) * r * R.d(weight).abs()
    if bias is not None:
        y, mag = y + R.d(bias), mag + R.d(bias).abs()
    return h, y, mag


def layernorm_backward(dy, h, weight, dres, eps):
    """dx, dweight, dbias and the magnitudes that their rounding errors scale with."""
    dy, h, w = R.d(dy), R.d(h), R.d(weight)
    mean = h.mean(-1, keepdim=True)
    c = h - mean
    r = 1.0 / torch.sqrt(c.square().mean(-1, keepdim=True) + eps)
    xhat, g = c * r, dy * w
    dx = r * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    xmag = xhat.abs() + (h.abs() + h.abs().mean(-1, keepdim=True)) * r  # of xhat's errors
    mag = r * (g.abs() + g.abs().mean(-1, keepdim=True) + xmag * (g.abs() * xhat.abs()).mean(-1, keepdim=True)
               + xhat.abs() * (g.abs() * xmag).mean(-1, keepdim=True))
    if dres is not None:
        dx, mag = dx + R.d(dres), mag + R.d(dres).abs()
    return dx, (dy * xhat).sum(0), dy.sum(0), mag, (dy.abs() * xmag).sum(0), dy.abs().sum(0)
