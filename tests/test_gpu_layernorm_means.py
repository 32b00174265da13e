"""Rows of layer norm whose spread is small beside their mean, or nothing: what the mean's own rounding would show in."""
import pytest
import torch

from tests import operator_refs as R
from tests.gpu_util import lib
from tests.test_gpu_layernorm import EPS, gen, steps

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32

# rows of a warp, of a CTA, and through the ring of either
SHAPES = [(8, 100), (8, 128), (8, 250), (8, 1000), (8, 1111), (8, 7168), (8, 8191), (8, 16383), (5000, 500), (5000, 513), (1300, 7168), (400, 16001)]


def short_values(rows, g):
    """bf16 values of every mantissa, sizes from 2^-6 to 2^16: 16384 of them have an exact sum in fp32."""
    size = torch.exp2(torch.randint(-6, 17, (rows, 1), generator=g, device=DEV).float())
    v = size * (1 + torch.randint(0, 128, (rows, 1), generator=g, device=DEV) / 128)
    return torch.where(torch.rand((rows, 1), generator=g, device=DEV) < 0.5, v, -v)


@pytest.mark.parametrize("rows, cols", SHAPES)
@pytest.mark.parametrize("t", [BF, F32])
def test_rows_of_one_short_value(rows, cols, t):
    """Their mean is their value: nothing is left of them, forward and backward."""
    dsa, g = lib(), gen(cols)
    x = short_values(rows, g).expand(rows, cols).contiguous().to(t)
    w, b = torch.randn(cols, generator=g, device=DEV).to(t), torch.randn(cols, generator=g, device=DEV).to(t)
    dy = torch.randn((rows, cols), generator=g, device=DEV).to(t)
    out, dx = torch.empty_like(x), torch.empty_like(x)
    dw, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    dsa.dsa_layernorm(x, w, b, EPS, out=out)
    assert torch.equal(out, b.expand(rows, cols))
    dsa.dsa_layernorm_backward(dy, x, w, EPS, dx, dw, dbias=db)
    assert (dw == 0).all()
    grad = R.d(dy) * R.d(w)
    mean, r = grad.mean(-1, keepdim=True), EPS ** -0.5
    ref, mag = r * (grad - mean), r * (grad.abs() + grad.abs().mean(-1, keepdim=True))
    R.check_close(dx, ref, ref.abs() * R.half_step(t) + steps(cols) * mag * (1 + R.half_step(t)), "dx")


@pytest.mark.parametrize("rows, cols", SHAPES)
def test_rows_of_one_short_value_have_no_norm_without_eps(rows, cols):
    dsa, g = lib(), gen(cols + 2)
    x = short_values(rows, g).expand(rows, cols).contiguous().to(BF)
    w, out = torch.ones(cols, dtype=BF, device=DEV), torch.zeros_like(x)
    dsa.dsa_layernorm(x, w, None, 0.0, out=out)
    assert torch.isnan(out).all()


@pytest.mark.parametrize("rows, cols", SHAPES)
def test_rows_of_one_long_value(rows, cols):
    """Sums of fp32 values round, and the mean is off by as much: no more than that shows."""
    dsa, g = lib(), gen(cols + 1)
    v = torch.rand((rows, 1), generator=g, device=DEV) + 0.01
    x = v.expand(rows, cols).contiguous()
    w, b = torch.randn(cols, generator=g, device=DEV), torch.randn(cols, generator=g, device=DEV)
    out = torch.empty_like(x)
    dsa.dsa_layernorm(x, w, b, EPS, out=out)
    xhat = steps(cols) * R.d(v) * EPS ** -0.5
    R.check_close(out, R.d(b).expand(rows, cols), xhat * R.d(w).abs() * 1.01 + 3 * R.FP32 * R.d(b).abs(), "out")


def test_the_root_is_rounded_once():
    """Rows of 1 and -1 have variance 1 and give 1 / sqrt(1 + eps) itself: off by its rounding and little more."""
    dsa = lib()
    for cols in (2, 512):
        x = torch.tensor([1.0, -1.0], device=DEV).repeat(cols // 2).expand(3, cols).contiguous()
        w, out, dx, dw = torch.ones(cols, device=DEV), torch.empty_like(x), torch.empty_like(x), torch.empty(cols, device=DEV)
        for eps in [float(e) for e in 4.0 ** (torch.rand(200, generator=torch.Generator().manual_seed(cols)) * 16 - 15)]:
            v = torch.tensor(1.0) + torch.tensor(eps)  # as fp32 rounds it
            ref = 1.0 / torch.sqrt(v.double())
            dsa.dsa_layernorm(x, w, None, eps, out=out)
            assert ((R.d(out).abs() - ref).abs() <= ref * R.FP32 * (1 + 2.0 ** -10)).all(), eps
            dsa.dsa_layernorm_backward(x[:1], x[:1], w, eps, dx[:1], dw)  # dweight = dy xhat
            assert ((R.d(dw) - ref).abs() <= ref * R.FP32 * (1 + 2.0 ** -10)).all(), eps


def test_rows_whose_variance_ends_in_infinity_or_zero():
    """1 / sqrt of what fp32 cannot hold: nothing of the row but the bias; of nothing, no number."""
    dsa, inf = lib(), float("inf")
    for cols in (2, 512, 8192):
        x = torch.tensor([1.0, -1.0], device=DEV).repeat(cols // 2).expand(2, cols) * torch.tensor([[2.0 ** 70], [0.0]], device=DEV)
        w, b, out = torch.ones(cols, device=DEV), torch.full((cols,), 0.5, device=DEV), torch.empty_like(x.contiguous())
        dsa.dsa_layernorm(x.contiguous(), w, b, 0.0, out=out)
        assert (out[0] == 0.5).all() and torch.isnan(out[1]).all()
        tiny = x[:1].contiguous() * 2.0 ** -75 * 2.0 ** -75  # its squares are below fp32's smallest (2^-150 itself is 0 in fp32)
        dsa.dsa_layernorm(tiny, w, b, 0.0, out=out[:1])
        assert (out[0].abs() == inf).all()


def test_the_root_of_the_smallest_and_largest_variances():
    """Rows of 2^k and -2^k: their variance is 4^k, below fp32's normal numbers and up to its largest."""
    dsa = lib()
    for cols in (2, 512, 8192):
        x = torch.tensor([1.0, -1.0], device=DEV).repeat(cols // 2).expand(127, cols) * torch.exp2(torch.arange(-74, 53, device=DEV))[:, None]
        x = x.contiguous()
        w, out, dx, dw = torch.ones(cols, device=DEV), torch.empty_like(x), torch.empty_like(x), torch.empty(cols, device=DEV)
        dsa.dsa_layernorm(x, w, None, 0.0, out=out)
        assert torch.equal(out, x.sign())
        dsa.dsa_layernorm_backward(torch.ones_like(x), x, w, 0.0, dx, dw)
        assert torch.equal(dw, 127 * x[0].sign())
