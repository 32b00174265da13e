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
