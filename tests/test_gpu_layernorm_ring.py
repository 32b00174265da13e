"""Layer norm where its rows go through the ring in shared memory: every form of its outputs, and in its inputs' place."""
import pytest
import torch

from tests import operator_refs as R
from tests import projection_refs as P
from tests.gpu_util import lib
from tests.test_gpu_layernorm import EPS, gen, steps

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8

# The ring takes rows of up to 1024 columns from 32 an SM on (a warp each), longer ones from 2 to 16 an SM on (a CTA each).
# Row counts that no CTA's share divides.
RING = [(4871, 264), (4873, 512), (4877, 1000), (4879, 1023), (4881, 1280), (4897, 2048), (2443, 5000), (1301, 4096), (311, 8192),
        (317, 8191), (309, 12001), (307, 16384)]


def layernorm64(x, res, w, b):
    """h, y and the magnitude that y's fp32 errors scale with, in fp64 where x is."""
    h = x.double() + (0 if res is None else res.double())
    mean = h.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt((h - mean).square().mean(-1, keepdim=True) + EPS)
    y = (h - mean) * r * w.double()
    mag = y.abs() + (h.abs() + h.abs().mean(-1, keepdim=True)) * r * w.double().abs()
    return (h, y, mag) if b is None else (h, y + b.double(), mag + b.double().abs())


def within(got, ref, bound, what):
    over = (got.double() - ref).abs() - bound
    assert torch.isfinite(got.double()).all() and (over <= 0).all(), f"{what}: {float(over.max()):.3g} over the bound"


def check(x, res, w, b, h, out, codes, scale, block, what):
    rows, cols = x.shape
    rh, ry, mag = layernorm64(x, res, w, b)
    tol, half = steps(cols) * mag, R.half_step(x.dtype)
    if h is not None:
        within(h, rh, rh.abs() * (half + R.FP32) + 1e-30, f"{what} h")
    if out is not None:
        within(out, ry, ry.abs() * half + tol * (1 + half) + 1e-30, f"{what} out")
    if codes is not None:
        width = block or cols

        def tops(v):  # of each piece
            return torch.nn.functional.pad(v.abs(), (0, -cols % width)).view(rows, -1, width).amax(-1)

        s = scale.double().view(rows, -1)
        assert (s > 0).all()
        # a largest value that is off by its own bound moves the scale by as much; the quotient rounds once
        within(s, tops(ry) / 448, tops(tol) / 448 + 2 * R.FP32 * tops(ry) / 448, f"{what} scale")
        s = s.repeat_interleave(width, 1)[:, :cols]
        q = ry / s
        within(P.values(codes), q, q.abs() * (R.E4M3 + 4 * R.FP32) + 2.0 ** -10 + 2 * tol / s, f"{what} codes")


@pytest.mark.parametrize("t, wt", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("rows, cols", RING)
def test_forms(rows, cols, t, wt):
    dsa, g = lib(), gen(rows + cols)
    x = (torch.randn((rows, cols), generator=g, device=DEV) + torch.randn((rows, 1), generator=g, device=DEV)).to(t)
    res = (torch.randn((rows, cols), generator=g, device=DEV) * 2).to(t)
    w, b = (torch.randn(cols, generator=g, device=DEV).to(wt) for _ in range(2))
    # residual, bias, block (None: no codes), h, out
    for r, bias, block, with_h, with_out in ((res, b, 128, True, True), (None, b, 0, False, True), (res, None, 0, True, False),
                                             (None, None, 128, True, False), (res, b, None, False, True)):
        def run():
            h, out = (torch.full_like(x, float("nan")) if k else None for k in (with_h, with_out))
            codes = scale = None
            if block is not None:
                codes = torch.full((rows, cols), 0x7F, dtype=U8, device=DEV)
                scale = torch.full((rows, -(-cols // 128) if block else 1), float("nan"), device=DEV)
            dsa.dsa_layernorm(x, w, bias, EPS, out=out, residual=r, residual_out=h, codes=codes, scale=scale, block=block or 0)
            return h, out, codes, scale

        got = run()
        check(x, r, w, bias, *got, block, f"{rows} x {cols} block {block}")
        for a, again in zip(got, run()):
            assert a is None or torch.equal(a, again)
    assert dsa.dsa_get_device_status() == 0


@pytest.mark.parametrize("rows, cols, t", [(1500, 8192, BF), (5000, 512, BF), (1200, 8191, BF), (4900, 1000, F32), (5000, 1023, BF),
                                           (4900, 2048, BF), (700, 16384, F32)])
def test_in_place_of_its_inputs(rows, cols, t):
    """residual_out in the residual's or x's place and out in x's, while later rows are on their way in."""
    dsa, g = lib(), gen(rows)
    x, r = (torch.randn((rows, cols), generator=g, device=DEV).to(t) for _ in range(2))
    w, b = (torch.randn(cols, generator=g, device=DEV).to(t) for _ in range(2))

    def run(x, r, out, h):
        codes, scale = torch.empty((rows, cols), dtype=U8, device=DEV), torch.empty((rows, -(-cols // 128)), device=DEV)
        dsa.dsa_layernorm(x, w, b, EPS, out=out, residual=r, residual_out=h, codes=codes, scale=scale, block=128)
        return out.clone(), h.clone(), codes, scale

    want = run(x, r, torch.empty_like(x), torch.empty_like(x))
    check(x, r, w, b, want[1], want[0], want[2], want[3], 128, "apart")
    for where in ("x", "r", "both"):
        x2, r2 = x.clone(), r.clone()
        got = run(x2, r2, x2 if where == "both" else torch.empty_like(x), x2 if where == "x" else r2)
        assert all(torch.equal(p, q) for p, q in zip(got, want)), where
    alone = run(x, None, torch.empty_like(x), torch.empty_like(x))
    x2 = x.clone()
    assert all(torch.equal(p, q) for k, (p, q) in enumerate(zip(run(x2, None, x2, torch.empty_like(x)), alone)))
    assert dsa.dsa_get_device_status() == 0
