"""Layer norm and its backward against fp64."""
import pytest
import torch

from tests import operator_refs as R
from tests import projection_refs as P
from tests.gpu_util import lib

pytestmark = pytest.mark.gpu
DEV, EPS = "cuda", 1e-6
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def steps(cols):
    """fp32 roundings of a row's sum and of what follows: a thread adds at most 32 values of its own, then ten steps of
    shuffles and shared memory; the norm, the weights and the bias take a dozen."""
    return (min(cols, 32) + 10 + 12) * R.FP32


def check_forward(x, res, w, b, h, out, codes, scale, block, what, eps=EPS):
    rh, ry, mag = P.layernorm(x, res, w, b, eps)
    if h is not None:
        R.check_close(h, rh, rh.abs() * (R.half_step(h.dtype) + R.FP32) + 1e-30, f"{what} h")
    tol = steps(x.shape[1]) * mag
    if out is not None:
        R.check_close(out, ry, ry.abs() * R.half_step(out.dtype) + tol * (1 + R.half_step(out.dtype)) + 1e-30, f"{what} out")
    if codes is not None:
        width = block or x.shape[1]
        for i, c0 in enumerate(range(0, x.shape[1], width)):
            y, t = ry[:, c0:c0 + width], tol[:, c0:c0 + width]
            top = y.abs().amax(-1, keepdim=True)
            rel = float((t / top.clamp(min=1e-300)).max())
            R.check_fp8(codes[:, c0:c0 + width], scale.view(x.shape[0], -1)[:, i], y, rel, 0, f"{what} fp8 {i}")


COLS = [1, 2, 7, 8, 64, 127, 128, 130, 256, 257, 512, 1000, 1024, 1111, 2048, 4096, 5000, 7168, 8191, 8192, 10001, 16384]


@pytest.mark.parametrize("t, wt", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("cols", COLS)
def test_forward_widths(cols, t, wt):
    dsa, g = lib(), gen(cols)
    for rows in (1, 3, 37):
        x = (torch.randn((rows, cols), generator=g, device=DEV) + torch.randn((rows, 1), generator=g, device=DEV)).to(t)
        res = (torch.randn((rows, cols), generator=g, device=DEV) * 2).to(t)
        w, b = (torch.randn(cols, generator=g, device=DEV).to(wt) for _ in range(2))
        for r, bias, block in ((None, b, 0), (res, None, 128), (res, b, 128)):
            h, out = torch.full_like(x, float("nan")), torch.full_like(x, float("nan"))
            codes, scale = torch.full((rows, cols), 0x7F, dtype=U8, device=DEV), torch.empty((rows, -(-cols // 128) if block else 1), device=DEV)
            got = dsa.dsa_layernorm(x, w, bias, EPS, out=out, residual=r, residual_out=h, codes=codes, scale=scale, block=block)
            assert got[0] is h and got[1] is out and got[2] is codes and got[3] is scale
            check_forward(x, r, w, bias, h, out, codes, scale, block, f"{rows} x {cols}")


@pytest.mark.parametrize("rows, cols, t", [(5000, 128, BF), (5000, 512, BF), (4999, 1000, F32), (3000, 2048, BF), (2000, 4096, F32),
                                           (1500, 8192, BF), (1200, 8191, BF), (700, 16384, F32), (1300, 16384, BF), (9001, 256, F32),
                                           (2500, 2047, F32)])
def test_many_rows(rows, cols, t):
    """Rows through the ring in shared memory, and their gradients."""
    dsa, g = lib(), gen(rows + cols)
    x = (torch.randn((rows, cols), generator=g, device=DEV) + torch.randn((rows, 1), generator=g, device=DEV)).to(t)
    res, dy, dres = ((torch.randn((rows, cols), generator=g, device=DEV)).to(t) for _ in range(3))
    w, b = (torch.randn(cols, generator=g, device=DEV).to(t) for _ in range(2))
    h, out = torch.empty_like(x), torch.empty_like(x)
    dsa.dsa_layernorm(x, w, b, EPS, out=out, residual=res, residual_out=h)
    check_forward(x, res, w, b, h, out, None, None, 0, f"{rows} x {cols}")
    for e in (None, dres):
        dx, dw, db = torch.full_like(x, float("nan")), torch.full((cols,), float("nan"), device=DEV), torch.full((cols,), float("nan"), device=DEV)
        dsa.dsa_layernorm_backward(dy, h, w, EPS, dx, dw, dbias=db, dres=e)
        check_backward(dy, h, w, e, dx, dw, db, f"{rows} x {cols}")
    assert dsa.dsa_get_device_status() == 0


def check_backward(dy, h, w, e, dx, dw, db, what, eps=EPS):
    rx, rw, rb, mag, wmag, bmag = P.layernorm_backward(dy, h, w, e, eps)
    rows, cols = h.shape
    tol = steps(cols)
    R.check_close(dx, rx, rx.abs() * R.half_step(dx.dtype) + 2 * tol * mag * (1 + R.half_step(dx.dtype)) + 1e-30, f"{what} dx")
    # a CTA's rows one after the other (up to rows of them), then the CTAs' sums: 10 in flight, 32 warps, 5 steps
    sums = (min(rows, 400) + 50) * R.FP32
    R.check_close(dw, rw, (sums + 2 * tol) * wmag + 1e-30, f"{what} dweight")
    if db is not None:
        R.check_close(db, rb, sums * bmag + 1e-30, f"{what} dbias")


@pytest.mark.parametrize("t, wt", [(BF, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("cols", COLS)
def test_backward_widths(cols, t, wt):
    dsa, g = lib(), gen(cols + 1)
    for rows in (1, 2, 41):
        h = (torch.randn((rows, cols), generator=g, device=DEV) * 2 + 1).to(t)
        dy, dres = (torch.randn((rows, cols), generator=g, device=DEV).to(t) for _ in range(2))
        w = torch.randn(cols, generator=g, device=DEV).to(wt)
        for e, with_bias in ((None, True), (dres, True), (dres, False)):
            dx, dw = torch.full_like(h, float("nan")), torch.full((cols,), float("nan"), device=DEV)
            db = torch.full((cols,), float("nan"), device=DEV) if with_bias else None
            got = dsa.dsa_layernorm_backward(dy, h, w, EPS, dx, dw, dbias=db, dres=e)
            assert got[0] is dx and got[1] is dw and got[2] is db
            check_backward(dy, h, w, e, dx, dw, db, f"{rows} x {cols}")


def test_gradients_are_those_of_differences():
    """dx, dweight and dbias against central differences of the fp64 definition."""
    dsa, g = lib(), gen(2)
    rows, cols, step = 3, 20, 1e-5
    h, dy = torch.randn((rows, cols), generator=g, device=DEV), torch.randn((rows, cols), generator=g, device=DEV)
    w, b = torch.randn(cols, generator=g, device=DEV), torch.randn(cols, generator=g, device=DEV)
    dx, dw, db = torch.empty_like(h), torch.empty_like(w), torch.empty_like(b)
    dsa.dsa_layernorm_backward(dy, h, w, EPS, dx, dw, dbias=db)

    def loss(h, w, b):
        return float((P.layernorm(h, None, w, b, EPS)[1] * R.d(dy)).sum())

    for k, (t, grad) in enumerate(((h, dx), (w, dw), (b, db))):
        args = [R.d(v).clone() for v in (h, w, b)]
        flat = args[k].view(-1)
        for i in range(flat.numel()):
            keep = float(flat[i])
            flat[i] = keep + step
            up = loss(*args)
            flat[i] = keep - step
            down = loss(*args)
            flat[i] = keep
            # second order of the step, and the fp64 difference's own rounding
            assert abs((up - down) / (2 * step) - float(grad.view(-1)[i])) <= 1e-4 * (1 + abs(float(grad.view(-1)[i])))


@pytest.mark.parametrize("cols", [64, 128, 1000, 4096, 16384])
@pytest.mark.parametrize("t", [BF, F32])
def test_large_common_offset(cols, t):
    """Rows whose mean is far larger than their spread: the variance is taken about the mean."""
    dsa, g = lib(), gen(8)
    x = (torch.randn((64, cols), generator=g, device=DEV) * 4 + 1000).to(t)
    x[0] = 1000
    x[0, -1] = 1008
    w, b = torch.ones(cols, dtype=t, device=DEV), torch.zeros(cols, dtype=t, device=DEV)
    out = torch.empty_like(x)
    dsa.dsa_layernorm(x, w, b, EPS, out=out)
    check_forward(x, None, w, b, None, out, None, None, 0, "offset")
    assert abs(float(out.double().mean())) < 0.01


def test_rows_apart_in_place_and_off_alignment():
    dsa, g = lib(), gen(3)
    for cols in (128, 130, 1024, 4096):
        for t in (BF, F32):
            for off, ld in ((0, cols + 8), (1, cols + 1), (3, cols + 5), (8, cols + 16)):
                rows = 9
                buf = torch.randn(rows * ld + off, generator=g, device=DEV).to(t)
                x = buf[off:].view(rows, ld)[:, :cols]
                keep, rest = x.clone(), buf[off:].view(rows, ld)[:, cols:].clone()
                w, b = (torch.randn(cols, generator=g, device=DEV).to(t) for _ in range(2))
                dsa.dsa_layernorm(x, w, b, EPS, out=x)  # in place
                check_forward(keep, None, w, b, None, x, None, None, 0, f"in place {cols} {off}")
                assert torch.equal(buf[off:].view(rows, ld)[:, cols:], rest)


def test_special_rows():
    """A row of equal values is the bias; NaN and infinities stay in their row."""
    dsa = lib()
    for cols in (8, 128, 1111, 4096):
        x = torch.randn((4, cols), device=DEV)
        x[0] = 3.25
        x[1, cols // 2] = float("nan")
        x[2, 0] = float("inf")
        w, b = torch.randn(cols, device=DEV), torch.randn(cols, device=DEV)
        out = torch.empty_like(x)
        dsa.dsa_layernorm(x, w, b, EPS, out=out)
        assert torch.equal(out[0], b)
        assert torch.isnan(out[1]).all() and not torch.isfinite(out[2]).any()
        check_forward(x[3:], None, w, b, None, out[3:], None, None, 0, "beside them")


def test_no_rows_and_graph_and_streams():
    dsa, g = lib(), gen(9)
    cols = 300
    w, b = torch.randn(cols, device=DEV), torch.randn(cols, device=DEV)
    empty = torch.empty((0, cols), device=DEV)
    dw, db = torch.full((cols,), 9.0, device=DEV), torch.full((cols,), 9.0, device=DEV)
    dsa.dsa_layernorm(empty, w, b, EPS, out=empty)
    dsa.dsa_layernorm_backward(empty, empty, w, EPS, empty, dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all()
    x, dy = torch.randn((50, cols), generator=g, device=DEV), torch.randn((50, cols), generator=g, device=DEV)
    out, dx = torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dsa.dsa_layernorm(x, w, b, EPS, out=out, stream=side)
    dsa.dsa_layernorm_backward(dy, x, w, EPS, dx, dw, dbias=db, stream=side)
    torch.cuda.synchronize()
    check_backward(dy, x, w, None, dx, dw, db, "side stream")
    ws = torch.empty(dsa.dsa_layernorm_backward_workspace_size(50, cols), dtype=U8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.dsa_layernorm(x, w, b, EPS, out=out)
        dsa.dsa_layernorm_backward(dy, x, w, EPS, dx, dw, dbias=db, workspace=ws)
    x.copy_(torch.randn((50, cols), generator=g, device=DEV) + 2)
    graph.replay()
    torch.cuda.synchronize()
    check_forward(x, None, w, b, None, out, None, None, 0, "replayed")
    check_backward(dy, x, w, None, dx, dw, db, "replayed")
    assert dsa.dsa_get_device_status() == 0
