"""FP8 codes and scales of a matrix and its transpose, per 128 values or per block, against the definition."""
import pytest
import torch

from tests import operator_refs as R
from tests import projection_refs as P
from tests.gpu_util import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def by_definition(x, block_rows, mode):
    """Codes and scales in fp32, operation by operation what the header states: exactly what the kernel has to give."""
    rows, cols = x.shape
    wide = torch.nn.functional.pad(x.float(), (0, -cols % 128, 0, -rows % block_rows))
    cut = wide.view(wide.shape[0] // block_rows, block_rows, -1, 128)
    # through fp64: a tensor over a number is taken as a product with the number's reciprocal, not as a quotient
    ratio = (cut.abs().amax((1, 3)).double() / 448.0).float()
    if mode == 1:
        m, e = torch.frexp(ratio)
        ratio = torch.ldexp(torch.ones_like(m), e - (m == 0.5).int())
        ratio = torch.where(m == 0, torch.zeros_like(ratio), ratio)
    scale = torch.where(ratio > 0, ratio, torch.ones_like(ratio))
    q = (cut / scale[:, None, :, None]).clamp(-448, 448)
    return q.to(torch.float8_e4m3fn).view(U8).view(wide.shape)[:rows, :cols], scale


def uneven(rows, cols, g):
    x = torch.randn((rows, cols), generator=g, device=DEV) * torch.randn((1, cols), generator=g, device=DEV).exp()
    x *= torch.randn((rows, 1), generator=g, device=DEV).mul_(2).exp_()
    x[rows // 2, cols // 2:] = 0  # a piece of zeros where the row is long
    return x


SIZES = [(1, 1), (1, 128), (1, 4096), (3, 130), (15, 64), (64, 4096), (127, 129), (128, 128), (129, 127), (200, 1111), (513, 640),
         (1000, 72), (2050, 257)]


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows, cols", SIZES)
@pytest.mark.parametrize("t", [BF, F32])
def test_sizes(rows, cols, block_rows, mode, t):
    dsa, g = lib(), gen(rows + 3 * cols)
    x = uneven(rows, cols, g).to(t)
    want = by_definition(x, block_rows, mode) + by_definition(x.T, block_rows, mode)
    for plain, turned in ((True, True), (True, False), (False, True)):
        got = [None] * 4
        if plain:
            got[0], got[1] = P.padded(rows, cols, DEV, 0x11), torch.full(want[1].shape, -1.0, device=DEV)
        if turned:
            got[2], got[3] = P.padded(cols, rows, DEV, 0x11), torch.full(want[3].shape, -1.0, device=DEV)
        assert dsa.dsa_quantize_fp8_blocks(x, *got, block_rows=block_rows, scale_mode=mode) == tuple(got)
        for i in range(4):
            if got[i] is None:
                continue
            a, b = got[i], want[i]
            if i % 2 == 0:  # the sign of zero is the input's
                assert torch.equal(a, b), (i, plain, turned)
                rest = a._base[:, a.shape[1]:]
                assert (rest == 0x11).all(), "bytes between rows"
            else:
                assert torch.equal(a, b), (i, plain, turned)
    assert dsa.dsa_get_device_status() == 0


@pytest.mark.parametrize("t", [BF, F32])
def test_any_address_and_stride(t):
    """Inputs and outputs off every alignment give what aligned ones give, and touch nothing between their rows."""
    dsa, g = lib(), gen(1)
    rows, cols = 150, 300
    x = uneven(rows, cols, g).to(t)
    for block_rows in (1, 128):
        want = by_definition(x, block_rows, 0) + by_definition(x.T, block_rows, 0)
        for off, ld in ((0, 300), (1, 301), (2, 304), (3, 303), (8, 320), (4, 316), (5, 309), (7, 300)):
            buf = torch.full((rows * ld + off + 16,), float("nan"), dtype=t, device=DEV)
            view = buf[off:off + rows * ld].view(rows, ld)[:, :cols]
            view.copy_(x)
            c = torch.full((rows * ld + off,), 0x11, dtype=U8, device=DEV)[off:].view(rows, ld)
            ct = torch.full((cols * (150 + off) + off,), 0x11, dtype=U8, device=DEV)[off:].view(cols, 150 + off)
            s, st = torch.empty(want[1].shape, device=DEV), torch.empty(want[3].shape, device=DEV)
            dsa.dsa_quantize_fp8_blocks(view, c[:, :cols], s, ct[:, :rows], st, block_rows=block_rows)
            assert torch.equal(c[:, :cols], want[0]) and torch.equal(s, want[1]), (off, ld)
            assert torch.equal(ct[:, :rows], want[2]) and torch.equal(st, want[3]), (off, ld)
            assert (c[:, cols:] == 0x11).all() and (ct[:, rows:] == 0x11).all()


def test_extreme_magnitudes():
    """The largest and smallest fp32 values: scales that underflow, quotients that could overflow on the way."""
    dsa = lib()
    x = torch.zeros((4, 256), device=DEV)
    x[0, 0], x[0, 1] = 3.4e38, -1.0
    x[1, 0], x[1, 1] = 1e-45, 1e-40
    x[2, 130], x[2, 131] = 1.2e-38, -1e-38
    x[3, :128] = torch.linspace(-1e30, 1e30, 128, device=DEV)
    for mode in (0, 1):
        want = by_definition(x, 1, mode) + by_definition(x.T, 1, mode)
        got = [P.padded(4, 256, DEV), torch.empty((4, 2), device=DEV), P.padded(256, 4, DEV), torch.empty((256, 1), device=DEV)]
        dsa.dsa_quantize_fp8_blocks(x, *got, scale_mode=mode)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_no_rows():
    dsa = lib()
    x = torch.empty((0, 256), dtype=BF, device=DEV)
    c, s = torch.empty((0, 256), dtype=U8, device=DEV), torch.empty((0, 2), device=DEV)
    ct, st = torch.empty((256, 0), dtype=U8, device=DEV), torch.empty((256, 0), device=DEV)
    dsa.dsa_quantize_fp8_blocks(x, c, s, ct, st)
    assert dsa.dsa_get_device_status() == 0
