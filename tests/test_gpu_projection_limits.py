"""The FP8 product, block quantisation and layer norm at the ends of what their documentation allows: offsets beyond 32
bits, very many rows, one tensor in two places, results in place of inputs."""
import pytest
import torch

from tests import operator_refs as R
from tests import projection_refs as P
from tests.gpu_util import lib
from tests.test_gpu_gemm_fp8 import check as check_gemm
from tests.test_gpu_gemm_fp8 import gen, operands

pytestmark = pytest.mark.gpu
DEV, EPS = "cuda", 1e-6
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def far(rows, cols, ld, dtype, like=None):
    """[rows, cols] with rows ld elements apart."""
    t = torch.empty((rows - 1) * ld + cols, dtype=dtype, device=DEV).as_strided((rows, cols), (ld, 1))
    if like is not None:
        t.copy_(like)
    return t


@pytest.mark.parametrize("M, N, K", [(40, 70, 300), (200, 150, 300), (150, 200, 2100)])
@pytest.mark.parametrize("block", [128, 1])
def test_product_of_rows_far_apart(M, N, K, block):
    dsa, g = lib(), gen(1)
    a, sa, b, sb = operands(M, N, K, block, g)
    want = torch.empty((M, N), device=DEV)
    dsa.dsa_gemm_fp8(a, sa, b, sb, want)
    check_gemm(want, a, sa, b, sb, "near")
    ld = ((1 << 32) // min(M, N) + 4096) // 16 * 16 * 2  # the last rows lie beyond 2^33 bytes
    out = far(M, N, ld // 4, F32)
    dsa.dsa_gemm_fp8(far(M, K, ld, U8, a), sa, far(N, K, ld, U8, b), sb, out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_codes_of_rows_far_apart(t, block_rows):
    dsa, g = lib(), gen(2)
    rows, cols = 50, 300
    x = torch.randn((rows, cols), generator=g, device=DEV).to(t)
    s_shape, t_shape = (P.pieces(rows) if block_rows == 128 else rows, 3), (3 if block_rows == 128 else cols, 1)

    def run(x, codes, codes_t):
        s, st = torch.zeros(s_shape, device=DEV), torch.zeros(t_shape, device=DEV)
        dsa.dsa_quantize_fp8_blocks(x, codes, s, codes_t, st, block_rows=block_rows)
        s2, c2 = torch.zeros_like(s), torch.empty_strided(codes.shape, codes.stride(), dtype=U8, device=DEV)
        dsa.dsa_quantize_fp8_blocks(x, c2, s2, block_rows=block_rows)
        assert torch.equal(s, s2) and torch.equal(codes, c2)
        return codes, s, codes_t, st

    want = run(x, torch.zeros((rows, cols), dtype=U8, device=DEV), torch.zeros((cols, rows), dtype=U8, device=DEV))
    ld, ld_t = (1 << 32) // 40 // 16 * 16, (1 << 32) // 240 // 16 * 16
    got = run(far(rows, cols, (1 << 32) // 40, t, x), far(rows, cols, ld, U8), far(cols, rows, ld_t, U8))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_norm_of_rows_far_apart():
    dsa, g = lib(), gen(3)
    rows = 20
    for cols in (128, 1030):
        x, r = (torch.randn((rows, cols), generator=g, device=DEV).to(BF) for _ in range(2))
        w, b = (torch.randn(cols, generator=g, device=DEV) for _ in range(2))
        h, y = torch.empty_like(x), torch.empty_like(x)
        dsa.dsa_layernorm(x, w, b, EPS, out=y, residual=r, residual_out=h)
        ld = (1 << 32) // 16 if cols == 128 else (1 << 32) // 16 + 1
        h2, y2 = far(rows, cols, ld, BF), far(rows, cols, ld, BF)
        dsa.dsa_layernorm(far(rows, cols, ld, BF, x), w, b, EPS, out=y2, residual=far(rows, cols, ld, BF, r), residual_out=h2)
        if cols == 128:
            assert torch.equal(y, y2) and torch.equal(h, h2)
        else:  # another order of a row's sums
            assert torch.equal(h, h2)
            _, ref, mag = P.layernorm(x, r, w, b, EPS)
            R.check_close(y2, ref, ref.abs() * R.BF16 + 40 * R.FP32 * mag + 1e-30, "far")


def test_more_rows_than_32_bits_count():
    dsa = lib()
    rows = (1 << 31) + 5
    x = torch.randint(-3, 4, (rows, 1), dtype=torch.int8, device=DEV).to(BF)
    want = torch.where(x > 0, 0x7E, torch.where(x < 0, 0xFE, 0)).to(U8)  # a value alone is its scale's largest
    codes, scale = torch.full((rows, 1), 1, dtype=U8, device=DEV), torch.zeros((rows, 1), device=DEV)
    dsa.dsa_quantize_fp8_blocks(x, codes, scale)
    assert torch.equal(codes, want)
    assert torch.equal(scale[-100000:], torch.where(x[-100000:] == 0, 1.0, x[-100000:].float().abs().double() / 448).float())
    scale_t = torch.zeros((1, P.pieces(rows)), device=DEV)
    codes_t = torch.full((1, rows), 1, dtype=U8, device=DEV)
    dsa.dsa_quantize_fp8_blocks(x, codes_t=codes_t, scale_t=scale_t)
    n = 1 << 20
    for lo in (0, (1 << 31) - n // 2 // 128 * 128, rows - rows % 128 - n):
        v = x[lo:lo + n + 128].flatten()
        v = torch.cat([v, torch.zeros(-len(v) % 128, dtype=BF, device=DEV)]).view(-1, 128).float()
        s = v.abs().amax(1)
        s = torch.where(s == 0, 1.0, s.double() / 448).float()
        assert torch.equal(scale_t[0, lo // 128:lo // 128 + len(s)], s)
        got = P.values(codes_t[0, lo:lo + n + 128])
        ref = (v.double() / s.double()[:, None]).flatten()[:len(got)]
        assert ((got - ref).abs() <= ref.abs() * R.E4M3 * (1 + 1e-5)).all()


def test_product_and_norm_of_very_many_rows():
    dsa, g = lib(), gen(4)
    rows, cols = (1 << 25) + 3, 128  # 2^32 values
    pick = torch.tensor([0, 1, 127, 128, 1 << 20, (1 << 24) - 1, 1 << 24, (1 << 25) - 1, 1 << 25, rows - 1], device=DEV)
    x = torch.randn((rows, cols), generator=g, device=DEV, dtype=BF)
    w, b = (torch.randn(cols, generator=g, device=DEV) for _ in range(2))
    y, codes, scale = torch.empty_like(x), torch.empty((rows, cols), dtype=U8, device=DEV), torch.empty((rows, 1), device=DEV)
    dsa.dsa_layernorm(x, w, b, EPS, out=y, codes=codes, scale=scale, block=128)
    _, ref, mag = P.layernorm(x[pick], None, w, b, EPS)
    R.check_close(y[pick], ref, ref.abs() * R.BF16 + 40 * R.FP32 * mag + 1e-30, "norm")
    bs, b8 = P.scales_like((1, 1), g, DEV), P.codes_like(65, cols, g, DEV)
    out = torch.empty((rows, 65), dtype=BF, device=DEV)
    dsa.dsa_gemm_fp8(codes, scale, b8, bs, out)
    check_gemm(out[pick], codes[pick], scale[pick], b8, bs, "product")
    del out, codes
    dx, dw, db = torch.empty_like(x), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    dsa.dsa_layernorm_backward(y, x, w, EPS, dx, dw, dbias=db)
    rx, _, _, xmag, _, _ = P.layernorm_backward(y[pick], x[pick], w, None, EPS)
    R.check_close(dx[pick], rx, rx.abs() * R.BF16 + 120 * R.FP32 * xmag + 1e-30, "dx")
    want, size = torch.zeros(cols, dtype=torch.float64, device=DEV), torch.zeros(cols, dtype=torch.float64, device=DEV)
    for part in y.split(1 << 22):
        want += part.double().sum(0)
        size += part.double().abs().sum(0)
    # a column's sum is a chain of each of the CTAs' rows, 304 CTAs of 32 rows at least at work, and theirs joined
    chain = rows / (304 * 32) + 500
    assert ((db.double() - want).abs() <= chain * R.FP32 * size).all()


@pytest.mark.parametrize("cols, t", [(128, F32), (100, BF), (1030, F32), (2048, BF), (8192, BF)])
def test_gradients_in_place(cols, t):
    """dx in dy's, dres's or h's place, and one tensor as dy, h and dres."""
    dsa, g = lib(), gen(5)
    rows = 333
    dy, h, e = (torch.randn((rows, cols), generator=g, device=DEV).to(t) for _ in range(3))
    w = torch.randn(cols, generator=g, device=DEV)

    def run(dy, h, e, dx):
        dw, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
        dsa.dsa_layernorm_backward(dy, h, w, EPS, dx, dw, dbias=db, dres=e)
        return dx, dw, db

    want = run(dy, h, e, torch.empty_like(h))
    for k in range(3):
        args = [dy.clone(), h.clone(), e.clone()]
        assert all(torch.equal(a, b) for a, b in zip(run(*args, args[k]), want))
    assert all(torch.equal(a, b) for a, b in zip(run(h, h, h, torch.empty_like(h)), run(h.clone(), h.clone(), h.clone(), torch.empty_like(h))))


@pytest.mark.parametrize("cols, t", [(128, BF), (100, F32), (1030, BF), (8192, BF), (4096, F32)])
def test_norm_in_place_of_its_inputs(cols, t):
    """residual_out in the residual's or x's place, out in x's, and one tensor as x and residual."""
    dsa, g = lib(), gen(6)
    x, r = (torch.randn((200, cols), generator=g, device=DEV).to(t) for _ in range(2))
    w, b = (torch.randn(cols, generator=g, device=DEV) for _ in range(2))

    def run(x, r, out, h):
        dsa.dsa_layernorm(x, w, b, EPS, out=out, residual=r, residual_out=h)
        return out.clone(), h.clone()

    want = run(x, r, torch.empty_like(x), torch.empty_like(x))
    for where in ("x", "r", "both"):
        x2, r2 = x.clone(), r.clone()
        got = run(x2, r2, x2 if where == "both" else torch.empty_like(x), x2 if where == "x" else r2)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), where
    twice = run(x, x, torch.empty_like(x), torch.empty_like(x))
    assert all(torch.equal(a, b) for a, b in zip(twice, run(x, x.clone(), torch.empty_like(x), torch.empty_like(x))))


@pytest.mark.parametrize("M, N, K", [(3, 5, (1 << 20) + 5), (70, 40, (1 << 20) + 5), (1, (1 << 20) + 3, 130), (60, 100001, 20), ((1 << 20) + 3, 1, 130)])
@pytest.mark.parametrize("block", [128, 1])
def test_product_of_long_sides(M, N, K, block):
    dsa, g = lib(), gen(9)
    ops = operands(M, N, K, block, g)
    out = torch.full((M, N), float("nan"), device=DEV)
    dsa.dsa_gemm_fp8(*ops, out)
    check_gemm(out, *ops, "long")
    assert dsa.dsa_get_device_status() == 0


@pytest.mark.parametrize("M, K", [(5, 300), (50, 1000), (300, 700), (2050, 1100)])
def test_product_of_a_tensor_with_itself(M, K):
    dsa, g = lib(), gen(7)
    a, sa = P.codes_like(M, K, g, DEV), P.scales_like((M, P.pieces(K)), g, DEV)
    out, want = torch.empty((M, M), device=DEV), torch.empty((M, M), device=DEV)
    dsa.dsa_gemm_fp8(a, sa, a, sa, out)
    dsa.dsa_gemm_fp8(a, sa, a.as_strided(a.shape, a.stride()), sa.clone(), want)
    assert torch.equal(out, want)
    check_gemm(out, a, sa, a, sa, "a a^T")


@pytest.mark.parametrize("rows, cols", [(19, 16385), (130, 2431), (300, 4099), (2433, 2003), (2500, 2000), (40001, 100), (1, 3000001)])
@pytest.mark.parametrize("t", [BF, F32])
def test_codes_alone_are_those_beside_the_transpose(rows, cols, t):
    """... whichever of the ways a number of pieces goes."""
    dsa, g = lib(), gen(8)
    x = (torch.randn((rows, cols), generator=g, device=DEV) * torch.exp(torch.randn((rows, 1), generator=g, device=DEV))).to(t)
    got = []
    for turned in (True, False):
        codes, scale = P.padded(rows, cols, DEV), torch.full((rows, P.pieces(cols)), -1.0, device=DEV)
        codes_t, scale_t = (P.padded(cols, rows, DEV), torch.empty((cols, P.pieces(rows)), device=DEV)) if turned else (None, None)
        dsa.dsa_quantize_fp8_blocks(x, codes, scale, codes_t, scale_t)
        got.append((codes, scale))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    s = got[0][1].double().repeat_interleave(128, 1)[:, :cols]
    ref = x.double() / s
    assert ((P.values(got[0][0]) - ref).abs() <= ref.abs() * (R.E4M3 * (1 + 1e-5)) + 2.0 ** -10).all()
