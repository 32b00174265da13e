"""The product of FP8 operands with a scale for every 128 values, against fp64."""
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


def operands(M, N, K, block, g):
    return (P.codes_like(M, K, g, DEV), P.scales_like((M, P.pieces(K)), g, DEV), P.codes_like(N, K, g, DEV),
            P.scales_like((P.pieces(N) if block == 128 else N, P.pieces(K)), g, DEV))


def check(out, a, a_scale, b, b_scale, what):
    ref, mag = P.gemm(a, a_scale, b, b_scale)
    R.check_close(out, ref.cpu(), P.gemm_bound(ref, mag, a.shape[1], out.dtype).cpu(), what)


SIZES = [(1, 1, 1), (1, 1, 128), (1, 704, 4096), (2, 127, 129), (7, 129, 127), (16, 128, 256), (17, 130, 1000), (31, 64, 2050), (33, 257, 128),
         (63, 300, 640), (64, 1536, 1536), (65, 192, 384), (100, 1000, 130), (127, 255, 513), (128, 128, 128), (129, 257, 129),
         (255, 130, 1024), (256, 256, 256), (257, 513, 300), (300, 1111, 2050), (513, 640, 777), (1000, 2000, 512), (2049, 1025, 384)]


@pytest.mark.parametrize("block", [128, 1])
@pytest.mark.parametrize("M, N, K", SIZES)
def test_sizes(M, N, K, block):
    dsa, g = lib(), gen(M * 31 + N * 7 + K + block)
    ops = operands(M, N, K, block, g)
    for t in (BF, F32):
        out = torch.full((M, N), float("nan"), dtype=t, device=DEV)
        assert dsa.dsa_gemm_fp8(*ops, out) is out
        check(out, *ops, f"{M} x {N} x {K} {t}")
    assert dsa.dsa_get_device_status() == 0


@pytest.mark.parametrize("M, N, K", [(5, 200, 300), (300, 200, 300), (513, 515, 640)])
@pytest.mark.parametrize("t", [BF, F32])
def test_output_rows_apart_and_at_any_address(M, N, K, t):
    """Strided output rows, from aligned ones to single elements off; what lies between them stays."""
    dsa, g = lib(), gen(3)
    ops = operands(M, N, K, 128, g)
    want = torch.empty((M, N), dtype=t, device=DEV)
    dsa.dsa_gemm_fp8(*ops, want)
    check(want, *ops, "contiguous")
    for off, ld in ((0, N + 32), (1, N + 3), (8, (N + 31) // 8 * 8 + 8), (2, N + 4)):
        buf = torch.full((M * ld + off + 8,), -7.0, dtype=t, device=DEV)
        view = buf[off:off + M * ld].view(M, ld)
        dsa.dsa_gemm_fp8(*ops, view[:, :N])
        assert torch.equal(view[:, :N], want), (off, ld)
        assert (view[:, N:] == -7.0).all() and (buf[:off] == -7.0).all() and (buf[off + M * ld:] == -7.0).all()


def test_operand_rows_apart():
    """Operands that are columns of wider tensors: bytes behind K are never used (they are NaN codes here)."""
    dsa, g = lib(), gen(4)
    for M, N, K in ((40, 300, 200), (400, 520, 200)):
        wide_a, wide_b = torch.full((M, 512), 0x7F, dtype=U8, device=DEV), torch.full((N, 768), 0x7F, dtype=U8, device=DEV)
        a, b = wide_a[:, 16:16 + K], wide_b[:, 256:256 + K]
        a.copy_(P.codes_like(M, K, g, DEV))
        b.copy_(P.codes_like(N, K, g, DEV))
        sa, sb = P.scales_like((M, 2), g, DEV), P.scales_like((P.pieces(N), 2), g, DEV)
        out = torch.empty((M, N), device=DEV)
        dsa.dsa_gemm_fp8(a, sa, b, sb, out)
        check(out, a, sa, b, sb, "columns of wider tensors")


@pytest.mark.parametrize("M, N", [(3, 200), (300, 400), (700, 700)])
@pytest.mark.parametrize("block", [128, 1])
def test_one_code_at_a_time(M, N, block):
    """A single value in each operand: its place and its two scales, exactly."""
    dsa = lib()
    K = 400
    for m, n, k in ((0, 0, 0), (M - 1, N - 1, K - 1), (M // 2, N // 3, 128), (M - 1, 0, 127), (0, N - 1, 256)):
        a, b = P.padded(M, K, DEV), P.padded(N, K, DEV)
        a.zero_()
        b.zero_()
        a[m, k], b[n, k] = 0x38, 0xC0  # 1 and -2
        sa = torch.zeros((M, 4), device=DEV)
        sb = torch.zeros((P.pieces(N) if block == 128 else N, 4), device=DEV)
        sa[m, k // 128], sb[n // 128 if block == 128 else n, k // 128] = 3.0, 0.25
        out = torch.full((M, N), float("nan"), device=DEV)
        dsa.dsa_gemm_fp8(a, sa, b, sb, out)
        want = torch.zeros((M, N), device=DEV)
        want[m, n] = -1.5
        assert torch.equal(out, want)


@pytest.mark.parametrize("M, N, K", [(4, 300, 700), (300, 400, 700), (600, 520, 300)])
def test_nan_stays_in_its_row_and_column(M, N, K):
    dsa, g = lib(), gen(5)
    a, sa, b, sb = operands(M, N, K, 1, g)
    clean = torch.empty((M, N), device=DEV)
    dsa.dsa_gemm_fp8(a, sa, b, sb, clean)
    a[M // 2, K - 1], sb[N // 2, 1] = 0xFF, float("inf")
    a[M // 2 - 1, 200] = 0  # whatever it meets there
    dsa.dsa_gemm_fp8(a, sa, b, sb, clean2 := torch.empty_like(clean))
    keep_m, keep_n = torch.ones(M, dtype=torch.bool), torch.ones(N, dtype=torch.bool)
    keep_m[[M // 2, M // 2 - 1]] = False
    keep_n[N // 2] = False
    assert torch.isnan(clean2[M // 2]).all()
    assert not torch.isfinite(clean2[:, N // 2]).any() or (P.values(b[N // 2, 128:256]) == 0).all()
    assert torch.equal(clean2[keep_m][:, keep_n], clean[keep_m][:, keep_n])


def test_empty_sizes():
    dsa = lib()
    z = torch.empty((0, 0), device=DEV)
    for M, N in ((3, 5), (300, 400), (1, 1)):
        out = torch.full((M, N + 3), 5.0, device=DEV)
        u = torch.empty((M, 0), dtype=U8, device=DEV)
        dsa.dsa_gemm_fp8(u, torch.empty((M, 0), device=DEV), torch.empty((N, 0), dtype=U8, device=DEV),
                         torch.empty((P.pieces(N), 0), device=DEV), out[:, :N])
        assert (out[:, :N] == 0).all() and (out[:, N:] == 5.0).all()
    u, s = torch.zeros((4, 128), dtype=U8, device=DEV), torch.ones((4, 1), device=DEV)
    none_u, none_s = torch.empty((0, 128), dtype=U8, device=DEV), torch.empty((0, 1), device=DEV)
    dsa.dsa_gemm_fp8(none_u, none_s, u, s, torch.empty((0, 4), device=DEV))
    dsa.dsa_gemm_fp8(u, s, none_u, none_s, torch.empty((4, 0), device=DEV))
    assert z.numel() == 0 and dsa.dsa_get_device_status() == 0


@pytest.mark.parametrize("M, N, K", [(1, 704, 4096), (64, 2048, 1536), (777, 1111, 2050), (1200, 1300, 900)])
def test_repeats_bit_for_bit(M, N, K):
    """... also beside other work on another stream."""
    dsa, g = lib(), gen(6)
    ops = operands(M, N, K, 128, g)
    want = torch.empty((M, N), device=DEV)
    dsa.dsa_gemm_fp8(*ops, want)
    check(want, *ops, "first")
    other, busy = torch.cuda.Stream(), torch.randn((2048, 2048), device=DEV)
    torch.cuda.synchronize()
    outs = []
    for i in range(20):
        if i >= 10:
            with torch.cuda.stream(other):
                busy @ busy
        outs.append(torch.empty_like(want))
        dsa.dsa_gemm_fp8(*ops, outs[-1])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_two_streams_and_a_graph():
    """Calls on two streams at once, and one captured and replayed on new operands."""
    dsa, g = lib(), gen(7)
    big, small = operands(700, 800, 1000, 1, g), operands(8, 1024, 2048, 128, g)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [(torch.empty((700, 800), device=DEV), torch.empty((8, 1024), dtype=BF, device=DEV)) for _ in range(5)]
    torch.cuda.synchronize()
    for o1, o2 in outs:
        dsa.dsa_gemm_fp8(*big, o1, stream=s1)
        dsa.dsa_gemm_fp8(*small, o2, stream=s2)
    torch.cuda.synchronize()
    for o1, o2 in outs:
        check(o1, *big, "stream 1")
        check(o2, *small, "stream 2")
    graph = torch.cuda.CUDAGraph()
    o1, o2 = outs[0]
    with torch.cuda.graph(graph):
        dsa.dsa_gemm_fp8(*big, o1)
        dsa.dsa_gemm_fp8(*small, o2)
    for _ in range(2):
        for t in (big[0], big[2], small[0], small[2]):
            t.copy_(P.codes_like(*t.shape, g, DEV))
        o1.fill_(float("nan"))
        o2.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(o1, *big, "replayed")
        check(o2, *small, "replayed")
    assert dsa.dsa_get_device_status() == 0
