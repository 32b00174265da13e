"""The FP8 product where tiles of each width, several tiles a CTA, and splits of K are what it takes, against fp64."""
import subprocess
import sys

import pytest
import torch

from tests import projection_refs as P
from tests.gpu_util import lib
from tests.test_gpu_gemm_fp8 import check, gen, operands

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8

# few tiles with K split in 8, 4 and 2, tiles that nearly fill the GPU, and several a CTA
SIZES = [(300, 700, 5001), (822, 727, 5397), (1987, 581, 7525), (520, 1600, 4100), (129, 1000, 8191), (300, 1111, 2305), (2040, 2100, 1900),
         (2039, 2301, 1801), (4500, 700, 4100), (3000, 4000, 1300), (4099, 2999, 140), (5000, 2600, 300), (130, 20001, 300), (20001, 130, 300)]


@pytest.mark.parametrize("block", [128, 1])
@pytest.mark.parametrize("M, N, K", SIZES)
def test_sizes(M, N, K, block):
    """Output rows at multiples of 16 bytes, and at single elements of an odd pitch; what lies between them stays."""
    dsa, g = lib(), gen(M + N + K + block)
    ops = operands(M, N, K, block, g)
    for t in (BF, F32):
        buf = torch.full((M, (N + 7) // 8 * 8), -7.0, dtype=t, device=DEV)
        dsa.dsa_gemm_fp8(*ops, buf[:, :N])
        check(buf[:, :N], *ops, f"{M} x {N} x {K} {t}")
        assert (buf[:, N:] == -7.0).all()
        odd = torch.full((M, N // 2 * 2 + 3), -7.0, dtype=t, device=DEV)
        dsa.dsa_gemm_fp8(*ops, odd[:, 1:N + 1])
        assert torch.equal(odd[:, 1:N + 1], buf[:, :N]) and (odd[:, 0] == -7.0).all() and (odd[:, N + 1:] == -7.0).all()
    assert dsa.dsa_get_device_status() == 0


@pytest.mark.parametrize("M, N, K", [(2040, 2100, 1900), (3000, 4000, 1300), (300, 700, 5001), (1987, 581, 7525)])
@pytest.mark.parametrize("block", [128, 1])
def test_one_code_at_a_time(M, N, K, block):
    dsa, k_pieces = lib(), P.pieces(K)
    a, b = P.padded(M, K, DEV), P.padded(N, K, DEV)
    a.zero_()
    b.zero_()
    sa = torch.zeros((M, k_pieces), device=DEV)
    sb = torch.zeros((P.pieces(N) if block == 128 else N, k_pieces), device=DEV)
    out = torch.empty((M, N), device=DEV)
    for m, n, k in ((0, 0, 0), (M - 1, N - 1, K - 1), (M // 2, N // 3, 1024), (M - 1, 191, 127), (127, N - 1, 256), (128, 192, 1151), (5, 256, 640)):
        nb = n // 128 if block == 128 else n
        a[m, k], b[n, k], sa[m, k // 128], sb[nb, k // 128] = 0x38, 0xC0, 3.0, 0.25  # 1 and -2
        out.fill_(float("nan"))
        dsa.dsa_gemm_fp8(a, sa, b, sb, out)
        assert out[m, n] == -1.5 and torch.count_nonzero(out) == 1, (m, n, k)
        a[m, k], b[n, k], sa[m, k // 128], sb[nb, k // 128] = 0, 0, 0.0, 0.0


@pytest.mark.parametrize("M, N, K", [(2040, 2100, 1900), (3000, 4000, 1300), (822, 727, 5397)])
@pytest.mark.parametrize("block", [128, 1])
def test_nan_and_repeats(M, N, K, block):
    """NaN codes in a row and an infinite scale of a row stay there; runs beside other work repeat bit for bit."""
    dsa, g = lib(), gen(8)
    a, sa, b, sb = operands(M, N, K, block, g)
    clean = torch.empty((M, N), device=DEV)
    dsa.dsa_gemm_fp8(a, sa, b, sb, clean)
    check(clean, a, sa, b, sb, "first")
    other, busy = torch.cuda.Stream(), torch.randn((2048, 2048), device=DEV)
    torch.cuda.synchronize()
    for _ in range(8):
        with torch.cuda.stream(other):
            busy @ busy
        again = torch.full_like(clean, float("nan"))
        dsa.dsa_gemm_fp8(a, sa, b, sb, again)
        assert torch.equal(again, clean)
    a[M // 2, K - 1], b[N // 3, 7], sa[M - 1, 0] = 0xFF, 0x7F, float("inf")
    dsa.dsa_gemm_fp8(a, sa, b, sb, again)
    keep_m, keep_n = torch.ones(M, dtype=torch.bool, device=DEV), torch.ones(N, dtype=torch.bool, device=DEV)
    keep_m[[M // 2, M - 1]] = False
    keep_n[N // 3] = False
    assert torch.isnan(again[M // 2]).all() and torch.isnan(again[:, N // 3]).all() and not torch.isfinite(again[M - 1]).any()
    assert torch.equal(again[keep_m][:, keep_n], clean[keep_m][:, keep_n])


FIRST = """
import torch
from tests.test_gpu_gemm_fp8 import check, gen, operands
from tests.gpu_util import lib
dsa, g = lib(), gen(9)
sets = [(operands(*s, b, g), torch.empty(s[:2], device="cuda")) for s in ((2040, 2100, 1900), (300, 700, 5001), (4, 300, 900)) for b in (128, 1)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for ops, out in sets:
        dsa.dsa_gemm_fp8(*ops, out)
for _ in range(2):
    for _, out in sets:
        out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    for ops, out in sets:
        check(out, *ops, "captured first")
print("captured first")
"""


def test_first_calls_of_a_process_captured():
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("M", [1, 20, 50])
@pytest.mark.parametrize("tiles", [16, 34, 35, 38, 68, 69, 76, 77, 152, 153])
def test_few_rows_by_every_number_of_tiles(M, tiles):
    """... with K split in 8, 4, 2 and not at all."""
    dsa, g = lib(), gen(tiles)
    ops = operands(M, 128 * tiles - 5, 2100, 128, g)
    out = torch.full((M, 128 * tiles - 5), float("nan"), device=DEV)
    dsa.dsa_gemm_fp8(*ops, out)
    check(out, *ops, f"{M} rows, {tiles} tiles")
