"""The FP8 product at the ends of what its scales may be: the two of a piece are multiplied first, in fp32."""
import pytest
import torch

from tests import operator_refs as R
from tests import projection_refs as P
from tests.gpu_util import lib
from tests.test_gpu_gemm_fp8 import gen

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8

# few rows in 16, 32 and 64 columns, with and without a split of K; tiles of 128, 192 and 256, with and without
SIZES = [(1, 200, 300), (5, 300, 4096), (30, 200, 1000), (60, 300, 2100), (60, 20000, 400), (200, 300, 2100), (300, 300, 300),
         (1000, 2000, 500), (2048, 4096, 600), (4096, 4096, 384)]


def small_codes(rows, cols, g):
    """Codes of -15 to 15 steps of 2^-9: a piece's sum is below 2^-3."""
    c = P.padded(rows, cols, DEV)
    c.copy_(torch.randint(0, 16, (rows, cols), generator=g, device=DEV) | torch.randint(0, 2, (rows, cols), generator=g, device=DEV) << 7)
    return c


@pytest.mark.parametrize("M, N, K", SIZES)
@pytest.mark.parametrize("block", [128, 1])
@pytest.mark.parametrize("ea, eb", [(-63, -63), (62, 62), (62, -63), (-63, 62), (0, 0)])
def test_scales_of_every_allowed_size(M, N, K, block, ea, eb):
    dsa, g = lib(), gen(M + N + K)
    a, b = small_codes(M, K, g), small_codes(N, K, g)

    def scales(rows, e):
        """From 2^e to 2^(e + 1), some of them 0."""
        s = torch.exp2(torch.rand((rows, P.pieces(K)), generator=g, device=DEV).clamp(max=0.999) + e)
        return torch.where(torch.rand(s.shape, generator=g, device=DEV) < 0.1, 0.0, s)

    sa, sb = scales(M, ea), scales(P.pieces(N) if block == 128 else N, eb)
    rows = torch.randperm(M, generator=g, device=DEV)[:64]
    for t in (F32, BF):
        out = torch.full((M, N), float("nan"), dtype=t, device=DEV)
        dsa.dsa_gemm_fp8(a, sa, b, sb, out)
        assert torch.isfinite(out).all()
        va = P.values(a[rows]) * P.spread(sa[rows], len(rows), K, 1)
        vb = P.values(b) * P.spread(sb, N, K, block)
        ref, mag = va @ vb.T, va.abs() @ vb.abs().T
        # projection_refs.gemm_bound without its floor: the types' smallest steps instead
        least = 2.0 ** -149 * (P.pieces(K) + 2) + (2.0 ** -134 if t == BF else 0.0)
        bound = (127 * 2 * R.FP32 + (P.pieces(K) + 12) * R.FP32) * mag + R.half_step(t) * ref.abs() + least
        over = (out[rows].double() - ref).abs() - bound
        assert (over <= 0).all(), float(over.max())
    assert dsa.dsa_get_device_status() == 0
