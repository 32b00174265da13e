"""Dense paged MLA call after call: the two CTAs of a pair hand tiles to one another, and what one of them must not
touch yet would show as a wrong row in one call of many."""
import pytest
import torch

from tests.gpu_util import lib
from tests.test_gpu_dense_mla import BF, DEV, SCALE, check, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,page,ctx,times", [
    (128, 32, [(i * 97) % 701 for i in range(300)], 300),
    (128, 64, [(i * 61) % 517 + 1 for i in range(300)], 300),
    (100, 128, [128] * 200, 300),
    (128, 64, [(i * 1237) % 9001 for i in range(40)], 200),
    (65, 32, [20000, 1, 130], 200),
    (16, 64, [1000], 300),
])
def test_the_same_bits_every_time(H, page, ctx, times):
    """Hundreds of calls without a wait between them; the first against 64 bits."""
    dsa = lib()
    p = problem(ctx, H, page, H + len(ctx))
    q, pool, bt, c = (t.to(DEV) for t in p)
    want, want_lse = torch.empty((len(ctx), H, 512), dtype=BF, device=DEV), torch.empty((len(ctx), H), device=DEV)
    out, lse, differ = torch.empty_like(want), torch.empty_like(want_lse), torch.zeros((), dtype=torch.int64, device=DEV)
    dsa.dsa_mla_decode_paged(q, pool, bt, c, SCALE, want, want_lse)
    for _ in range(times):
        dsa.dsa_mla_decode_paged(q, pool, bt, c, SCALE, out, lse)
        differ += (out.view(torch.int16) != want.view(torch.int16)).sum() + (lse != want_lse).sum()
    assert differ.item() == 0
    check(want, want_lse, *p, rows=range(0, len(ctx), max(1, len(ctx) // 24)))
    assert dsa.dsa_get_device_status() == 0
