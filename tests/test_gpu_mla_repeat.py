"""Paged sparse MLA gives the bits of the contiguous call, every time: many short rows on persistent clusters, where a
block's partial scores must not land over the ones that are still being read."""
import dataclasses

import pytest
import torch

from tests.test_gpu_varlen import DEV, W, lib, run_paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,k,times", [([300, 1000, 77, 513, 64, 1250], 256, 100), ([130] * 9, 128, 60), ([75], 128, 60)])
def test_paged_equals_contiguous_every_time(lens, k, times):
    dsa = lib()
    cfg = dataclasses.replace(W.CONFIGS["decode_paged"], seed=7)
    v = W.varlen_inputs(cfg, DEV, lens)
    _, idx, out, lse = run_paged(dsa, v, k, cfg.sm_scale)
    if dsa.dsa_sparse_mla_decode_workspace_size(lse.shape[0], lse.shape[1], k):
        pytest.skip("rows are split: joined parts round otherwise")
    starts = v["seq_starts"][v["seq"]].to(DEV).to(torch.int32)[:, None]
    want, want_lse = torch.empty_like(out), torch.empty_like(lse)
    dsa.dsa_sparse_mla_prefill(v["q"], v["kv_concat"], torch.where(idx >= 0, idx + starts, idx), cfg.sm_scale, want, want_lse)
    for _ in range(times):
        out.zero_()
        dsa.dsa_sparse_mla_decode_paged(v["q"], v["kv_pool"], v["block_table"], v["ctx"], idx, cfg.sm_scale, out, lse)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("T,S,k,few,times", [(4096, 3000, 128, 0.5, 60), (1999, 700, 64, 0.9, 100), (64, 4096, 2048, 0.0, 100),
                                             (20, 5000, 512, 0.3, 100)])
def test_prefill_and_decode_give_the_same_bits_every_time(T, S, k, few, times):
    """Rows of no, few and all k entries: prefill, and the same rows over pages, call after call, without a wait between
    them.  ``few`` of the rows have at most two blocks."""
    dsa, page = lib(), 64
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    q = torch.randn((T, 128, 576), generator=g, device=DEV, dtype=torch.bfloat16)
    pages = -(-S // page)
    kv = torch.randn((pages * page, 576), generator=g, device=DEV, dtype=torch.bfloat16)
    order = torch.rand((T, S), generator=g, device=DEV).argsort(1)[:, :k].sort(1).values.to(torch.int32)
    n = torch.randint(0, k + 1, (T, 1), generator=g, device=DEV)
    n = torch.where(torch.rand((T, 1), generator=g, device=DEV) < few, n % min(k + 1, 129), n)
    n[0], n[-1] = 0, k
    idx = torch.where(torch.arange(k, device=DEV) < n, order, -1)
    table = torch.arange(pages, device=DEV, dtype=torch.int32).expand(T, pages).contiguous()
    ctx = torch.full((T,), S, device=DEV, dtype=torch.int32)
    calls = [lambda o, l: dsa.dsa_sparse_mla_prefill(q, kv[:S], idx, 0.04, o, l),
             lambda o, l: dsa.dsa_sparse_mla_decode_paged(q, kv.view(pages, page, 576), table, ctx, idx, 0.04, o, l)]
    for call in calls:
        want, want_lse = torch.empty((T, 128, 512), device=DEV, dtype=torch.bfloat16), torch.empty((T, 128), device=DEV)
        out, lse, differ = torch.empty_like(want), torch.empty_like(want_lse), torch.zeros((), device=DEV, dtype=torch.int64)
        call(want, want_lse)
        for _ in range(times):
            call(out, lse)
            differ += (out.view(torch.int16) != want.view(torch.int16)).sum() + (lse != want_lse).sum()
        assert differ.item() == 0 and dsa.dsa_get_device_status() == 0
        # Rows of the first call, spread over the batch, against 64 bits.  A weight is off by half a step of bf16 (2^-8) and
        # what its score is: sums of 576 products, |z| terms adding up to 15 or so, by 40 half steps of fp32 at the most
        # (4e-5); out is rounded once more (2^-8).  The sixteenth on top takes the scores and the products of these.
        for t in range(0, T, max(1, T // 40)):
            sel = idx[t, : int(n[t])].long()
            if not len(sel):
                assert not want[t].any() and torch.isneginf(want_lse[t]).all()
                continue
            z = q[t].double() @ kv[sel].double().T * 0.04
            ref = torch.softmax(z, -1) @ kv[sel, :512].double()
            mean = torch.softmax(z, -1) @ kv[sel, :512].double().abs()
            assert ((want[t].double() - ref).abs() <= 2**-8 * (1 + 2**-4) * (mean + ref.abs())).all()
            assert ((want_lse[t].double() - torch.logsumexp(z, -1)).abs() <= 1e-4).all()
