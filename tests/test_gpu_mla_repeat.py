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
