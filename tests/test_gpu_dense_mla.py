"""dsa_mla_decode_paged on the GPU against dense attention in fp64.

Bounds.  Output: a weight rounded to bf16 (one half step of the sum of p |v|), the output's own half step, and
the scores' fp32 error through the softmax.  A score is a sum of 576 exact products in fp32: at most 576 steps
of 2^-23 of sum |q||k| scale, which is also what its error adds to the LSE and, relative, to a weight."""
import math

import pytest
import torch

from tests import operator_refs as R
from tests.gpu_util import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, I32 = torch.bfloat16, torch.int32
SCALE = 1.0 / 24.0


def problem(ctx, H, page, seed, std=1.0, spare=2):
    """Sequences of the given lengths over a shuffled pool whose unused slots hold NaN."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(c, 0) // page) for c in ctx]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=g).to(I32)
    bt = torch.full((len(ctx), max(max(need), 1)), -1, dtype=I32)
    pool = torch.full((total, page, 576), float("nan"), dtype=BF)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = perm[at:at + n]
        for j in range(n):
            used = min(page, ctx[b] - j * page)
            pool[int(perm[at + j]), :used] = (torch.randn((used, 576), generator=g) * std).to(BF)
        at += n
    q = torch.randn((len(ctx), H, 576), generator=g).to(BF)
    return q, pool, bt, torch.tensor(ctx, dtype=I32)


def call(q, pool, bt, ctx, scale=SCALE, **kw):
    dsa = lib()
    out = torch.full((q.shape[0], q.shape[1], 512), 7.0, dtype=BF, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    dsa.dsa_mla_decode_paged(q.to(DEV), pool.to(DEV), bt.to(DEV), ctx.to(DEV), scale, out, lse, **kw)
    return out, lse


def rows_of(pool, bt, b, n):
    page = pool.shape[1]
    s = torch.arange(n)
    return pool.view(-1, 576)[bt[b, s // page].long() * page + s % page]


def check(out, lse, q, pool, bt, ctx, scale=SCALE, rows=None):
    for b in rows if rows is not None else range(len(ctx)):
        n = max(int(ctx[b]), 0)
        o, l, pv, big = R.dense_mla(q[b], rows_of(pool, bt, b, n), scale)
        ds = 576 * 2.0 ** -23 * big
        if n == 0:
            assert (out[b] == 0).all() and (lse[b] == -math.inf).all(), f"row {b}: empty"
            continue
        R.check_close(out[b], o, (R.BF16 + 2 * ds + 1e-5) * pv + R.BF16 * o.abs() + 1e-30, f"row {b} (ctx {n}) out")
        R.check_close(lse[b], l, ds + 1e-5 + 4 * R.FP32 * l.abs(), f"row {b} (ctx {n}) lse")


@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("H", [1, 7, 16, 64, 65, 128])
def test_lengths_heads_pages(H, page):
    ctx = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 0, 255, 257, 1000, 4097, -5]
    p = problem(ctx, H, page, H + page)
    lib().dsa_get_device_status()
    out, lse = call(*p)
    check(out, lse, *p)
    assert lib().dsa_get_device_status() == 0
    out2, lse2 = call(*p)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("ctx", [[1], [20000], [3, 0, 0, 0], [0], [0] * 5, [130] * 300, list(range(200)), [9000, 1, 1, 9000, 64]])
def test_batches(ctx):
    """One row over every SM, empty rows first, last and alone, many rows, shares that cross several rows."""
    p = problem(ctx, 16, 64, len(ctx))
    out, lse = call(*p)
    check(out, lse, *p, rows=range(0, len(ctx), max(1, len(ctx) // 24)))


@pytest.mark.parametrize("std,scale", [(1.0, 1.0), (8.0, 1.0), (1e-3, 1e-4), (1.0, 1e3)])
def test_sharp_and_flat_softmax(std, scale):
    """Scores of hundreds, where one key has all of the weight, and of nothing, where all have the same.  A score's
    bound past 2^-7 says nothing about the weights any more: there the row must still be finite, with its LSE right."""
    p = problem([700, 65, 1], 16, 64, 4, std=std)
    out, lse = call(*p, scale=scale)
    assert torch.isfinite(out).all()
    for b in range(3):
        o, l, pv, big = R.dense_mla(p[0][b], rows_of(p[1], p[2], b, int(p[3][b])), scale)
        ds = 576 * 2.0 ** -23 * big
        R.check_close(lse[b], l, ds + 1e-5 + 4 * R.FP32 * l.abs(), "lse")
        if ds < 2.0 ** -7:
            R.check_close(out[b], o, (R.BF16 + 2 * ds + 1e-5) * pv + R.BF16 * o.abs() + 1e-30, "out")


def test_closed_forms():
    """Equal keys give their value and log n; zero queries the mean and log n."""
    q, pool, bt, ctx = problem([777, 300], 16, 64, 8)
    rows = rows_of(pool, bt, 0, 777)
    s = torch.arange(777)
    pool.view(-1, 576)[bt[0, s // 64].long() * 64 + s % 64] = rows[:1]
    q[1] = 0
    out, lse = call(q, pool, bt, ctx)
    same = rows[0, :512].double().expand(16, 512)
    R.check_close(out[0], same, 2 * R.BF16 * same.abs() + 1e-30, "equal keys")
    R.check_close(lse[1], torch.full((16,), math.log(300), dtype=torch.float64), 1e-5, "lse of zeros")
    check(out, lse, q, pool, bt, ctx, rows=[1])


def test_bad_pages_and_lengths():
    dsa = lib()
    q, pool, bt, ctx = problem([300, 300, 300], 16, 64, 5, spare=0)
    bt[0, 1], bt[1] = pool.shape[0], -1
    ctx[2] = 100000  # past the table: clamped to its 320 slots, of which the last 20 hold NaN
    pool[torch.isnan(pool)] = 0.5
    dsa.dsa_get_device_status()
    out, lse = call(q, pool, bt, ctx)
    assert dsa.dsa_get_device_status() == dsa.DSA_DEV_BAD_PAGE | dsa.DSA_DEV_BAD_POSITION
    left = torch.cat([torch.arange(64), torch.arange(128, 300)])
    kv = pool.view(-1, 576)[bt[0, left // 64].long() * 64 + left % 64]
    for b, rows in ((0, kv), (2, rows_of(pool, bt, 2, 320))):
        o, l, pv, big = R.dense_mla(q[b], rows, SCALE)
        ds = 576 * 2.0 ** -23 * big
        R.check_close(out[b], o, (R.BF16 + 2 * ds + 1e-5) * pv + R.BF16 * o.abs() + 1e-30, f"row {b}")
        R.check_close(lse[b], l, ds + 1e-5 + 4 * R.FP32 * l.abs(), "lse")
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()


def test_pool_past_32_bit_offsets():
    """Pages whose byte and element offsets pass 2^32 and 2^31."""
    pages = 2 ** 32 // (64 * 576 * 2) + 2 ** 31 // (64 * 576 * 2) + 9
    pool = torch.empty((pages, 64, 576), dtype=BF, device=DEV)
    q, small, bt, ctx = problem([1000, 130], 16, 64, 6, spare=0)
    far = torch.arange(small.shape[0]) * -1 + (pages - 1)
    pool[far.to(DEV)] = small.to(DEV)
    dsa = lib()
    out, lse = torch.empty((2, 16, 512), dtype=BF, device=DEV), torch.empty((2, 16), device=DEV)
    table = torch.where(bt >= 0, far[bt.clamp(min=0).long()].to(I32), bt)
    dsa.dsa_mla_decode_paged(q.to(DEV), pool, table.to(DEV), ctx.to(DEV), SCALE, out, lse)
    check(out, lse, q, small, bt, ctx)


def test_agrees_with_sparse_decode_over_every_position():
    """A selection that holds all positions is dense attention."""
    dsa = lib()
    q, pool, bt, ctx = problem([1000, 2048, 77], 128, 64, 12)
    out, lse = call(q, pool, bt, ctx)
    idx = torch.arange(2048, dtype=I32).expand(3, 2048).contiguous()
    idx = torch.where(idx < ctx[:, None], idx, torch.full_like(idx, -1)).to(DEV)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    dsa.dsa_sparse_mla_decode_paged(q.to(DEV), pool.to(DEV), bt.to(DEV), ctx.to(DEV), idx, SCALE, o2, l2)
    check(out, lse, q, pool, bt, ctx)
    check(o2, l2, q, pool, bt, ctx)


def test_streams_workspaces_and_graphs():
    dsa = lib()
    probs = [problem([5000, 100, 64], 128, 64, 40), problem([900, 3000], 16, 32, 41)]
    want = [call(*p) for p in probs]
    need = [dsa.dsa_mla_decode_workspace_size(len(p[3]), p[0].shape[1]) for p in probs]
    ins = [[t.to(DEV) for t in p] for p in probs]
    outs = [(torch.zeros_like(o), torch.zeros_like(l)) for o, l in want]
    wss = [torch.full((max(n, 1) + 256,), 0xFF, dtype=torch.uint8, device=DEV) for n in need]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for given in (False, True):  # side by side, the allocator's workspaces and then the caller's
        for i, s in enumerate(streams):
            dsa.dsa_mla_decode_paged(*ins[i], SCALE, *outs[i], workspace=wss[i][:need[i]] if given else None, stream=s)
        torch.cuda.synchronize()
        for (o, l), (ro, rl) in zip(outs, want):
            assert torch.equal(o, ro) and torch.equal(l, rl)
            o.zero_(), l.zero_()
    for w, n in zip(wss, need):
        assert (w[n:] == 0xFF).all()  # nothing past the stated size
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # two captured calls, workspaces of their own, in one order
        for i in range(2):
            dsa.dsa_mla_decode_paged(*ins[i], SCALE, *outs[i], workspace=wss[i])
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for (o, l), (ro, rl) in zip(outs, want):
            assert torch.equal(o, ro) and torch.equal(l, rl)
            o.zero_(), l.zero_()
    ins[0][3].copy_(torch.tensor([17, 100, 0], dtype=I32))  # lengths are read at replay
    graph.replay()
    p = probs[0][:3] + (torch.tensor([17, 100, 0], dtype=I32),)
    check(*outs[0], *p)


def test_nan_reaches_its_rows_and_heads_only():
    """A NaN key of a whole row, of a row in parts, and a NaN query head."""
    q, pool, bt, ctx = problem([300, 20000, 64, 500], 16, 64, 50)
    pool.view(-1, 576)[int(bt[0, 0]) * 64 + 5, 570] = float("nan")
    pool.view(-1, 576)[int(bt[1, 100]) * 64 + 63, 3] = float("nan")
    q[3, 7, 100] = float("nan")
    out, lse = call(q, pool, bt, ctx)
    assert torch.isnan(out[:2]).all() and torch.isnan(lse[:2]).all()
    assert torch.isnan(out[3, 7]).all() and torch.isnan(lse[3, 7])
    keep = [h for h in range(16) if h != 7]
    check(out, lse, q, pool, bt, ctx, rows=[2])
    check(out[:, keep], lse[:, keep], q[:, keep], pool, bt, ctx, rows=[3])


def test_batches_in_turn_share_a_workspace():
    """Calls of other sizes on one stream, nothing between them, over one workspace: each as if alone."""
    dsa = lib()
    probs = [problem(c, h, 64, 60 + i) for i, (c, h) in enumerate(
        [([6000, 1, 700], 128), ([0, 0], 128), ([40], 3), ([100] * 90, 16), ([9000], 64)])]
    want = [call(*p) for p in probs]
    ins = [[t.to(DEV) for t in p] for p in probs]
    ws = torch.full((max(dsa.dsa_mla_decode_workspace_size(len(p[3]), p[0].shape[1]) for p in probs),), 0xFF, dtype=torch.uint8,
                    device=DEV)
    outs = [[(torch.empty_like(o), torch.empty_like(l)) for _ in range(6)] for o, l in want]
    torch.cuda.synchronize()
    for k in range(6):
        for i, p in enumerate(ins):
            dsa.dsa_mla_decode_paged(*p, SCALE, *outs[i][k], workspace=ws)
    for (o, l), got in zip(want, outs):
        for go, gl in got:
            assert torch.equal(go, o) and torch.equal(gl, l)


@pytest.mark.parametrize("B", [74, 75, 76, 77, 150, 400])
@pytest.mark.parametrize("H", [3, 100])
def test_as_many_rows_as_clusters(B, H):
    """Around the number of CTA pairs, where parts of rows are recorded by row or by pair: rows of one tile, of many and
    none, over a workspace that holds anything."""
    g = torch.Generator().manual_seed(B)
    ctx = torch.randint(0, 140, (B,), generator=g)
    ctx[torch.randint(0, B, (5,), generator=g)] = torch.tensor([3000, 1500, 129, 128, 700])
    p = problem(ctx.tolist(), H, 64, B + H)
    need = lib().dsa_mla_decode_workspace_size(B, H)
    ws = torch.randint(0, 256, (need,), generator=torch.Generator(device=DEV).manual_seed(B), dtype=torch.uint8, device=DEV)
    out, lse = call(*p, workspace=ws)
    check(out, lse, *p)


@pytest.mark.parametrize("ctx", [[300, 0, 9000, 64], [20000]])
def test_tensors_that_start_at_16_bytes(ctx):
    """q, the pool and out no multiple of 32 bytes: the same bits, and nothing beside out."""
    q, pool, bt, lens = problem(ctx, 100, 64, 70)
    want = call(q, pool, bt, lens)

    def shifted(t, fill=0.0):
        buf = torch.full((t.numel() + 16,), fill, dtype=t.dtype, device=DEV)
        view = buf[8:8 + t.numel()].view(t.shape)
        assert view.data_ptr() % 32 == 16
        view.copy_(t)
        return view, buf

    out, buf = shifted(torch.empty((len(ctx), 100, 512), dtype=BF), 5.0)
    lse = torch.empty((len(ctx), 100), device=DEV)
    buf[:8] = 5.0
    buf[-8:] = 5.0
    lib().dsa_mla_decode_paged(shifted(q)[0], shifted(pool)[0], bt.to(DEV), lens.to(DEV), SCALE, out, lse)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert (buf[:8] == 5.0).all() and (buf[-8:] == 5.0).all()
