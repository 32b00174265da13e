"""Dense paged MLA where the running maximum moves: the accumulated output is then scaled down in tensor memory, and every
tile's part of the output has to come through it.

A head's scores come from one of the 64 rotated columns, so that they are single exact products.  They climb from tile to
tile by more than the 2^8 that the kernel lets pass, in other tiles for other heads, and the values fall as the scores
climb: tiles of one head weigh alike in the output, and a part that was scaled by the wrong factor, or not, shows.

Bounds, relative to sum p |v|: half a step of bf16 for the weights and for the output; per score a few half steps of fp32 at
the largest score (its product with the scale, the maximum's, their difference), the same at every move of the maximum, and
2^-22 for each approximate exponential: ds.  fp32 sums of some thousand terms: 2^-13.
"""
import math

import pytest
import torch

from tests import operator_refs as R
from tests.gpu_util import lib
from tests.test_gpu_dense_mla import BF, DEV, call, problem, rows_of

pytestmark = pytest.mark.gpu
TILE = 128


def climbing(ctx, H, page, step, every, fall):
    """Head h looks at rotated column h % 64; column g climbs by `step` (log2 of the weight) at the tiles j with
    (j + g) % every == 0.  Values of tile j are of size 2^(-fall j)."""
    q, pool, bt, c = problem(ctx, H, page, 7 * H + len(ctx), std=0.0)
    g = torch.Generator().manual_seed(H)
    most = max(ctx)
    tile = torch.arange(most) // TILE
    level = torch.stack([torch.tensor([sum((i + col) % every == 0 for i in range(1, int(j) + 1)) for j in range(int(tile[-1]) + 1)])
                         for col in range(64)])[:, tile].T.double()  # [most, 64]
    score = (level * step + torch.rand((most, 64), generator=g).double()) * math.log(2.0)
    q.zero_()
    for h in range(H):
        q[:, h, 512 + h % 64] = 1.0
    flat = pool.view(-1, 576)
    for b, n in enumerate(ctx):
        s = torch.arange(n)
        row = bt[b, s // page].long() * page + s % page
        flat[row, 512:] = score[:n].to(BF)
        flat[row, :512] = (torch.randn((n, 512), generator=g) * 2.0 ** (-fall * tile[:n, None].float())).to(BF)
    return q, pool, bt, c


def wrong_rescale(q, kv, skip):
    """What comes of leaving the accumulated output of the columns `skip` as it is at the last move (fp64)."""
    s = q.double() @ kv.double().T
    tiles = -(-kv.shape[0] // TILE)
    m, acc, l, moves = torch.full((q.shape[0], 1), -math.inf, dtype=torch.float64), 0.0, 0.0, []
    for j in range(tiles):
        z = s[:, j * TILE:(j + 1) * TILE]
        top = z.amax(-1, keepdim=True)
        move = top * math.log2(math.e) > m * math.log2(math.e) + 8
        new = torch.where(move, top, m)
        f = torch.exp(m - new)
        f = torch.where(torch.isfinite(m), f, torch.zeros_like(f))
        fs = f.expand(-1, 512).clone()
        if j == tiles - 1:
            fs[:, skip] = 1.0
        p = torch.exp(z - new)
        acc = acc * fs + p @ kv[j * TILE:(j + 1) * TILE, :512].double()
        l = l * f + p.sum(-1, keepdim=True)
        m = new
        moves.append(move)
    return acc / l, torch.cat(moves, 1).sum(1)


@pytest.mark.parametrize("H,page,ctx,step,every,fall", [
    (128, 64, [700] * 100, 9.0, 1, 9.0),       # rows that one pair keeps whole, moves in every tile
    (128, 32, [897, 300, 640, 129] * 25, 10.0, 2, 5.0),
    (100, 64, [1000 + 31 * i for i in range(90)], 12.0, 3, 4.0),
    (65, 128, [1152] * 80, 30.0, 3, 8.0),      # most of the old weight goes at once
    (128, 64, [3000] * 6, 3.5, 1, 3.0),        # rows in parts of several tiles; moves in every third
    (16, 32, [2500] * 9, 9.0, 2, 4.0),
    (7, 64, [5000], 2.0, 1, 2.0),              # one row over every pair: the join does what the move does elsewhere
])
def test_the_maximum_climbs(H, page, ctx, step, every, fall):
    p = climbing(ctx, H, page, step, every, fall)
    out, lse = call(*p, scale=1.0)
    q, pool, bt, _ = p
    for b in range(0, len(ctx), max(1, len(ctx) // 6)):
        kv = rows_of(pool, bt, b, ctx[b])
        o, l, pv, big = R.dense_mla(q[b], kv, 1.0)
        tiles = -(-ctx[b] // TILE)
        ds = (8 + tiles) * R.FP32 * big * math.log2(math.e) + tiles * 2.0 ** -22
        bound = (R.BF16 + 2 * ds + 2.0 ** -13) * pv + R.BF16 * o.abs() + 1e-30
        R.check_close(out[b], o, bound, f"row {b} out")
        R.check_close(lse[b], l, 2 * ds + 1e-5 + 4 * R.FP32 * l.abs(), f"row {b} lse")
        if len(ctx) > 76 and every == 1:  # the bound sees a move that leaves some columns out
            wrong, moves = wrong_rescale(q[b], kv, slice(96, 128))
            assert (moves >= tiles - 1).all() and ((wrong - o).abs() > bound)[:, 96:128].float().mean() > 0.9
    assert lib().dsa_get_device_status() == 0


def test_the_maximum_climbs_in_some_heads_and_falls_in_others():
    """Heads of one warp that move beside heads that do not, and scores that fall."""
    H, ctx = 128, [1100] * 90
    q, pool, bt, c = climbing(ctx, H, 64, 9.0, 2, 2.0)
    q[:, 1::3] *= -1
    q[:, 2::3] *= 0.25
    out, lse = call(q, pool, bt, c, scale=1.0)
    for b in (0, 41, 89):
        o, l, pv, big = R.dense_mla(q[b], rows_of(pool, bt, b, ctx[b]), 1.0)
        ds = 17 * R.FP32 * big * math.log2(math.e) + 9 * 2.0 ** -22
        R.check_close(out[b], o, (R.BF16 + 2 * ds + 2.0 ** -13) * pv + R.BF16 * o.abs() + 1e-30, f"row {b} out")
        R.check_close(lse[b], l, 2 * ds + 1e-5 + 4 * R.FP32 * l.abs(), f"row {b} lse")
