"""The norm, projections, rotations, cache writes and both attentions run together as a layer of a served model and as
the indexer's warm-up step, against the same chain in fp64.

The projections are PyTorch products, taken as given: the fp64 chain starts again from each one's output, so every
operator is held to its own rounding.  Attention bounds as in the dense attention's tests, with the cache's and
queries' bf16 rows as the inputs."""
import math

import pytest
import torch

from tests import operator_refs as R
from tests.gpu_util import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
D, H, HI, PAGE, EPS, SCALE = 512, 16, 32, 64, 1e-6, 1 / 24.0


class Layer:
    """Weights, caches and block tables of one layer."""

    def __init__(self, lens, steps, g):
        def w(*shape):
            return (torch.randn(shape, generator=g, device=DEV) / math.sqrt(shape[0])).to(BF)

        self.norm, self.kv_norm = (1 + 0.1 * torch.randn(n, generator=g, device=DEV).to(BF) for n in (D, 512))
        self.wkv, self.wkI, self.wq, self.wqr, self.wqI, self.ww = w(D, 576), w(D, 128), w(D, H * 512), w(D, H * 64), w(D, HI * 128), w(D, HI)
        pages = [-(-(n + steps) // PAGE) for n in lens]
        perm = torch.randperm(sum(pages), generator=torch.Generator().manual_seed(2)).to(I32)
        self.table = torch.full((len(lens), max(pages)), -1, dtype=I32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.kv = torch.full((at, PAGE, 576), float("nan"), dtype=BF, device=DEV)
        self.k8 = torch.full((at, PAGE, 128), 0x7F, dtype=U8, device=DEV)
        self.ks = torch.full((at, PAGE), float("nan"), device=DEV)
        self.dev_table, self.freq = self.table.to(DEV), R.inv_freq().to(DEV)

    def project(self, dsa, x, res, pos, seq):
        """Norm, projections, cache append and queries of T tokens."""
        T = x.shape[0]
        h, y = torch.empty_like(x), torch.empty_like(x)
        dsa.dsa_rmsnorm(x, self.norm, EPS, out=y, residual=res, residual_out=h)
        kvkI = torch.cat([y @ self.wkv, y @ self.wkI], 1)  # one fused projection: kv and kI are slices of it
        dsa.dsa_cache_append(pos, self.dev_table, self.freq, kv=kvkI[:, :576], kv_pool=self.kv, kI=kvkI[:, 576:], k8_pool=self.k8,
                             ks_pool=self.ks, seq=seq, kv_weight=self.kv_norm, eps=EPS)
        q = torch.empty((T, H, 576), dtype=BF, device=DEV)
        q[..., :512] = (y @ self.wq).view(T, H, 512)
        qr, qI = (y @ self.wqr).view(T, H, 64), (y @ self.wqI).view(T, HI, 128)
        q8, qs = torch.empty((T, HI, 128), dtype=U8, device=DEV), torch.empty(T, device=DEV)
        dsa.dsa_rope_queries(pos, self.freq, q_rope=qr, q=q, qI=qI, q8=q8, q_scale=qs)
        return dict(h=h, y=y, kv=kvkI[:, :576], kI=kvkI[:, 576:], q=q, qr=qr, qI=qI, q8=q8, qs=qs, w=(y @ self.ww).float())

    def rows(self, pool, b, n):
        s = torch.arange(n)
        return pool.view(-1, pool.shape[-1])[(self.table[b, s // PAGE].long() * PAGE + s % PAGE).to(DEV)]


def check_projected(layer, p, x, res, pos):
    rh, ry = R.rmsnorm(x, res, layer.norm, EPS)
    R.check_close(p["h"], rh, rh.abs() * (R.BF16 + R.FP32) + 1e-30, "h")
    R.check_close(p["y"], ry, ry.abs() * (R.BF16 + 24 * R.FP32) + 1e-30, "y")
    rot = R.rotate_main(R.d(p["qr"]), pos.cpu(), R.inv_freq())
    R.check_close(p["q"][..., 512:], rot, rot.abs() * R.BF16 + 2.0 ** -18, "q rotated")


@pytest.mark.parametrize("lens", [[70, 1, 129, 64], [300]])
def test_prefill_then_decode_steps(lens):
    """Prompts of several lengths, then three tokens each: the caches hold what fp64 says, dense decode is attention
    over them, and selecting every position gives the same; slots behind the sequences stay untouched."""
    dsa, steps = lib(), 3
    g = torch.Generator(device=DEV)
    g.manual_seed(len(lens))
    layer = Layer(lens, steps, g)
    dsa.dsa_get_device_status()
    pos = torch.cat([torch.arange(n) for n in lens]).to(I32).to(DEV)
    seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).to(I32).to(DEV)
    x, res = (torch.randn((len(pos), D), generator=g, device=DEV).to(BF) for _ in range(2))
    p = layer.project(dsa, x, res, pos, seq)
    check_projected(layer, p, x, res, pos)
    kept = {b: (p["kv"][seq == b], p["kI"][seq == b]) for b in range(len(lens))}
    for b, n in enumerate(lens):
        kv, kI = (R.d(t) for t in kept[b])
        lat = R.rmsnorm(kv[:, :512], None, layer.kv_norm, EPS)[1]
        want = torch.cat([lat, R.rotate_main(kv[:, 512:], torch.arange(n), R.inv_freq())], 1)
        got = layer.rows(layer.kv, b, n)
        R.check_close(got, want, want.abs() * (R.BF16 + 24 * R.FP32) + kv.abs().max() * 2.0 ** -19, f"cache {b}")
        R.check_fp8(layer.rows(layer.k8, b, n), layer.rows(layer.ks.unsqueeze(-1), b, n)[:, 0],
                    R.rotate_index(kI, torch.arange(n), R.inv_freq()), 2.0 ** -19, 0, f"index cache {b}")
        tail = layer.kv[layer.table[b, -1 if len(lens) == 1 else (n - 1) // PAGE], n % PAGE or PAGE:]
        assert torch.isnan(tail).all()
    B = len(lens)
    for step in range(steps):
        ctx = torch.tensor([n + step + 1 for n in lens], dtype=I32, device=DEV)
        x, res = (torch.randn((B, D), generator=g, device=DEV).to(BF) for _ in range(2))
        p = layer.project(dsa, x, res, ctx - 1, None)
        check_projected(layer, p, x, res, ctx - 1)
        out, lse = torch.empty((B, H, 512), dtype=BF, device=DEV), torch.empty((B, H), device=DEV)
        dsa.dsa_mla_decode_paged(p["q"], layer.kv, layer.dev_table, ctx, SCALE, out, lse)
        # the sparse path: index scores of the cached keys, all of them selected
        ld = int(ctx.max())
        logits, idx = torch.full((B, ld), float("nan"), device=DEV), torch.empty((B, 512), dtype=I32, device=DEV)
        dsa.dsa_indexer_logits(p["q8"], p["qs"], p["w"], layer.k8, layer.ks, ctx - 1, logits, block_table=layer.dev_table)
        dsa.dsa_topk(logits, ctx, 512, idx)
        out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
        dsa.dsa_sparse_mla_decode_paged(p["q"], layer.kv, layer.dev_table, ctx, idx, SCALE, out2, lse2)
        codes = R.e4m3_values()
        for b in range(B):
            n = int(ctx[b])
            o, l, pv, big = R.dense_mla(p["q"][b], layer.rows(layer.kv, b, n), SCALE)
            ds = 576 * 2.0 ** -23 * big
            for got, gl, what in ((out, lse, "dense"), (out2, lse2, "sparse")):
                R.check_close(got[b], o, (R.BF16 + 2 * ds + 1e-5) * pv + R.BF16 * o.abs() + 1e-30, f"{what} {b}")
                R.check_close(gl[b], l, ds + 1e-5 + 4 * R.FP32 * l.abs(), f"{what} lse {b}")
            k = codes[layer.rows(layer.k8, b, n).long().cpu()] * R.d(layer.rows(layer.ks.unsqueeze(-1), b, n))
            q = codes[p["q8"][b].long().cpu()] * float(p["qs"][b])
            ref = (torch.relu(q @ k.T) * R.d(p["w"][b])[:, None]).sum(0)
            assert (R.d(logits[b, :n]) - ref).abs().max() <= 1e-3 * ref.abs().max()  # the indexer's stated tolerance
    assert dsa.dsa_get_device_status() == 0


def test_scores_depend_on_distance_alone():
    """Moving a whole sequence by any distance leaves dense attention as it was, up to the rotated parts' rounding:
    the rotation of queries and keys cancels but for their distance."""
    dsa, g = lib(), torch.Generator(device=DEV)
    g.manual_seed(4)
    n = 200
    kv, q = torch.randn((n, 576), generator=g, device=DEV).to(BF), torch.randn((1, H, 576), generator=g, device=DEV).to(BF)
    freq, got = R.inv_freq().to(DEV), []
    for start in (0, 64 * 1000):
        table = torch.full((1, start // PAGE + 4), -1, dtype=I32, device=DEV)
        table[0, start // PAGE:] = torch.arange(4, dtype=I32, device=DEV)
        pool = torch.zeros((4, PAGE, 576), dtype=BF, device=DEV)
        pos = torch.arange(start, start + n, dtype=I32, device=DEV)
        dsa.dsa_cache_append(pos, table, freq, kv=kv, kv_pool=pool, seq=torch.zeros(n, dtype=I32, device=DEV))
        qq = q.clone()
        dsa.dsa_rope_queries(pos[-1:], freq, q_rope=qq[..., 512:], q=qq)
        out, lse = torch.empty((1, H, 512), dtype=BF, device=DEV), torch.empty((1, H), device=DEV)
        dsa.dsa_mla_decode_paged(qq, pool, torch.arange(4, dtype=I32, device=DEV).view(1, 4), torch.tensor([n], dtype=I32, device=DEV),
                                 SCALE, out, lse)
        got.append((R.d(out), R.d(lse)))
    # a score's rotated part: 64 products of two bf16-rounded factors, each side off by 2^-8 of its size
    slack = 2 * 2 * R.BF16 * float((R.d(q[..., 512:]).norm(dim=-1).max() * R.d(kv[:, 512:]).norm(dim=-1).max())) * SCALE
    assert (got[0][1] - got[1][1]).abs().max() <= slack + 1e-4
    assert (got[0][0] - got[1][0]).abs().max() <= 2 * slack * float(R.d(kv[:, :512]).abs().max())


def test_warmup_gradients_through_the_rotation_and_norm():
    """One warm-up step of the indexer over a norm's output: dq and dk of dsa_indexer_warmup turned back, through the
    projections (plain products) and the norm's backward, against fp64 from the same dq and dk."""
    dsa, g = lib(), torch.Generator(device=DEV)
    g.manual_seed(6)
    T = 96
    layer = Layer([T], 1, g)
    x = torch.randn((T, D), generator=g, device=DEV).to(BF)
    pos = torch.arange(T, dtype=I32, device=DEV)
    p = layer.project(dsa, x, torch.zeros_like(x), pos, torch.zeros(T, dtype=I32, device=DEV))
    kv, k8 = layer.rows(layer.kv, 0, T).contiguous(), layer.rows(layer.k8, 0, T).contiguous()
    ks = layer.rows(layer.ks.unsqueeze(-1), 0, T)[:, 0].contiguous()
    loss, dw = torch.empty(T, device=DEV), torch.empty((T, HI), device=DEV)
    dq, dk = torch.empty((T, HI, 128), device=DEV), torch.empty((T, 128), device=DEV)
    dsa.dsa_indexer_warmup(p["q"], kv, SCALE, p["q8"], p["qs"], p["w"], k8, ks, pos, loss, dw, dq, dk)
    assert torch.isfinite(loss).all() and float(dq.abs().max()) > 0 and float(dk.abs().max()) > 0
    dqI, dkI = torch.empty_like(dq), torch.empty_like(dk)
    dsa.dsa_index_rope_backward(dq, pos, layer.freq, dqI)
    dsa.dsa_index_rope_backward(dk, pos, layer.freq, dkI)
    for got, src in ((dqI, dq), (dkI, dk)):
        ref = R.rotate_index(R.d(src), -pos.cpu().long(), R.inv_freq())
        R.check_close(got, ref, 2.0 ** -20 * 2 * R.d(src).abs().max() + ref.abs() * R.FP32, "turned back")
    dy = dqI.view(T, -1) @ layer.wqI.float().T + dkI @ layer.wkI.float().T + dw @ layer.ww.float().T
    dx, dwn = torch.empty((T, D), device=DEV), torch.empty(D, device=DEV)
    dsa.dsa_rmsnorm_backward(dy, p["h"].float(), layer.norm, EPS, dx, dwn)
    rx, rw, mag, wmag = R.rmsnorm_backward(dy, p["h"].float(), layer.norm, None, EPS)
    R.check_close(dx, rx, rx.abs() * R.FP32 + 48 * R.FP32 * mag + 1e-30, "dx")
    R.check_close(dwn, rw, 160 * R.FP32 * wmag + 1e-30, "dweight")


def test_decode_step_captured_and_replayed():
    """A decode step of all operators in one graph: a replay with new tokens, positions and lengths gives what the
    calls give, and padded rows of the batch (pos -1, ctx 0) leave caches alone and get zeros."""
    dsa, g = lib(), torch.Generator(device=DEV)
    g.manual_seed(8)
    lens = [70, 10, 200, 64]
    layer = Layer(lens, 4, g)
    B = len(lens)
    pos = torch.cat([torch.arange(n) for n in lens]).to(I32).to(DEV)
    seq = torch.repeat_interleave(torch.arange(B), torch.tensor(lens)).to(I32).to(DEV)
    layer.project(dsa, torch.randn((len(pos), D), generator=g, device=DEV).to(BF), torch.zeros((len(pos), D), dtype=BF, device=DEV), pos, seq)
    x, res = torch.zeros((B, D), dtype=BF, device=DEV), torch.zeros((B, D), dtype=BF, device=DEV)
    at, ctx = torch.zeros(B, dtype=I32, device=DEV), torch.zeros(B, dtype=I32, device=DEV)
    out, lse = torch.empty((B, H, 512), dtype=BF, device=DEV), torch.empty((B, H), device=DEV)

    def step():
        p = layer.project(dsa, x, res, at, None)
        dsa.dsa_mla_decode_paged(p["q"], layer.kv, layer.dev_table, ctx, SCALE, out, lse)

    at.copy_(torch.tensor([n - 1 for n in lens]))
    ctx.copy_(torch.tensor(lens))
    before = [t.clone() for t in (layer.kv, layer.k8, layer.ks)]
    step()
    for t, b in zip((layer.kv, layer.k8, layer.ks), before):
        t.copy_(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        x.copy_(torch.randn((B, D), generator=g, device=DEV))
        new = [n + k for n in lens]
        new[k % B] = -1
        at.copy_(torch.tensor(new))
        ctx.copy_(torch.tensor([n + 1 for n in new]))
        graph.replay()
        torch.cuda.synchronize()
        o, l, state = out.clone(), lse.clone(), [t.clone() for t in (layer.kv, layer.k8, layer.ks)]
        assert (o[k % B] == 0).all() and (l[k % B] == -math.inf).all()
        step()
        # a row whose token an earlier step left out attends to a slot that still holds NaN: NaN on both sides
        for a, b in zip([o, l] + state, (out, lse, layer.kv, layer.k8, layer.ks)):
            assert torch.equal(torch.nan_to_num(a.float(), nan=-7.0), torch.nan_to_num(b.float(), nan=-7.0))
        for b, n in enumerate(new):
            assert torch.isfinite(out[b]).all() == (n < 0 or n == lens[b] or b >= k)
    assert dsa.dsa_get_device_status() == 0
