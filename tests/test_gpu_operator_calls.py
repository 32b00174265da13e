"""Calls of the norm, rotation, cache and dense-attention operators as programs mix them: from several threads, first
of all under capture, with broadcast and repeated inputs."""
import subprocess
import sys
import threading

import pytest
import torch

from tests import operator_refs as R
from tests.gpu_util import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def step(seed, stream=None):
    """A small step over all of the calls, as a function that enqueues it, and the tensors that it writes."""
    dsa = lib()
    g = torch.Generator().manual_seed(seed)
    T, H, HI, page = 5 + seed, 16, 32, 64
    x = torch.randn((T, 1024), generator=g).to(BF).to(DEV)
    w = torch.randn(1024, generator=g).to(BF).to(DEV)
    pos = torch.randint(0, 120, (T,), generator=g).to(I32).to(DEV)
    bt = torch.randperm(2 * T, generator=g).to(I32).view(T, 2).to(DEV)
    fr = R.inv_freq().to(DEV)
    kv, kI = torch.randn((T, 576), generator=g).to(BF).to(DEV), torch.randn((T, 128), generator=g).to(BF).to(DEV)
    qr, qI = torch.randn((T, H, 64), generator=g).to(BF).to(DEV), torch.randn((T, HI, 128), generator=g).to(BF).to(DEV)
    pool = torch.randn((2 * T, page, 576), generator=g).to(BF).to(DEV)
    res = dict(y=torch.zeros_like(x), dx=torch.zeros_like(x), dw=torch.zeros(1024, device=DEV), pool=pool,
               k8=torch.zeros((2 * T, page, 128), dtype=torch.uint8, device=DEV), ks=torch.zeros((2 * T, page), device=DEV),
               q=torch.randn((T, H, 576), generator=g).to(BF).to(DEV),
               q8=torch.zeros((T, HI, 128), dtype=torch.uint8, device=DEV), qs=torch.zeros(T, device=DEV),
               dI=torch.zeros((T, HI, 128), device=DEV), out=torch.zeros((T, H, 512), dtype=BF, device=DEV),
               lse=torch.zeros((T, H), device=DEV))
    gI = torch.randn((T, HI, 128), generator=g).to(DEV)

    def run():
        dsa.dsa_rmsnorm(x, w, 1e-6, out=res["y"], stream=stream)
        dsa.dsa_rmsnorm_backward(res["y"], x, w, 1e-6, res["dx"], res["dw"], stream=stream)
        dsa.dsa_cache_append(pos, bt, fr, kv, res["pool"], kI, res["k8"], res["ks"], stream=stream)
        dsa.dsa_rope_queries(pos, fr, qr, res["q"], qI, res["q8"], res["qs"], stream=stream)
        dsa.dsa_index_rope_backward(gI, pos, fr, res["dI"], stream=stream)
        dsa.dsa_mla_decode_paged(res["q"], res["pool"], bt, pos, 0.04, res["out"], res["lse"], stream=stream)

    return run, res


def same(a, b):
    return a.dtype == b.dtype and torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_threads_with_streams_of_their_own():
    want = []
    for i in range(4):
        run, res = step(i)
        run()
        torch.cuda.synchronize()
        want.append(res)
    streams = [torch.cuda.Stream() for _ in range(4)]
    steps = [step(i, s) for i, s in enumerate(streams)]
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(40):
                    steps[i][0]()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not errors
    for (_, res), ref in zip(steps, want):
        for k in res:
            assert same(res[k], ref[k]), k
    assert lib().dsa_get_device_status() == 0


def test_a_failed_call_in_one_thread_leaves_anothers_error_alone():
    dsa = lib()
    x, w = torch.zeros((2, 64), dtype=BF, device=DEV), torch.zeros(64, dtype=BF, device=DEV)
    seen = {}

    def work(name, **kw):
        for _ in range(50):
            try:
                dsa.dsa_rmsnorm(x, w, out=x, **kw)
            except Exception as e:  # noqa: BLE001
                seen.setdefault(name, set()).add(str(e))

    threads = [threading.Thread(target=work, args=("eps",), kwargs=dict(eps=-1.0)),
               threading.Thread(target=work, args=("block",), kwargs=dict(eps=1e-6, block=64))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert all("eps" in m for m in seen["eps"]) and all("block" in m for m in seen["block"])


FIRST = """
import torch
from tests.test_gpu_operator_calls import step, same
run, res = step(3, None)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run()
graph.replay()
torch.cuda.synchronize()
run2, ref = step(3, None)
run2()
torch.cuda.synchronize()
assert all(same(res[k], ref[k]) for k in res)
print("captured first")
"""


def test_first_calls_of_a_process_captured():
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_broadcast_queries_and_repeated_inputs():
    """One rotated query for all heads (a head stride of zero), one vector for all tokens; x as its own residual."""
    dsa = lib()
    g = torch.Generator().manual_seed(5)
    pos = torch.randint(0, 4000, (6,), generator=g).to(I32)
    fr = R.inv_freq()
    one = torch.randn((6, 1, 64), generator=g).to(BF)
    for src in (one.to(DEV).expand(6, 9, 64), one[:1].to(DEV).expand(6, 9, 64)):
        q = torch.zeros((6, 9, 576), dtype=BF, device=DEV)
        dsa.dsa_rope_queries(pos.to(DEV), fr.to(DEV), q_rope=src, q=q)
        ref = R.rotate_main(R.d(src), pos, fr)
        # the half turns' rounding (pi half steps of the angle), cosine and sine (2), products and sum (2); then bf16
        mag = R.d(src).abs().unflatten(-1, (32, 2)).sum(-1, keepdim=True).expand(6, 9, 32, 2).flatten(-2)
        R.check_close(q[:, :, 512:], ref, R.BF16 * ref.abs() + 8 * R.FP32 * mag, "rotated")
        assert (q[:, :, :512] == 0).all()
    x, w = torch.randn((7, 520), generator=g).to(BF), torch.randn(520, generator=g).to(BF)
    xd = x.to(DEV)
    out, h = torch.empty_like(xd), torch.empty_like(xd)
    dsa.dsa_rmsnorm(xd, w.to(DEV), 1e-6, out=out, residual=xd, residual_out=h)
    assert torch.equal(h, 2 * xd)
    _, ref = R.rmsnorm(x, x, w, 1e-6)
    # half steps: 20 of the sum of squares (8 in a chunk, shuffles, warps), halved by the root; 8 of what follows
    R.check_close(out, ref, (R.BF16 + 24 * R.FP32) * ref.abs(), "norm of 2x")


def test_appends_whose_tokens_share_pages_and_sequences():
    """Many tokens of one sequence in one call, padding among them, then the same ones again."""
    dsa = lib()
    g = torch.Generator().manual_seed(6)
    T = 200
    pos = torch.randperm(256, generator=g)[:T].to(I32)
    pos[::9] = -1
    seq = torch.ones(T, dtype=I32)
    bt = torch.tensor([[0, 1, 2, 3], [7, 5, 4, 6]], dtype=I32)
    kv = torch.randn((T, 576), generator=g).to(BF)
    pool = torch.full((8, 64, 576), 3.0, dtype=BF, device=DEV)
    for _ in range(2):
        dsa.dsa_cache_append(pos.to(DEV), bt.to(DEV), R.inv_freq().to(DEV), kv=kv.to(DEV), kv_pool=pool, seq=seq.to(DEV))
        flat = pool.view(-1, 576).cpu()
        used = torch.zeros(8 * 64, dtype=torch.bool)
        for t in range(T):
            p = int(pos[t])
            if p >= 0:
                slot = int(bt[1, p // 64]) * 64 + p % 64
                used[slot] = True
                assert torch.equal(flat[slot, :512], kv[t, :512])
        assert (flat[~used] == 3.0).all()


@pytest.mark.parametrize("T,HI", [(1, 1), (7, 33), (90, 1), (40, 64)])
def test_index_gradients_that_start_at_16_bytes(T, HI):
    """g and dx no multiple of 32 bytes, in place too, with padding between."""
    dsa = lib()
    g = torch.Generator().manual_seed(T)
    pos = torch.randint(0, 9000, (T,), generator=g).to(I32)
    pos[1::5] = -1
    v = torch.randn((T, HI, 128), generator=g)
    buf = torch.zeros(T * HI * 128 + 4, device=DEV)
    src = buf[4:].view(T, HI, 128)
    assert src.data_ptr() % 32 == 16
    src.copy_(v)
    freq = R.inv_freq()
    ref = torch.where((pos < 0)[:, None, None], 0.0, R.rotate_index(R.d(v), -pos.clamp(min=0), freq))
    pair = v.double()[..., :64].unflatten(-1, (2, 32)).abs().sum(-2)
    mag = torch.cat([pair, pair, torch.zeros_like(pair), torch.zeros_like(pair)], -1)
    dx = torch.empty((T, HI, 128), dtype=BF, device=DEV)
    dsa.dsa_index_rope_backward(src, pos.to(DEV), freq.to(DEV), dx)
    R.check_close(dx, ref, R.BF16 * ref.abs() + 8 * R.FP32 * mag, "bf16")
    dsa.dsa_index_rope_backward(src, pos.to(DEV), freq.to(DEV), src)
    R.check_close(src, ref, 8 * R.FP32 * mag, "fp32, in place")
    assert (buf[:4] == 0).all()


@pytest.mark.parametrize("T", [1, 152, 153, 1000])
def test_query_parts_alone_and_together(T):
    """Few tokens take a CTA for each part, many one for both: the results are those of the parts called alone."""
    dsa = lib()
    g = torch.Generator().manual_seed(T)
    pos = torch.randint(-50, 5000, (T,), generator=g).to(I32).to(DEV)
    fr = R.inv_freq().to(DEV)
    qr, qI = torch.randn((T, 70, 64), generator=g).to(BF).to(DEV), torch.randn((T, 40, 128), generator=g).to(DEV)

    def outs():
        return (torch.zeros((T, 70, 576), dtype=BF, device=DEV), torch.zeros((T, 40, 128), dtype=torch.uint8, device=DEV),
                torch.zeros(T, device=DEV))

    a, b = outs(), outs()
    dsa.dsa_rope_queries(pos, fr, qr, a[0], qI, a[1], a[2])
    dsa.dsa_rope_queries(pos, fr, qr, b[0])
    dsa.dsa_rope_queries(pos, fr, qI=qI, q8=b[1], q_scale=b[2])
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert (a[2][pos < 0] == 0).all() and (a[2][pos >= 0] > 0).all()


@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("rows,cols", [(5, 1000), (5, 1001), (3, 130), (5000, 520), (4900, 521), (700, 6000), (700, 6001)])
def test_norm_outputs_in_every_combination(rows, cols, with_residual):
    """Each subset of the outputs holds what the call with all of them gives; outputs that are not asked for are not
    needed."""
    dsa = lib()
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    x, res = (torch.randn((rows, cols), generator=g, device=DEV).to(BF) for _ in range(2))
    w = torch.randn(cols, generator=g, device=DEV)

    def outs():
        return dict(out=torch.zeros_like(x), residual_out=torch.zeros_like(x), codes=torch.zeros((rows, cols), dtype=torch.uint8, device=DEV))

    for block in (0, 128):
        shape = (rows,) if block == 0 else (rows, -(-cols // 128))
        given = dict(residual=res) if with_residual else {}
        full, fscale = outs(), torch.zeros(shape, device=DEV)
        dsa.dsa_rmsnorm(x, w, 1e-6, scale=fscale, block=block, **full, **given)
        if not with_residual:
            assert torch.equal(full["residual_out"], x)
        for k in range(1, 7):
            some = {n: t for i, (n, t) in enumerate(outs().items()) if k >> i & 1}
            scale = torch.zeros(shape, device=DEV) if "codes" in some else None
            dsa.dsa_rmsnorm(x, w, 1e-6, scale=scale, block=block, **some, **given)
            for n, t in some.items():
                assert torch.equal(t, full[n]), (n, k)
            assert scale is None or torch.equal(scale, fscale)


def test_tensors_without_memory_are_refused():
    """Meta, sparse and fake tensors: an error from the Python form, nothing launched, and the next call works."""
    from torch._subclasses.fake_tensor import FakeTensorMode

    dsa = lib()
    x, w = torch.ones((4, 64), dtype=BF, device=DEV), torch.ones(64, dtype=BF, device=DEV)
    with FakeTensorMode(allow_non_fake_inputs=True):
        fake = torch.empty((4, 64), dtype=BF, device=DEV)
    for bad in (torch.empty((4, 64), dtype=BF, device="meta"), x.to_sparse(), fake, None, 3):
        out = torch.zeros_like(x)
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            dsa.dsa_rmsnorm(bad, w, 1e-6, out=out)
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            dsa.dsa_rmsnorm(x, w, 1e-6, out=out, residual=bad if bad is not None else 5)
        torch.cuda.synchronize()
        assert (out == 0).all()
        dsa.dsa_rmsnorm(x, w, 0.0, out=out)
        assert (out == 1).all()


@pytest.mark.parametrize("H,HI", [(64, 32), (65, 32), (64, 33), (1, 1), (7, 31)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_queries_of_few_heads(H, HI, dtype):
    """Around the heads that half the threads do for, against fp64."""
    dsa = lib()
    g = torch.Generator().manual_seed(H * HI)
    T = 200
    pos = torch.randint(0, 70000, (T,), generator=g).to(I32)
    fr = R.inv_freq()
    qr, qI = torch.randn((T, H, 64), generator=g).to(BF), torch.randn((T, HI, 128), generator=g).to(dtype)
    q = torch.zeros((T, H, 576), dtype=BF, device=DEV)
    q8, qs = torch.zeros((T, HI, 128), dtype=torch.uint8, device=DEV), torch.zeros(T, device=DEV)
    dsa.dsa_rope_queries(pos.to(DEV), fr.to(DEV), qr.to(DEV), q, qI.to(DEV), q8, qs)
    ref = R.rotate_main(R.d(qr), pos, fr)
    mag = R.d(qr).abs().unflatten(-1, (32, 2)).sum(-1, keepdim=True).expand(T, H, 32, 2).flatten(-2)
    R.check_close(q[:, :, 512:], ref, R.BF16 * ref.abs() + 8 * R.FP32 * mag, "main")
    y = R.rotate_index(R.d(qI), pos, fr).flatten(1)
    # a rotated value is off by 8 half steps of |a| + |b|, at most twice the pair's larger rotated magnitude and so the amax
    R.check_fp8(q8.flatten(1), qs, y, 16 * R.FP32, 0, "index")
