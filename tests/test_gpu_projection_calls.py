"""The binding of the FP8 product, block quantisation and layer norm calls: the native path and the Python one do the same,
wrong arguments are refused with their names before anything is launched, and calls mix as programs mix them."""
import subprocess
import sys
import threading

import pytest
import torch

from tests import projection_refs as P
from tests.gpu_util import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
NAMES = ["dsa_layernorm", "dsa_layernorm_backward", "dsa_quantize_fp8_blocks", "dsa_gemm_fp8"]


def rand(*shape, dtype=F32, g=None):
    return torch.randn(shape, generator=g).to(dtype).to(DEV)


def zeros(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype, device=DEV)


def calls():
    """name -> (arguments, the outputs)."""
    g = torch.Generator().manual_seed(1)
    dg = torch.Generator(device=DEV)
    dg.manual_seed(1)
    out, h, codes, scale = zeros(4, 256), zeros(4, 256), zeros(4, 256, dtype=U8), zeros(4, 2)
    dx, dw, db = zeros(4, 256), zeros(256), zeros(256)
    c, s, ct, st = zeros(40, 320, dtype=U8), zeros(40, 3), zeros(300, 48, dtype=U8), zeros(300, 1)
    prod = zeros(20, 70, dtype=BF)
    wide = rand(4, 300, g=g)
    return {
        "dsa_layernorm": (dict(x=wide[:, 40:296], weight=rand(256, dtype=BF, g=g), bias=rand(256, dtype=BF, g=g), eps=1e-6, out=out,
                               residual=rand(4, 256, g=g), residual_out=h, codes=codes, scale=scale, block=128), (out, h, codes, scale)),
        "dsa_layernorm_backward": (dict(dy=rand(4, 256, g=g), h=rand(4, 256, g=g), weight=rand(256, g=g), eps=1e-6, dx=dx, dweight=dw,
                                        dbias=db, dres=rand(4, 256, g=g)), (dx, dw, db)),
        "dsa_quantize_fp8_blocks": (dict(x=rand(40, 300, dtype=BF, g=g), codes=c[:, :300], scale=s, codes_t=ct[:, :40], scale_t=st),
                                    (c, s, ct, st)),
        "dsa_gemm_fp8": (dict(a=P.codes_like(20, 300, dg, DEV), a_scale=P.scales_like((20, 3), dg, DEV), b=P.codes_like(70, 300, dg, DEV),
                              b_scale=P.scales_like((70, 3), dg, DEV), out=prod), (prod,)),
    }


class Nothing:
    def __getattr__(self, name):
        return lambda *a: NotImplemented


@pytest.mark.parametrize("name", NAMES)
def test_native_and_python_paths_agree(name, monkeypatch):
    dsa = lib()
    kw, outs = calls()[name]
    taken, native = [], dsa._fast

    class Spy:
        def __getattr__(self, n):
            def f(*a):
                rc = getattr(native, n)(*a)
                taken.append(rc)
                return rc
            return f

    monkeypatch.setattr(dsa, "_fast", Spy())
    getattr(dsa, name)(**kw)
    first = [t.clone() for t in outs]
    assert taken == [0]  # a plain call is made natively
    for other in (Nothing(), native):
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        monkeypatch.setattr(dsa, "_fast", other)
        side = torch.cuda.Stream()
        getattr(dsa, name)(**kw, stream=side)
        side.synchronize()
        for a, b in zip(outs, first):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_wrong_tensors_are_refused_by_name(name):
    dsa = lib()
    kw, outs = calls()[name]
    for arg, t in kw.items():
        if not isinstance(t, torch.Tensor):
            continue
        wrong = {"host": t.cpu(), "dtype": t.to(torch.float16), "shape": t.unsqueeze(0).contiguous(), "object": t.tolist()}
        if t.dim() > 1:
            bigger = torch.empty(t.shape[:-1] + (2 * t.shape[-1],), dtype=t.dtype, device=DEV)
            wrong["strided"] = bigger[..., ::2]
        for kind, w in wrong.items():
            with pytest.raises((TypeError, ValueError)) as e:
                getattr(dsa, name)(**{**kw, arg: w})
            assert arg in str(e.value) or kind != "strided", (arg, kind, str(e.value))
    torch.cuda.synchronize()
    for t in outs:
        assert (t == 0).all()  # nothing was launched


def test_library_refusals_reach_python():
    dsa = lib()
    kw, _ = calls()["dsa_gemm_fp8"]
    tight = torch.zeros((20, 300), dtype=U8, device=DEV)  # rows at 300 bytes
    with pytest.raises(dsa.DsaError, match="16-byte"):
        dsa.dsa_gemm_fp8(**{**kw, "a": tight})
    with pytest.raises(dsa.DsaError, match="16-byte"):
        dsa.dsa_gemm_fp8(**{**kw, "b": torch.zeros((70, 320), dtype=U8, device=DEV)[:, 1:301]})
    kw, _ = calls()["dsa_quantize_fp8_blocks"]
    with pytest.raises(dsa.DsaError, match="go together"):
        dsa.dsa_quantize_fp8_blocks(**{**kw, "scale": None})
    with pytest.raises(dsa.DsaError, match="no output"):
        dsa.dsa_quantize_fp8_blocks(kw["x"])
    with pytest.raises(dsa.DsaError, match="scale_mode"):
        dsa.dsa_quantize_fp8_blocks(**kw, scale_mode=2)
    kw, _ = calls()["dsa_layernorm"]
    with pytest.raises(dsa.DsaError, match="block"):
        dsa.dsa_layernorm(**{**kw, "block": 64, "scale": zeros(4, 4)})
    kw, _ = calls()["dsa_layernorm_backward"]
    with pytest.raises(dsa.DsaError, match="workspace"):
        dsa.dsa_layernorm_backward(**kw, workspace=zeros(256, dtype=U8))


def step(seed, stream=None):
    """A small step over all of the calls, as a function that enqueues it, and the tensors that it writes."""
    dsa = lib()
    g = torch.Generator().manual_seed(seed)
    T, D, N = 70 + 60 * seed, 520, 384
    x, w, b = rand(T, D, dtype=BF, g=g), rand(D, dtype=BF, g=g), rand(D, dtype=BF, g=g)
    wt, dy = rand(N, D, dtype=BF, g=g), rand(T, N, dtype=BF, g=g)
    kd, kn, kt = P.pieces(D), P.pieces(N), P.pieces(T)
    r = dict(y=zeros(T, D, dtype=BF), c=zeros(T, 528, dtype=U8), s=zeros(T, kd), ct=zeros(D, (T + 15) // 16 * 16, dtype=U8), st=zeros(D, kt),
             w8=zeros(N, 528, dtype=U8), ws=zeros(kn, kd), w8t=zeros(D, N, dtype=U8), wst=zeros(kd, kn),
             d8=zeros(T, N, dtype=U8), ds=zeros(T, kn), d8t=zeros(N, (T + 15) // 16 * 16, dtype=U8), dst=zeros(N, kt),
             out=zeros(T, N, dtype=BF), dx=zeros(T, D, dtype=BF), dwt=zeros(N, D), dh=zeros(T, D, dtype=BF), dw=zeros(D), db=zeros(D))

    def run():
        dsa.dsa_layernorm(x, w, b, 1e-6, out=r["y"], stream=stream)
        dsa.dsa_quantize_fp8_blocks(r["y"], r["c"][:, :D], r["s"], r["ct"][:, :T], r["st"], stream=stream)
        dsa.dsa_quantize_fp8_blocks(wt, r["w8"][:, :D], r["ws"], r["w8t"], r["wst"], block_rows=128, stream=stream)
        dsa.dsa_gemm_fp8(r["c"][:, :D], r["s"], r["w8"][:, :D], r["ws"], r["out"], stream=stream)
        dsa.dsa_quantize_fp8_blocks(dy, r["d8"], r["ds"], r["d8t"][:, :T], r["dst"], stream=stream)
        dsa.dsa_gemm_fp8(r["d8"], r["ds"], r["w8t"], r["wst"], r["dx"], stream=stream)
        dsa.dsa_gemm_fp8(r["d8t"][:, :T], r["dst"], r["ct"][:, :T], r["st"], r["dwt"], stream=stream)
        dsa.dsa_layernorm_backward(r["dx"], x, w, 1e-6, r["dh"], r["dw"], dbias=r["db"], stream=stream)

    return run, r


def same(a, b):
    return torch.equal(a.view(U8), b.view(U8))


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
                for _ in range(20):
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


FIRST = """
import torch
from tests.test_gpu_projection_calls import step, same
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


def test_two_graphs_share_a_workspace():
    """Two captured backward passes over one workspace, replayed one after the other in either order."""
    dsa = lib()
    g = torch.Generator().manual_seed(3)
    rows, cols = 600, 512
    ws = torch.empty(dsa.dsa_layernorm_backward_workspace_size(rows, cols), dtype=U8, device=DEV)
    sets = []
    for i in range(2):
        kw = dict(dy=rand(rows, cols, g=g), h=rand(rows, cols, g=g), weight=rand(cols, g=g), eps=1e-6, dx=zeros(rows, cols), dweight=zeros(cols),
                  dbias=zeros(cols))
        dsa.dsa_layernorm_backward(**kw)
        torch.cuda.synchronize()
        want = [kw[k].clone() for k in ("dx", "dweight", "dbias")]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dsa.dsa_layernorm_backward(**kw, workspace=ws)
        sets.append((graph, kw, want))
    for order in ((0, 1), (1, 0), (0, 0)):
        for _, kw, _ in sets:
            for k in ("dx", "dweight", "dbias"):
                kw[k].zero_()
        for i in order:
            sets[i][0].replay()
        torch.cuda.synchronize()
        for i in set(order):
            for k, w in zip(("dx", "dweight", "dbias"), sets[i][2]):
                assert torch.equal(sets[i][1][k], w)
