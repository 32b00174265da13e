"""The binding of the norm, rotation and dense MLA calls on the GPU: the native path and the Python one do the same,
and wrong arguments are refused with their names before anything is launched."""
import pytest
import torch

from tests import operator_refs as R
from tests.gpu_util import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def zeros(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype, device=DEV)


def rand(*shape, dtype=F32):
    return torch.randn(shape, device=DEV).to(dtype)


def calls():
    """name -> (function name, arguments, the outputs)."""
    fr = R.inv_freq().to(DEV)
    pos = torch.tensor([3, 70, -1, 5], dtype=I32, device=DEV)
    bt = torch.arange(8, dtype=I32, device=DEV).view(4, 2)
    q8, qs, k8, ks = zeros(4, 2, 128, dtype=U8), zeros(4), zeros(8, 64, 128, dtype=U8), zeros(8, 64)
    out, h, codes, scale = zeros(4, 256), zeros(4, 256), zeros(4, 256, dtype=U8), zeros(4, 2)
    pool, q, dx, dw = zeros(8, 64, 576, dtype=BF), zeros(4, 3, 576, dtype=BF), zeros(4, 256), zeros(256)
    o, lse, di = zeros(4, 16, 512, dtype=BF), zeros(4, 16), zeros(4, 2, 128, dtype=BF)
    ctx = torch.tensor([1, 128, 0, 77], dtype=I32, device=DEV)
    wide = rand(4, 300)
    return {
        "dsa_rmsnorm": (dict(x=wide[:, 40:296], weight=rand(256, dtype=BF), eps=1e-6, out=out, residual=rand(4, 256), residual_out=h,
                             codes=codes, scale=scale, block=128), (out, h, codes, scale)),
        "dsa_rmsnorm_backward": (dict(dy=rand(4, 256), h=rand(4, 256), weight=rand(256), eps=1e-6, dx=dx, dweight=dw), (dx, dw)),
        "dsa_cache_append": (dict(pos=pos, block_table=bt, inv_freq=fr, kv=rand(4, 600, dtype=BF)[:, 8:584], kv_pool=pool, kI=rand(4, 128),
                                  k8_pool=k8, ks_pool=ks, seq=torch.tensor([3, 2, 0, 1], dtype=I32, device=DEV),
                                  kv_weight=rand(512)), (pool, k8, ks)),
        "dsa_rope_queries": (dict(pos=pos, inv_freq=fr, q_rope=rand(4, 3, 192, dtype=BF)[..., 128:], q=q, qI=rand(4, 2, 128), q8=q8,
                                  q_scale=qs), (q, q8, qs)),
        "dsa_index_rope_backward": (dict(g=rand(4, 2, 128), pos=pos, inv_freq=fr, dx=di), (di,)),
        "dsa_mla_decode_paged": (dict(q=rand(4, 16, 576, dtype=BF), kv_pool=rand(8, 64, 576, dtype=BF), block_table=bt, ctx_len=ctx,
                                      sm_scale=0.04, out=o, lse=lse), (o, lse)),
    }


class Nothing:
    def __getattr__(self, name):
        return lambda *a: NotImplemented


@pytest.mark.parametrize("name", ["dsa_rmsnorm", "dsa_rmsnorm_backward", "dsa_cache_append", "dsa_rope_queries",
                                  "dsa_index_rope_backward", "dsa_mla_decode_paged"])
def test_native_and_python_paths_agree(name, monkeypatch):
    dsa = lib()
    kw, outs = calls()[name]
    taken = []
    native = dsa._fast

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
    for t in outs:
        t.zero_()
    monkeypatch.setattr(dsa, "_fast", Nothing())
    getattr(dsa, name)(**kw)
    for a, b in zip(outs, first):
        assert torch.equal(a, b)
    for t in outs:
        t.zero_()
    monkeypatch.setattr(dsa, "_fast", native)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    getattr(dsa, name)(**kw, stream=side)
    side.synchronize()
    for a, b in zip(outs, first):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["dsa_rmsnorm", "dsa_rmsnorm_backward", "dsa_cache_append", "dsa_rope_queries",
                                  "dsa_index_rope_backward", "dsa_mla_decode_paged"])
def test_wrong_tensors_are_refused_by_name(name):
    dsa = lib()
    kw, outs = calls()[name]
    func = getattr(dsa, name)
    for arg, t in kw.items():
        if not isinstance(t, torch.Tensor):
            continue
        wrong = {"host": t.cpu(), "dtype": t.to(torch.float16), "shape": t.unsqueeze(0).contiguous(), "object": t.tolist()}
        if t.dim() > 1 and arg not in ("block_table",):
            bigger = torch.empty(t.shape[:-1] + (2 * t.shape[-1],), dtype=t.dtype, device=DEV)
            wrong["strided"] = bigger[..., ::2]
        for kind, w in wrong.items():
            with pytest.raises((TypeError, ValueError)) as e:
                func(**{**kw, arg: w})
            assert arg in str(e.value) or kind in ("shape", "host", "object", "dtype"), (arg, kind, str(e.value))
    torch.cuda.synchronize()
    for t in outs:
        assert (t == 0).all()  # nothing was launched


def test_library_refusals_reach_python():
    dsa = lib()
    kw, _ = calls()["dsa_rmsnorm"]
    with pytest.raises(dsa.DsaError, match="go together"):
        dsa.dsa_rmsnorm(**{**kw, "scale": None})
    with pytest.raises(dsa.DsaError, match="block"):
        dsa.dsa_rmsnorm(**{**kw, "block": 64, "scale": zeros(4, 4)})
    kw, _ = calls()["dsa_mla_decode_paged"]
    with pytest.raises(dsa.DsaError, match="workspace"):
        dsa.dsa_mla_decode_paged(**kw, workspace=zeros(256, dtype=U8))
    with pytest.raises(dsa.DsaError, match="sm_scale"):
        dsa.dsa_mla_decode_paged(**{**kw, "sm_scale": 0.0})
    with pytest.raises(dsa.DsaError, match="page_size"):
        dsa.dsa_mla_decode_paged(**{**kw, "kv_pool": zeros(8, 48, 576, dtype=BF)})
    kw, _ = calls()["dsa_cache_append"]
    with pytest.raises(dsa.DsaError, match="aligned"):
        dsa.dsa_cache_append(**{**kw, "kv": rand(4, 600, dtype=BF)[:, 1:577]})
    with pytest.raises(ValueError, match="kv or kI"):
        dsa.dsa_cache_append(**{**kw, "kv": None, "kI": None})
