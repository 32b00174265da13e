"""Refusals of the norm, cache-append, query-rotation and dense-MLA calls, taken on the host (no GPU)."""
import ctypes

import pytest
import torch

P, F, L = ctypes.c_void_p, ctypes.c_float, ctypes.c_int64
fake = P(4096)  # never dereferenced: every call below fails its host checks first, or has nothing to do


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_02_gb300 import build

    path = build.build()
    import sparse_attention_02_gb300 as dsa

    return dsa.load_library(path)


def test_rmsnorm_refusals(lib):
    def call(x=fake, ldx=64, res=None, ldr=0, w=fake, rows=4, cols=64, dt=0, wt=0, eps=1e-6, h=None, ldh=0, out=fake, ldo=64,
             codes=None, scale=None, block=0, mode=0):
        return lib.dsa_rmsnorm(x, L(ldx), res, L(ldr), w, L(rows), cols, dt, wt, F(eps), h, L(ldh), out, L(ldo), codes, scale,
                               block, mode, None)

    assert call(rows=0) == 0
    assert call(rows=-1) == 1 and call(cols=0) == 1 and call(cols=16385, ldx=16385, ldo=16385) == 2
    assert call(dt=2) == 1 and call(wt=-1) == 1 and call(mode=2) == 1 and call(block=64) == 1
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1 and call(eps=float("inf")) == 1
    assert call(x=None) == 1 and call(w=None) == 1 and call(out=None) == 1
    assert call(codes=fake) == 1 and call(scale=fake) == 1
    assert call(ldx=63) == 1 and call(ldo=63) == 1 and call(res=fake, ldr=10) == 1 and call(h=fake, ldh=0) == 1
    assert call(rows=1 << 31) == 2 and call(ldx=1 << 45) == 2
    assert "rows too large" in lib.dsa_last_error().decode()


def test_rmsnorm_backward_refusals(lib):
    def call(dy=fake, h=fake, w=fake, rows=0, cols=64, dt=0, wt=0, eps=1e-6, dx=fake, dw=fake):
        return lib.dsa_rmsnorm_backward(dy, h, w, None, L(rows), cols, dt, wt, F(eps), dx, dw, None, 0, None)

    assert call(dw=None) == 1 and call(rows=-1) == 1 and call(cols=0) == 1 and call(cols=16385) == 2
    assert call(dt=5) == 1 and call(wt=5) == 1 and call(eps=-1.0) == 1
    for name in ("dy", "h", "w", "dx"):
        assert call(rows=4, **{name: None}) == 1
    assert call(rows=1 << 31) == 2
    assert lib.dsa_rmsnorm_backward_workspace_size(L(-1), 64) == 0
    assert lib.dsa_rmsnorm_backward_workspace_size(L(0), 64) == 0
    assert lib.dsa_rmsnorm_backward_workspace_size(L(4), 16385) == 0


def test_cache_append_refusals(lib):
    def call(pos=fake, seq=None, T=4, bt=fake, ns=4, mp=2, np_=8, ps=64, fr=fake, kv=fake, ld=576, w=None, wt=0, eps=1e-6, kp=fake,
             kI=fake, ldI=128, kt=0, mode=0, k8=fake, ks=fake):
        return lib.dsa_cache_append(pos, seq, T, bt, ns, mp, np_, ps, fr, kv, L(ld), w, wt, F(eps), kp, kI, L(ldI), kt, mode, k8, ks, None)

    assert call(T=0) == 0 and call(T=0, ns=0) == 0
    assert call(T=-1) == 1 and call(ns=0) == 1 and call(mp=0) == 1 and call(np_=0) == 1
    assert call(ps=16) == 2 and call(ps=96) == 2
    assert call(wt=2) == 1 and call(kt=2) == 1 and call(mode=2) == 1 and call(eps=-1.0) == 1
    assert call(pos=None) == 1 and call(bt=None) == 1 and call(fr=None) == 1 and call(kp=None) == 1
    assert call(kv=None, kI=None) == 1 and call(k8=None) == 1 and call(ks=None) == 1
    assert call(ns=3) == 1                                    # four tokens, no seq, three table rows
    assert call(ld=575) == 1 and call(ldI=100) == 1 and call(ld=1 << 45) == 2
    assert call(kv=P(4104)) == 3 and call(ld=580) == 3 and call(kp=P(4100)) == 3 and call(w=P(4098)) == 3
    assert call(kI=P(4104)) == 3 and call(ldI=132) == 3 and call(k8=P(4104)) == 3
    assert call(kI=fake, kt=1, ldI=130) == 3


def test_rope_queries_refusals(lib):
    def call(pos=fake, fr=fake, T=4, qr=fake, st=8192, sh=64, H=128, q=fake, qI=fake, HI=64, it=0, mode=0, q8=fake, qs=fake):
        return lib.dsa_rope_queries(pos, fr, T, qr, L(st), L(sh), H, q, qI, HI, it, mode, q8, qs, None)

    assert call(T=0) == 0 and call(T=-1) == 1
    assert call(pos=None) == 1 and call(fr=None) == 1 and call(q=None) == 1 and call(q8=None) == 1 and call(qs=None) == 1
    assert call(qr=None, qI=None) == 1
    assert call(H=0) == 2 and call(H=129) == 2 and call(HI=0) == 2 and call(HI=65) == 2
    assert call(it=3) == 1 and call(mode=3) == 1 and call(st=-8) == 1 and call(sh=1 << 45) == 1
    assert call(qr=P(4104)) == 3 and call(q=P(4104)) == 3 and call(qI=P(4104)) == 3 and call(q8=P(4104)) == 3 and call(sh=68) == 3


def test_index_rope_backward_refusals(lib):
    def call(g=fake, pos=fake, fr=fake, T=4, HI=64, dx=fake, dt=0):
        return lib.dsa_index_rope_backward(g, pos, fr, T, HI, dx, dt, None)

    assert call(T=0) == 0 and call(T=-1) == 1 and call(HI=0) == 2 and call(HI=65) == 2 and call(dt=2) == 1
    assert call(g=None) == 1 and call(pos=None) == 1 and call(fr=None) == 1 and call(dx=None) == 1
    assert call(g=P(4104)) == 3 and call(dx=P(4104)) == 3


def test_dense_mla_refusals(lib):
    def call(q=fake, kv=fake, np_=8, ps=64, bt=fake, mp=2, ctx=fake, B=2, H=128, sc=0.04, out=fake, lse=fake, ws=P(1 << 20),
             n=1 << 40):
        return lib.dsa_mla_decode_paged(q, kv, np_, ps, bt, mp, ctx, B, H, F(sc), out, lse, ws, n, None)

    assert call(B=0) == 0 and call(B=-1) == 1 and call(B=65536) == 2
    assert call(H=0) == 2 and call(H=129) == 2 and call(ps=16) == 2 and call(np_=0) == 1 and call(mp=0) == 1
    assert call(np_=1 << 25, ps=128) == 2 and call(mp=1 << 25, ps=128) == 2
    for name in ("q", "kv", "bt", "ctx", "out", "lse"):
        assert call(**{name: None}) == 1
    assert call(q=P(4104)) == 3 and call(kv=P(4104)) == 3 and call(out=P(4104)) == 3
    assert call(sc=0.0) == 1 and call(sc=float("nan")) == 1 and call(sc=2e30) == 1
    need = lib.dsa_mla_decode_workspace_size(2, 128)
    assert need > 0 and call(n=need - 1) == 4 and call(ws=None) == 4 and call(ws=P((1 << 20) + 64)) == 3
    assert lib.dsa_mla_decode_workspace_size(0, 16) == 0 and lib.dsa_mla_decode_workspace_size(1, 129) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes(monkeypatch):
    """The binding's own checks come before the library: dtypes, shapes and devices."""
    import sparse_attention_02_gb300 as dsa

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x, w = torch.zeros(2, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_rmsnorm(x, w, 1e-6, out=x)
    with pytest.raises(TypeError):
        dsa.dsa_rmsnorm(x.half(), w, 1e-6, out=x)
    with pytest.raises(TypeError):
        dsa.dsa_rmsnorm(x[0], w, 1e-6, out=x)
    with pytest.raises(ValueError, match="kv or kI"):
        dsa.dsa_cache_append(w, x, w)
    with pytest.raises(ValueError, match="q_rope or qI"):
        dsa.dsa_rope_queries(w.int(), w.double())
    with pytest.raises(ValueError, match="128"):
        dsa.dsa_index_rope_backward(x, w, w, x)
    with pytest.raises(TypeError):
        dsa.dsa_mla_decode_paged(x, x, x, w, 1.0, x, x)


def test_misaligned_elements_and_token_counts_are_refused(lib):
    """Addresses that are no multiple of an element, which a kernel could only fault on."""
    odd, two, four = P(4097), P(4098), P(4100)

    def norm(x=fake, w=fake, res=None, dt=0, wt=0, h=None, out=fake, codes=None, scale=None):
        return lib.dsa_rmsnorm(x, L(64), res, L(64), w, L(4), 64, dt, wt, F(1e-6), h, L(64), out, L(64), codes, scale, 0, 0, None)

    assert norm(x=odd) == 3 and norm(res=odd) == 3 and norm(h=odd) == 3 and norm(out=odd) == 3 and norm(w=odd) == 3
    assert norm(x=two, dt=1) == 3 and norm(w=two, wt=1) == 3 and norm(codes=odd, scale=two) == 3

    def back(dy=fake, h=fake, w=fake, e=None, dt=0, wt=0, dx=fake, dw=fake):
        return lib.dsa_rmsnorm_backward(dy, h, w, e, L(4), 64, dt, wt, F(1e-6), dx, dw, fake, 1 << 40, None)

    assert back(dy=odd) == 3 and back(h=odd) == 3 and back(e=odd) == 3 and back(dx=odd) == 3 and back(dw=two) == 3
    assert back(w=odd) == 3 and back(w=two, wt=1) == 3 and back(dx=two, dt=1) == 3

    def append(pos=fake, seq=None, T=4, bt=fake, fr=fake, ks=fake):
        return lib.dsa_cache_append(pos, seq, T, bt, T, 2, 8, 64, fr, None, L(0), None, 0, F(1e-6), None, fake, L(128), 0, 0, fake, ks, None)

    assert append(pos=two) == 3 and append(seq=two) == 3 and append(bt=two) == 3 and append(fr=four) == 3 and append(ks=two) == 3
    assert append(T=(1 << 30) + 1) == 2

    def queries(pos=fake, fr=fake, qs=fake):
        return lib.dsa_rope_queries(pos, fr, 4, None, L(0), L(0), 0, None, fake, 64, 0, 0, fake, qs, None)

    assert queries(pos=two) == 3 and queries(fr=four) == 3 and queries(qs=two) == 3

    def turn_back(pos=fake, fr=fake, T=4):
        return lib.dsa_index_rope_backward(fake, pos, fr, T, 1, fake, 0, None)

    assert turn_back(pos=two) == 3 and turn_back(fr=four) == 3 and turn_back(T=(1 << 30) + 1) == 2

    def attend(bt=fake, ctx=fake, lse=fake):
        return lib.dsa_mla_decode_paged(fake, fake, 8, 64, bt, 2, ctx, 2, 128, F(0.04), fake, lse, P(1 << 20), 1 << 40, None)

    assert attend(bt=two) == 3 and attend(ctx=two) == 3 and attend(lse=two) == 3
