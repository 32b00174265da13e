"""Refusals of the FP8 product, block quantisation and layer norm calls, taken on the host (no GPU)."""
import ctypes

import pytest
import torch

P, F, L = ctypes.c_void_p, ctypes.c_float, ctypes.c_int64
fake = P(4096)  # never dereferenced: every call below fails its host checks first, or has nothing to do
odd, two = P(4097), P(4098)


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_02_gb300 import build

    path = build.build()
    import sparse_attention_02_gb300 as dsa

    return dsa.load_library(path)


def test_gemm_refusals(lib):
    def call(a=fake, lda=256, sa=fake, b=fake, ldb=256, sb=fake, br=128, M=4, N=64, K=256, out=fake, ldo=64, t=0):
        return lib.dsa_gemm_fp8(a, L(lda), sa, b, L(ldb), sb, br, M, N, K, out, L(ldo), t, None)

    assert call(M=0) == 0 and call(N=0) == 0 and call(M=0, a=None, out=None) == 0
    assert call(M=-1) == 1 and call(N=-1) == 1 and call(K=-1) == 1
    assert call(br=0) == 1 and call(br=64) == 1 and call(t=2) == 1
    for name in ("a", "sa", "b", "sb", "out"):
        assert call(**{name: None}) == 1
    assert call(lda=240) == 1 and call(ldb=255) == 1 and call(ldo=63) == 1
    assert call(lda=257) == 3 and call(ldb=264) == 3 and call(a=P(4104)) == 3 and call(b=P(4104)) == 3
    assert call(sa=two) == 3 and call(sb=two) == 3 and call(out=odd) == 3 and call(out=two, t=1) == 3
    big = (1 << 30) + 1
    assert call(M=big) == 2 and call(N=big, ldo=big) == 2 and call(K=big, lda=1 << 31, ldb=1 << 31) == 2
    assert call(M=1 << 30, lda=1 << 20) == 2 and call(M=1 << 30, N=1 << 30, ldo=1 << 30) == 2
    assert "too large" in lib.dsa_last_error().decode()


def test_quantize_blocks_refusals(lib):
    def call(x=fake, ldx=300, rows=4, cols=300, dt=0, br=1, mode=0, c=fake, ldc=304, s=fake, ct=fake, ldt=16, st=fake):
        return lib.dsa_quantize_fp8_blocks(x, L(ldx), L(rows), L(cols), dt, br, mode, c, L(ldc), s, ct, L(ldt), st, None)

    assert call(rows=0) == 0 and call(rows=0, x=None) == 0
    assert call(rows=-1) == 1 and call(cols=0) == 1 and call(dt=2) == 1 and call(br=2) == 1 and call(mode=2) == 1
    assert call(x=None) == 1 and call(s=None) == 1 and call(c=None) == 1 and call(st=None) == 1 and call(ct=None) == 1
    assert call(c=None, s=None, ct=None, st=None) == 1
    assert call(ldx=299) == 1 and call(ldc=299) == 1 and call(ldt=3) == 1
    assert call(rows=1 << 40, ldt=1 << 40) == 2 and call(ldx=1 << 45) == 2 and call(ldc=1 << 45) == 2 and call(ldt=1 << 45) == 2
    assert call(x=odd) == 3 and call(x=two, dt=1) == 3 and call(s=two) == 3 and call(st=two) == 3


def test_layernorm_refusals(lib):
    def call(x=fake, ldx=64, res=None, ldr=0, w=fake, b=fake, rows=4, cols=64, dt=0, wt=0, eps=1e-6, h=None, ldh=0, out=fake, ldo=64,
             codes=None, scale=None, block=0, mode=0):
        return lib.dsa_layernorm(x, L(ldx), res, L(ldr), w, b, L(rows), cols, dt, wt, F(eps), h, L(ldh), out, L(ldo), codes, scale,
                                 block, mode, None)

    assert call(rows=0) == 0
    assert call(rows=-1) == 1 and call(cols=0) == 1 and call(cols=16385, ldx=16385, ldo=16385) == 2
    assert call(dt=2) == 1 and call(wt=-1) == 1 and call(mode=2) == 1 and call(block=64) == 1
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1 and call(eps=float("inf")) == 1
    assert call(x=None) == 1 and call(w=None) == 1 and call(out=None) == 1 and call(codes=fake) == 1 and call(scale=fake) == 1
    assert call(ldx=63) == 1 and call(ldo=63) == 1 and call(res=fake, ldr=10) == 1 and call(h=fake, ldh=0) == 1
    assert call(rows=1 << 31) == 2 and call(ldx=1 << 45) == 2
    assert call(x=odd) == 3 and call(res=odd, ldr=64) == 3 and call(out=odd) == 3 and call(w=odd) == 3 and call(b=odd) == 3
    assert call(b=two, wt=1) == 3 and call(x=two, dt=1) == 3 and call(codes=odd, scale=two) == 3


def test_layernorm_backward_refusals(lib):
    def call(dy=fake, h=fake, w=fake, e=None, rows=4, cols=64, dt=0, wt=0, eps=1e-6, dx=fake, dw=fake, db=fake, ws=fake, n=1 << 40):
        return lib.dsa_layernorm_backward(dy, h, w, e, L(rows), cols, dt, wt, F(eps), dx, dw, db, ws, n, None)

    assert call(dw=None) == 1 and call(rows=-1) == 1 and call(cols=0) == 1 and call(cols=16385) == 2
    assert call(dt=5) == 1 and call(wt=5) == 1 and call(eps=-1.0) == 1 and call(rows=1 << 31) == 2
    for name in ("dy", "h", "w", "dx"):
        assert call(**{name: None}) == 1
    assert call(dy=odd) == 3 and call(h=odd) == 3 and call(e=odd) == 3 and call(dx=odd) == 3 and call(dw=two) == 3 and call(db=two) == 3
    assert call(w=two, wt=1) == 3
    need = lib.dsa_layernorm_backward_workspace_size(L(4), 64)
    assert need >= 2 * lib.dsa_rmsnorm_backward_workspace_size(L(4), 64) > 0
    assert call(n=need - 1) == 4 and call(ws=None) == 4 and call(ws=P(4104)) == 3
    assert lib.dsa_layernorm_backward_workspace_size(L(-1), 64) == 0
    assert lib.dsa_layernorm_backward_workspace_size(L(4), 16385) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes(monkeypatch):
    """The binding's own checks come before the library: dtypes, shapes and devices."""
    import sparse_attention_02_gb300 as dsa

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x, w, u = torch.zeros(2, 8), torch.zeros(8), torch.zeros(2, 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_layernorm(x, w, w, 1e-6, out=x)
    with pytest.raises(TypeError):
        dsa.dsa_layernorm(x.half(), w, w, 1e-6, out=x)
    with pytest.raises(TypeError):
        dsa.dsa_layernorm(x[0], w, None, 1e-6, out=x)
    with pytest.raises(TypeError):
        dsa.dsa_layernorm_backward(x, x.half(), w, 1e-6, x, w)
    with pytest.raises(TypeError):
        dsa.dsa_quantize_fp8_blocks(u)
    with pytest.raises(ValueError, match="block_rows"):
        dsa.dsa_quantize_fp8_blocks(x, block_rows=64)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_quantize_fp8_blocks(x, codes=u)
    with pytest.raises(TypeError):
        dsa.dsa_gemm_fp8(u[0], w, u, x, x)
    with pytest.raises(TypeError):
        dsa.dsa_gemm_fp8(u, x, u, x, u)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_gemm_fp8(u, x, u, x, x)
