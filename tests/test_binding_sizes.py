"""Numbers that the library's int arguments cannot hold are refused by the binding: cut to 32 bits, they would pass the
library's checks as other sizes (no GPU)."""
import ctypes

import pytest
import torch

P, F, L = ctypes.c_void_p, ctypes.c_float, ctypes.c_int64
fake = P(4096)  # never dereferenced: every call fails a check on the host, or has nothing to do
BIG = [1 << 31, (1 << 32) + 64, 1 << 32, (1 << 63) + 5, (1 << 64) + 3, -(1 << 31) - 1, -(1 << 32) + 64]
U8, F32 = torch.uint8, torch.float32


@pytest.fixture(scope="module")
def dsa():
    from sparse_attention_02_gb300 import build

    build.build()
    import sparse_attention_02_gb300 as dsa

    return dsa


@pytest.mark.parametrize("n", BIG)
def test_no_int_argument_is_cut(dsa, n):
    lib = dsa.load_library(dsa.LIB_PATH)
    for M, N, K in ((n, 1, 256), (1, n, 256), (1, 1, n)):
        with pytest.raises(ctypes.ArgumentError):
            lib.dsa_gemm_fp8(fake, L(1 << 40), fake, fake, L(1 << 40), fake, 128, M, N, K, fake, L(1 << 40), 0, None)
    with pytest.raises(ctypes.ArgumentError):
        lib.dsa_layernorm(fake, L(64), None, L(0), fake, None, L(0), n, 0, 0, F(1e-6), None, L(0), fake, L(64), None, None, 0, 0, None)
    with pytest.raises(ctypes.ArgumentError):
        lib.dsa_rmsnorm(fake, L(64), None, L(0), fake, L(0), n, 0, 0, F(1e-6), None, L(0), fake, L(64), None, None, 0, 0, None)
    for size in (lib.dsa_layernorm_backward_workspace_size, lib.dsa_rmsnorm_backward_workspace_size):
        with pytest.raises(ctypes.ArgumentError):
            size(L(4), n)
    with pytest.raises(ctypes.ArgumentError):
        lib.dsa_topk(fake, L(64), n, fake, 4, fake, None)
    with pytest.raises(ctypes.ArgumentError):
        lib.dsa_topk(fake, L(64), 0, fake, n, fake, None)
    with pytest.raises(ctypes.ArgumentError):
        lib.dsa_indexer_topk_workspace_size(n, 1, 64, 128, 16)


def test_ints_that_fit_still_reach_the_library(dsa):
    lib = dsa.load_library(dsa.LIB_PATH)
    assert lib.dsa_gemm_fp8(fake, L(256), fake, fake, L(256), fake, 128, -(1 << 31), 1, 256, fake, L(64), 0, None) == 1
    assert lib.dsa_gemm_fp8(fake, L(256), fake, fake, L(256), fake, 128, (1 << 31) - 1, 1, 256, fake, L(64), 0, None) == 2
    assert lib.dsa_gemm_fp8(fake, L(256), fake, fake, L(256), fake, 128, ctypes.c_int(0), 1, 256, fake, L(64), 0, None) == 0
    assert lib.dsa_topk(fake, L(64), False, fake, 4, fake, None) in (0, 1)
    for wrong in (1.0, "4", None):
        with pytest.raises(ctypes.ArgumentError):
            lib.dsa_gemm_fp8(fake, L(256), fake, fake, L(256), fake, 128, wrong, 1, 256, fake, L(64), 0, None)


def empty(*shape, dtype=F32):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("n", [1 << 31, 1 << 32, (1 << 32) + 256])
def test_tensors_with_sizes_beyond_the_librarys_are_refused(dsa, n, monkeypatch):
    """... as the library refuses sizes that it can still be told, by DsaError 2.  The addresses and strides are taken from
    tensors without memory."""
    monkeypatch.setattr(dsa, "_native", lambda *a: False)
    monkeypatch.setattr(dsa, "_device", lambda: 0)
    monkeypatch.setattr(dsa, "_raw_stream", lambda stream, cur: 0)
    monkeypatch.setattr(dsa, "_at", lambda t, cur, name, dtype, shape: 4096)
    monkeypatch.setattr(dsa, "_at_rows", lambda t, cur, name, dtype, shape: (4096, max(t.stride(0), 16)))
    ws = empty(64, dtype=U8)
    monkeypatch.setattr(dsa, "_workspace", lambda workspace, need, cur, stream: (4096, 1 << 40, ws))

    def refused(f, *args, **kw):
        with pytest.raises(dsa.DsaError) as e:
            f(*args, **kw)
        assert e.value.code == 2 and str(n) in str(e.value)

    s = empty(1, -(-n // 128))
    refused(dsa.dsa_gemm_fp8, empty(1, n, dtype=U8), s, empty(1, n, dtype=U8), s, empty(1, 1))
    refused(dsa.dsa_gemm_fp8, empty(n, 16, dtype=U8), empty(n, 1), empty(1, 16, dtype=U8), empty(1, 1), empty(n, 1))
    refused(dsa.dsa_gemm_fp8, empty(1, 16, dtype=U8), empty(1, 1), empty(n, 16, dtype=U8), empty(n, 1), empty(1, n))
    x, w = empty(1, n), empty(n)
    refused(dsa.dsa_layernorm, x, w, w, 1e-6, out=x)
    refused(dsa.dsa_rmsnorm, x, w, 1e-6, out=x)
    refused(dsa.dsa_layernorm_backward, x, x, w, 1e-6, x, w)
    refused(dsa.dsa_rmsnorm_backward, x, x, w, 1e-6, x, w)
    refused(dsa.dsa_layernorm_backward_workspace_size, 4, n)
    refused(dsa.dsa_rmsnorm_backward_workspace_size, 4, n)
