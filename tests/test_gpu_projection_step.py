"""The norms, block quantisation and FP8 products run together as a layer's projections of a served model and as their
training step, against the same chain in fp64.

Each operator's reference starts again from the inputs that it was given, so that each is held to its own rounding; the
projections as wholes are held to what FP8 operands cost."""
import math

import pytest
import torch

from tests import operator_refs as R
from tests import projection_refs as P
from tests.gpu_util import lib

pytestmark = pytest.mark.gpu
DEV, EPS, PAGE = "cuda", 1e-6, 64
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
D, N = 1024, 704  # hidden width; latent rows and index keys of one fused projection


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


class Projection:
    """A weight [n, k] with its FP8 codes in both layouts."""

    def __init__(self, dsa, n, k, g):
        self.w = (torch.randn((n, k), generator=g, device=DEV) / math.sqrt(k)).to(BF)
        self.codes, self.scale = P.padded(n, k, DEV), torch.empty((P.pieces(n), P.pieces(k)), device=DEV)
        self.codes_t, self.scale_t = P.padded(k, n, DEV), torch.empty((P.pieces(k), P.pieces(n)), device=DEV)
        dsa.dsa_quantize_fp8_blocks(self.w, self.codes, self.scale, self.codes_t, self.scale_t, block_rows=128)


def check_product(out, a, a_scale, b, b_scale, what):
    ref, mag = P.gemm(a, a_scale, b, b_scale)
    R.check_close(out, ref.cpu(), P.gemm_bound(ref, mag, a.shape[1], out.dtype).cpu(), what)


def check_whole(out, exact, mag, what):
    """E4M3 operands: each factor off by at most half a step of 2^-4 relative, or of its scale's smallest (2^-10 / 448 of the
    piece's largest value, far below); two factors a product."""
    err = (out.double() - exact).abs()
    assert (err <= (2 * R.E4M3 + R.E4M3 ** 2 + R.BF16) * mag + 2.0 ** -9 * mag.max()).all(), f"{what}: off by {float(err.max()):.3g}"


@pytest.mark.parametrize("T", [1, 5, 130, 700])
def test_serving_projections(T):
    """Residual, norm and FP8 codes, the fused projection to latent rows and index keys, the keys' layer norm, and the
    cache append that takes both as slices of the product."""
    dsa, g = lib(), gen(T)
    proj = Projection(dsa, N, D, g)
    x, res = (torch.randn((T, D), generator=g, device=DEV).to(BF) for _ in range(2))
    w = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(BF)
    kw, kb = (torch.randn(128, generator=g, device=DEV).to(BF) for _ in range(2))
    h, y = torch.empty_like(x), torch.empty_like(x)
    codes, scale = torch.empty((T, D), dtype=U8, device=DEV), torch.empty((T, D // 128), device=DEV)
    dsa.dsa_rmsnorm(x, w, EPS, out=y, residual=res, residual_out=h, codes=codes, scale=scale, block=128)
    out = torch.empty((T, N), dtype=BF, device=DEV)
    dsa.dsa_gemm_fp8(codes, scale, proj.codes, proj.scale, out)
    check_product(out, codes, scale, proj.codes, proj.scale, "projection")
    yd, wd = R.rmsnorm(x, res, w, EPS)[1].to(DEV), proj.w.double()
    check_whole(out, yd @ wd.T, yd.abs() @ wd.abs().T, "projection as a whole")
    kI = torch.empty((T, 128), dtype=BF, device=DEV)
    dsa.dsa_layernorm(out[:, 576:], kw, kb, EPS, out=kI)
    _, ref, mag = P.layernorm(out[:, 576:], None, kw, kb, EPS)
    R.check_close(kI, ref, ref.abs() * R.BF16 + 40 * R.FP32 * mag + 1e-30, "index keys")
    pages = -(-T // PAGE)
    table = torch.arange(pages, dtype=I32, device=DEV).view(1, pages)
    kv = torch.zeros((pages, PAGE, 576), dtype=BF, device=DEV)
    k8, ks = torch.zeros((pages, PAGE, 128), dtype=U8, device=DEV), torch.zeros((pages, PAGE), device=DEV)
    pos = torch.arange(T, dtype=I32, device=DEV)
    dsa.dsa_cache_append(pos, table, R.inv_freq().to(DEV), kv=out[:, :576], kv_pool=kv, kI=kI, k8_pool=k8, ks_pool=ks,
                         seq=torch.zeros(T, dtype=I32, device=DEV))
    assert torch.equal(kv.view(-1, 576)[:T, :512], out[:, :512])
    R.check_fp8(k8.view(-1, 128)[:T], ks.view(-1)[:T], R.rotate_index(R.d(kI), torch.arange(T), R.inv_freq()), 2.0 ** -19, 0, "index cache")
    assert dsa.dsa_get_device_status() == 0


@pytest.mark.parametrize("T", [1, 77, 300])
def test_training_step(T):
    """A projection between two norms and its backward: the gradient quantised for both products, the input's and the
    weight's gradient, and the norms' gradients, against fp64 from each operator's own inputs and, as wholes, against
    autograd."""
    dsa, g = lib(), gen(T + 10)
    n = 384
    proj = Projection(dsa, n, D, g)
    h = torch.randn((T, D), generator=g, device=DEV).to(BF)
    w1, w2, b2 = (torch.randn(k, generator=g, device=DEV).to(BF) for k in (D, n, n))
    y = torch.empty_like(h)
    a8, a_s = torch.empty((T, D), dtype=U8, device=DEV), torch.empty((T, D // 128), device=DEV)
    dsa.dsa_rmsnorm(h, w1, EPS, out=y, codes=a8, scale=a_s, block=128)
    at8, at_s = P.padded(D, T, DEV), torch.empty((D, P.pieces(T)), device=DEV)
    dsa.dsa_quantize_fp8_blocks(y, codes_t=at8, scale_t=at_s)
    z, o = torch.empty((T, n), dtype=BF, device=DEV), torch.empty((T, n), dtype=BF, device=DEV)
    dsa.dsa_gemm_fp8(a8, a_s, proj.codes, proj.scale, z)
    dsa.dsa_layernorm(z, w2, b2, EPS, out=o)
    # backward
    do = torch.randn((T, n), generator=g, device=DEV).to(BF)
    dz, dw2, db2 = torch.empty_like(z), torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    dsa.dsa_layernorm_backward(do, z, w2, EPS, dz, dw2, dbias=db2)
    rx, rw, rb, mag, wmag, bmag = P.layernorm_backward(do, z, w2, None, EPS)
    R.check_close(dz, rx, rx.abs() * R.BF16 + 120 * R.FP32 * mag + 1e-30, "dz")
    R.check_close(dw2, rw, 450 * R.FP32 * wmag + 1e-30, "dw2")
    R.check_close(db2, rb, 400 * R.FP32 * bmag + 1e-30, "db2")
    d8, d_s = torch.empty((T, n), dtype=U8, device=DEV), torch.empty((T, P.pieces(n)), device=DEV)
    dt8, dt_s = P.padded(n, T, DEV), torch.empty((n, P.pieces(T)), device=DEV)
    dsa.dsa_quantize_fp8_blocks(dz, d8, d_s, dt8, dt_s)
    dy, dw = torch.empty((T, D), dtype=BF, device=DEV), torch.empty((n, D), device=DEV)
    dsa.dsa_gemm_fp8(d8, d_s, proj.codes_t, proj.scale_t, dy)
    dsa.dsa_gemm_fp8(dt8, dt_s, at8, at_s, dw)
    check_product(dy, d8, d_s, proj.codes_t, proj.scale_t, "dy")
    check_product(dw, dt8, dt_s, at8, at_s, "dw")
    dzd, yd, wd = dz.double(), y.double(), proj.w.double()
    check_whole(dy, dzd @ wd, dzd.abs() @ wd.abs(), "dy as a whole")
    check_whole(dw, dzd.T @ yd, dzd.abs().T @ yd.abs(), "dw as a whole")
    dh, dw1 = torch.empty_like(h), torch.empty(D, device=DEV)
    dsa.dsa_rmsnorm_backward(dy, h, w1, EPS, dh, dw1)
    # the whole step against autograd of its definition, by the cosine of each gradient: FP8 operands turn a product's
    # result by no more than their own relative error, 2^-4 a factor at most and a third of it on average
    hd, w1d, wtd, w2d, b2d = (t.double().requires_grad_(True) for t in (h, w1, proj.w, w2, b2))
    v = hd / torch.sqrt(hd.square().mean(-1, keepdim=True) + EPS) * w1d
    q = v @ wtd.T
    c = q - q.mean(-1, keepdim=True)
    (c / torch.sqrt(c.square().mean(-1, keepdim=True) + EPS) * w2d + b2d).backward(do.double())
    for got, ref, what in ((dh, hd.grad, "dh"), (dw, wtd.grad, "dw"), (dw2, w2d.grad, "dw2"), (db2, b2d.grad, "db2")):
        a, b = got.double().flatten(), ref.flatten()
        assert float(a @ b / (a.norm() * b.norm())) >= 1 - (4 * R.E4M3) ** 2 / 2, what
    assert dsa.dsa_get_device_status() == 0


def test_padded_batch_in_one_graph():
    """A captured decode step's projections over a batch with unused rows: a replay gives each row what it gets alone,
    whatever the other rows hold."""
    dsa, g = lib(), gen(20)
    T = 6
    proj = Projection(dsa, N, D, g)
    w, kw, kb = (torch.randn(k, generator=g, device=DEV).to(BF) for k in (D, 128, 128))
    x = torch.zeros((T, D), dtype=BF, device=DEV)
    codes, scale = torch.empty((T, D), dtype=U8, device=DEV), torch.empty((T, D // 128), device=DEV)
    out, kI = torch.empty((T, N), dtype=BF, device=DEV), torch.empty((T, 128), dtype=BF, device=DEV)

    def step(x, codes, scale, out, kI):
        dsa.dsa_rmsnorm(x, w, EPS, codes=codes, scale=scale, block=128)
        dsa.dsa_gemm_fp8(codes, scale, proj.codes, proj.scale, out)
        dsa.dsa_layernorm(out[:, 576:], kw, kb, EPS, out=kI)

    step(x, codes, scale, out, kI)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(x, codes, scale, out, kI)
    for used in (T, 3, 1):
        x.copy_(torch.randn((T, D), generator=g, device=DEV))
        x[used:] = float("nan")  # rows that nothing uses
        graph.replay()
        torch.cuda.synchronize()
        for r in range(used):
            alone = [torch.empty_like(t[:1]) for t in (codes, scale, out, kI)]
            step(x[r:r + 1].clone(), *alone)
            for a, b in zip(alone, (codes, scale, out, kI)):
                assert torch.equal(a[0], b[r])
