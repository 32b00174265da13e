"""dsa_rmsnorm (+ backward), dsa_cache_append, dsa_rope_queries and dsa_index_rope_backward on the GPU against
their definitions in fp64.

Bounds.  y = h r w: h one rounding, the sum of squares at most 8 + 4 + 10 additions in a chain (its relative
error halves under the root), root, quotient, mean and two products one each: under 24 half steps of fp32, plus
the output type's own.  A rotated value: the angle's fp32 fraction of a turn (pi 2^-24), sine and cosine (2
steps), two products and a sum: under 2^-20 (|a| + |b|)."""
import pytest
import torch

from tests import operator_refs as R
from tests.gpu_util import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL_Y = 24 * R.FP32
REL_ROT = 2.0 ** -20
EPS = 1e-6
U8, F32, BF, I32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


SHAPES = [(1, 1), (3, 7), (5, 8), (4, 64), (2, 255), (33, 256), (9, 257), (3, 1000), (6, 1024), (2, 1025), (700, 2048),
          (5, 4096), (3, 4104), (2, 8192), (2, 8193), (1, 16384), (3, 16383)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_rmsnorm(rows, cols, dtype):
    dsa, g = lib(), gen(rows * 131 + cols)
    x, res = normal(g, rows, cols, dtype=dtype), normal(g, rows, cols, dtype=dtype, std=3.0)
    for residual, wt, block, mode in ((res, dtype, 0, 0), (None, F32, 128, 0), (res, BF, 128, 1), (None, dtype, 0, 1)):
        w = normal(g, cols, std=0.3).add_(1).to(wt)
        h, out = torch.empty_like(x), torch.empty_like(x)
        n = -(-cols // 128) if block else 1
        codes, scale = torch.empty((rows, cols), dtype=U8, device=DEV), torch.empty((rows, n), device=DEV)
        dsa.dsa_rmsnorm(x, w, EPS, out=out, residual=residual, residual_out=h, codes=codes, scale=scale, block=block,
                        scale_mode=mode)
        rh, ry = R.rmsnorm(x, residual, w, EPS)
        R.check_close(h, rh, rh.abs() * (R.half_step(dtype) + R.FP32) + 1e-30, "h")
        R.check_close(out, ry, ry.abs() * (R.half_step(dtype) + REL_Y) + 1e-30, "out")
        for b in range(n):
            cut = slice(b * 128, (b + 1) * 128) if block else slice(None)
            R.check_fp8(codes[:, cut], scale[:, b], ry[:, cut], REL_Y, mode, f"block {b}")
        # parts alone give the same bytes, and codes agree with the quantiser on the fp32 output
        h2, out2, c2, s2 = torch.empty_like(h), torch.empty_like(out), torch.empty_like(codes), torch.empty_like(scale)
        dsa.dsa_rmsnorm(x, w, EPS, residual=residual, residual_out=h2)
        dsa.dsa_rmsnorm(x, w, EPS, residual=residual, out=out2)
        dsa.dsa_rmsnorm(x, w, EPS, residual=residual, codes=c2, scale=s2, block=block, scale_mode=mode)
        assert torch.equal(h, h2) and torch.equal(out, out2) and torch.equal(codes, c2) and torch.equal(scale, s2)
        if dtype == F32 and not block:
            qc, qs = torch.empty_like(codes), torch.empty(rows, device=DEV)
            dsa.dsa_quantize_fp8(out, qc, qs, mode)
            assert torch.equal(qc, codes) and torch.equal(qs, scale[:, 0])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols,off", [(512, 0), (512, 1), (1000, 8), (4096, 3), (130, 5)])
def test_rmsnorm_strided_misaligned_and_in_place(cols, off, dtype):
    """Rows inside a wider tensor, at any element offset, and outputs over their inputs: the bytes beside them stay,
    and every layout gives the values of the contiguous call."""
    dsa, g = lib(), gen(cols + off)
    rows, width = 9, cols + 40
    wide = normal(g, rows, width, dtype=dtype)
    x, res, w = wide[:, off:off + cols], normal(g, rows, cols, dtype=dtype), normal(g, cols).to(dtype)
    h0, o0 = torch.empty((rows, cols), dtype=dtype, device=DEV), torch.empty((rows, cols), dtype=dtype, device=DEV)
    dsa.dsa_rmsnorm(x.contiguous(), w, EPS, out=o0, residual=res, residual_out=h0)
    hw = torch.full((rows, width), 7.0, dtype=dtype, device=DEV)
    ow = hw.clone()
    dsa.dsa_rmsnorm(x, w, EPS, out=ow[:, off:off + cols], residual=res, residual_out=hw[:, off:off + cols])
    for wide_out, ref in ((hw, h0), (ow, o0)):
        want = torch.full_like(wide_out, 7.0)
        want[:, off:off + cols] = ref
        assert torch.equal(wide_out, want)
    r2, x2 = res.clone(), x.clone(memory_format=torch.contiguous_format)
    dsa.dsa_rmsnorm(x2, w, EPS, out=x2, residual=r2, residual_out=r2)  # both in place
    assert torch.equal(r2, h0) and torch.equal(x2, o0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rmsnorm_extreme_rows(dtype):
    dsa = lib()
    x = torch.zeros((4, 640), dtype=dtype, device=DEV)
    x[1], x[2, 5], x[3] = 1e-6, 3e4, torch.linspace(-2e4, 2e4, 640, device=DEV).to(dtype)
    w = torch.ones(640, dtype=dtype, device=DEV)
    out, codes, scale = torch.empty_like(x), torch.empty((4, 640), dtype=U8, device=DEV), torch.empty((4, 5), device=DEV)
    dsa.dsa_rmsnorm(x, w, EPS, out=out, codes=codes, scale=scale, block=128)
    _, ry = R.rmsnorm(x, None, w, EPS)
    R.check_close(out, ry, ry.abs() * (R.half_step(dtype) + REL_Y) + 1e-30, "out")
    assert (out[0] == 0).all() and (codes[0] == 0).all() and (scale[0] == 1).all()
    dsa.dsa_rmsnorm(torch.empty((0, 64), dtype=dtype, device=DEV), w[:64], EPS, out=torch.empty((0, 64), dtype=dtype, device=DEV))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", SHAPES + [(0, 96), (5000, 40), (1300, 1111)])
def test_rmsnorm_backward(rows, cols, dtype):
    """dx under 48 half steps of its terms' magnitudes (two reduced sums instead of one); dweight's chain is the
    rows of one CTA, then of one warp of the joining kernel, then 8."""
    dsa, g = lib(), gen(rows + 7 * cols)
    dy, h, dres = (normal(g, rows, cols, dtype=dtype, std=s) for s in (1.0, 2.0, 1.0))
    for extra, wt in ((None, dtype), (dres, F32)):
        w = normal(g, cols, std=0.3).add_(1).to(wt)
        dx, dw = torch.empty_like(h), torch.full((cols,), 7.0, device=DEV)
        dsa.dsa_rmsnorm_backward(dy, h, w, EPS, dx, dw, dres=extra)
        rx, rw, mag, wmag = R.rmsnorm_backward(dy, h, w, extra, EPS)
        R.check_close(dx, rx, rx.abs() * R.half_step(dtype) + 48 * R.FP32 * mag + 1e-30, "dx")
        R.check_close(dw, rw, (rows / 100 + 128) * R.FP32 * wmag + 1e-30, "dweight")
        dx2, dw2, hh = torch.empty_like(dx), torch.empty_like(dw), h.clone()
        ws = torch.full((max(1, dsa.dsa_rmsnorm_backward_workspace_size(rows, cols)),), 0xFF, dtype=U8, device=DEV)
        dsa.dsa_rmsnorm_backward(dy, hh, w, EPS, hh, dw2, dres=extra, workspace=ws)  # in place, dirty workspace
        assert torch.equal(hh, dx) and torch.equal(dw2, dw)


def test_rmsnorm_backward_against_differences():
    """Central differences of sum(dy * y + dres * h) in fp64 with a step of 1e-4: off by under 1e-6 of the terms."""
    dsa, g = lib(), gen(5)
    dy, h, dres, w = normal(g, 2, 48), normal(g, 2, 48), normal(g, 2, 48), normal(g, 48).add_(1)
    dx, dw = torch.empty_like(h), torch.empty(48, device=DEV)
    dsa.dsa_rmsnorm_backward(dy, h, w, EPS, dx, dw, dres=dres)

    def loss(hh, ww):
        return float((R.d(dy) * R.rmsnorm(hh, None, ww, EPS)[1]).sum() + (R.d(dres) * hh).sum())

    for arg, got in ((0, dx), (1, dw)):
        base = [R.d(h), R.d(w)]
        for i in range(base[arg].numel()):
            v = []
            for sign in (1, -1):
                t = [b.clone() for b in base]
                t[arg].view(-1)[i] += sign * 1e-4
                v.append(loss(*t))
            diff = (v[0] - v[1]) / 2e-4
            assert abs(float(got.view(-1)[i]) - diff) <= 2e-5 * (1 + abs(diff)), (arg, i)


def paged(g, lens, page, extra_pages=3):
    """Block table of sequences with room for ``lens`` tokens, pages shuffled, -1 where a sequence has none."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + extra_pages
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(3)).to(I32)
    bt = torch.full((len(lens), max(need)), -1, dtype=I32)
    at = 0
    for i, n in enumerate(need):
        bt[i, :n] = perm[at:at + n]
        at += n
    return bt, total


def pools(g, total, page):
    return (normal(g, total, page, 576, dtype=BF), torch.randint(0, 256, (total, page, 128), dtype=U8, generator=g, device=DEV),
            normal(g, total, page))


@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("kdtype,wtype,mode", [(BF, BF, 0), (F32, F32, 1), (BF, None, 0)])
def test_cache_append(page, kdtype, wtype, mode):
    dsa, g = lib(), gen(page)
    lens = [1, 33, page, page + 1, 200]
    bt, total = paged(g, lens, page)
    pos = torch.cat([torch.arange(n) for n in lens]).to(I32)
    seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).to(I32)
    order = torch.randperm(len(pos), generator=torch.Generator().manual_seed(1))  # tokens in any order
    pos, seq = pos[order], seq[order]
    pos[7] = -1  # padding inside the batch
    T, freq = len(pos), R.inv_freq()
    kvw = normal(g, T, 640, dtype=BF, std=2.0)
    kv = kvw[:, 64:]                                    # a slice of a fused projection
    kI = normal(g, T, 256, dtype=kdtype)[:, :128]
    kI[3] = 0                                           # a zero key: scale 1
    w = None if wtype is None else normal(g, 512, std=0.3).add_(1).to(wtype)
    kvp, k8p, ksp = pools(g, total, page)
    before = [t.clone() for t in (kvp, k8p, ksp)]
    dsa.dsa_get_device_status()
    dsa.dsa_cache_append(pos.to(DEV), bt.to(DEV), freq.to(DEV), kv=kv, kv_pool=kvp, kI=kI, k8_pool=k8p, ks_pool=ksp,
                         seq=seq.to(DEV), kv_weight=w, eps=EPS, scale_mode=mode)
    assert dsa.dsa_get_device_status() == 0
    live = pos >= 0
    slot = (bt[seq.long(), (pos.clamp(min=0) // page).long()].long() * page + pos.clamp(min=0).long() % page)[live]
    p, kvd, kId = pos[live], R.d(kv)[live], R.d(kI)[live]
    lat = kvd[:, :512] if w is None else R.rmsnorm(kvd[:, :512], None, w, EPS)[1]
    got = kvp.view(-1, 576)[slot.to(DEV)]
    if w is None:
        assert torch.equal(got[:, :512].cpu(), kv[live.to(DEV)][:, :512].cpu())
    else:
        R.check_close(got[:, :512], lat, lat.abs() * (R.BF16 + REL_Y) + 1e-30, "latent")
    rot = R.rotate_main(kvd[:, 512:], p, freq)
    mag = kvd[:, 512:].abs().view(-1, 32, 2).sum(-1).repeat_interleave(2, -1)
    R.check_close(got[:, 512:], rot, rot.abs() * R.BF16 + 2 * REL_ROT * mag + 1e-30, "rotated part")
    R.check_fp8(k8p.view(-1, 128)[slot.to(DEV)], ksp.view(-1)[slot.to(DEV)], R.rotate_index(kId, p, freq), 2 * REL_ROT, mode, "index")
    for t, b, width in zip((kvp, k8p, ksp), before, (576, 128, 1)):  # every other slot keeps its bytes
        keep = torch.ones(total * page, dtype=torch.bool)
        keep[slot] = False
        keep = keep.to(DEV)
        assert torch.equal(t.view(total * page, width)[keep], b.view(total * page, width)[keep])
    # one cache at a time, one token per table row: the same bytes
    kvp2, k8p2, ksp2 = (b.clone() for b in before)
    rows_bt = bt[seq.long()].contiguous().to(DEV)
    dsa.dsa_cache_append(pos.to(DEV), rows_bt, freq.to(DEV), kv=kv, kv_pool=kvp2, kv_weight=w, eps=EPS)
    dsa.dsa_cache_append(pos.to(DEV), rows_bt, freq.to(DEV), kI=kI, k8_pool=k8p2, ks_pool=ksp2, scale_mode=mode)
    assert torch.equal(kvp, kvp2) and torch.equal(k8p, k8p2) and torch.equal(ksp, ksp2)


def test_cache_append_bad_pages_and_positions():
    """Tokens whose page or position is out of range write nothing and raise their status bits; the others are written."""
    dsa, g = lib(), gen(9)
    page, freq = 64, R.inv_freq().to(DEV)
    kvp, k8p, ksp = pools(g, 4, page)
    bt = torch.tensor([[0, 4], [-1, 1], [2, 3]], dtype=I32, device=DEV)
    kv, kI = normal(g, 6, 576, dtype=BF), normal(g, 6, 128, dtype=BF)

    def call(pos, seq):
        before = [t.clone() for t in (kvp, k8p, ksp)]
        dsa.dsa_cache_append(torch.tensor(pos, dtype=I32, device=DEV), bt, freq, kv=kv[:len(pos)], kv_pool=kvp, kI=kI[:len(pos)],
                             k8_pool=k8p, ks_pool=ksp, seq=torch.tensor(seq, dtype=I32, device=DEV))
        changed = (kvp != before[0]).any(-1).view(-1).nonzero().flatten().tolist()
        return dsa.dsa_get_device_status(), changed

    dsa.dsa_get_device_status()
    assert call([64, 5], [0, 2]) == (4, [2 * page + 5])            # page 4 of a pool of 4
    assert call([3, 70], [1, 1]) == (4, [1 * page + 6])            # page -1
    assert call([128, 1], [2, 2]) == (2, [2 * page + 1])           # past the table
    assert call([2147483647, 2], [2, 2]) == (2, [2 * page + 2])
    assert call([0, 0, 3], [3, -1, 2]) == (2, [2 * page + 3])      # no such sequence
    assert call([-1, -2147483648, 4], [99, 0, 2]) == (0, [2 * page + 4])  # padding is no error, whatever its seq
    assert call([], []) == (0, [])


@pytest.mark.parametrize("base", [10000.0, 1e6])
def test_far_positions(base):
    """Angles stay exact at positions where fp32 products have lost them."""
    dsa, g = lib(), gen(11)
    freq = R.inv_freq(base)
    pos = torch.tensor([0, 1, 65535, 131071, 1000003, 16777217, 2147483647], dtype=I32)
    T = len(pos)
    q_rope, q = normal(g, T, 3, 64, dtype=BF), torch.zeros((T, 3, 576), dtype=BF, device=DEV)
    qI = normal(g, T, 2, 128)
    q8, qs = torch.empty((T, 2, 128), dtype=U8, device=DEV), torch.empty(T, device=DEV)
    dsa.dsa_rope_queries(pos.to(DEV), freq.to(DEV), q_rope=q_rope, q=q, qI=qI, q8=q8, q_scale=qs)
    # freq's own rounding is exact on both sides; the fixed-point step is off by 2^-53 turns a position,
    # the fp64 reference's product by 2^-53 of the angle: 2^31 positions make at most 2^-20
    ref = R.rotate_main(R.d(q_rope), pos, freq)
    mag = R.d(q_rope).abs().view(T, 3, 32, 2).sum(-1).repeat_interleave(2, -1)
    R.check_close(q[..., 512:], ref, ref.abs() * R.BF16 + 4 * REL_ROT * mag, "rotated")
    R.check_fp8(q8.view(T, -1), qs, R.rotate_index(R.d(qI), pos, freq).view(T, -1), 4 * REL_ROT, 0, "index")


@pytest.mark.parametrize("T,H,HI,idtype", [(1, 128, 64, BF), (5, 16, 32, F32), (64, 128, 64, F32), (3, 1, 1, BF), (7, 33, 63, BF)])
def test_rope_queries(T, H, HI, idtype):
    dsa, g = lib(), gen(T + H)
    freq, pos = R.inv_freq(), torch.randint(0, 131072, (T,), generator=torch.Generator().manual_seed(T)).to(I32)
    wide = normal(g, T, H, 192, dtype=BF)
    q = normal(g, T, H, 576, dtype=BF)
    nope, qI = q[..., :512].clone(), normal(g, T, HI, 128, dtype=idtype)
    for mode in (0, 1):
        q8, qs = torch.empty((T, HI, 128), dtype=U8, device=DEV), torch.empty(T, device=DEV)
        dsa.dsa_rope_queries(pos.to(DEV), freq.to(DEV), q_rope=wide[..., 128:], q=q, qI=qI, q8=q8, q_scale=qs, scale_mode=mode)
        ref = R.rotate_main(R.d(wide[..., 128:]), pos, freq)
        mag = R.d(wide[..., 128:]).abs().view(T, H, 32, 2).sum(-1).repeat_interleave(2, -1)
        R.check_close(q[..., 512:], ref, ref.abs() * R.BF16 + REL_ROT * mag + 1e-30, "q")
        assert torch.equal(q[..., :512], nope)
        R.check_fp8(q8.view(T, -1), qs, R.rotate_index(R.d(qI), pos, freq).view(T, -1), 2 * REL_ROT, mode, "q8")
    # heads before tokens, each part alone, and in place: the same bytes
    swapped = wide[..., 128:].transpose(0, 1).contiguous().transpose(0, 1)
    q2, q3 = q.clone(), q.clone()
    q2[..., 512:] = 0
    q3[..., 512:] = wide[..., 128:]
    dsa.dsa_rope_queries(pos.to(DEV), freq.to(DEV), q_rope=swapped, q=q2)
    dsa.dsa_rope_queries(pos.to(DEV), freq.to(DEV), q_rope=q3[..., 512:], q=q3)
    q82, qs2 = torch.empty_like(q8), torch.empty_like(qs)
    dsa.dsa_rope_queries(pos.to(DEV), freq.to(DEV), qI=qI, q8=q82, q_scale=qs2, scale_mode=1)
    assert torch.equal(q2, q) and torch.equal(q3, q) and torch.equal(q82, q8) and torch.equal(qs2, qs)


def test_rope_queries_padding():
    dsa, g = lib(), gen(2)
    pos = torch.tensor([4, -1, 6], dtype=I32, device=DEV)
    q, q8, qs = normal(g, 3, 4, 576, dtype=BF), torch.full((3, 8, 128), 9, dtype=U8, device=DEV), torch.full((3,), 7.0, device=DEV)
    before = q.clone()
    dsa.dsa_rope_queries(pos, R.inv_freq().to(DEV), q_rope=normal(g, 3, 4, 64, dtype=BF), q=q, qI=normal(g, 3, 8, 128), q8=q8, q_scale=qs)
    assert torch.equal(q[1], before[1]) and (q8[1] == 9).all() and qs[1] == 7
    assert not torch.equal(q[0], before[0]) and not torch.equal(q[2], before[2]) and qs[0] != 7 and qs[2] != 7


@pytest.mark.parametrize("T,HI", [(1, 1), (5, 64), (300, 1), (65, 3), (17, 32), (2, 63)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_index_rope_backward(T, HI, dtype):
    dsa, gn = lib(), gen(T * HI)
    freq, pos = R.inv_freq(), torch.randint(0, 131072, (T,), generator=torch.Generator().manual_seed(T)).to(I32)
    if T > 2:
        pos[2] = -1
    g = normal(gn, T, HI, 128)
    dx = torch.full((T, HI, 128), 7.0, dtype=dtype, device=DEV)
    dsa.dsa_index_rope_backward(g, pos.to(DEV), freq.to(DEV), dx)
    ref = R.rotate_index(R.d(g), -pos.long(), freq)
    ref[pos < 0] = 0
    mag = torch.cat([(R.d(g)[..., :32].abs() + R.d(g)[..., 32:64].abs()).repeat(1, 1, 2), torch.zeros(T, HI, 64, dtype=torch.float64)], -1)
    R.check_close(dx, ref, ref.abs() * R.half_step(dtype) + REL_ROT * mag, "dx")
    if HI == 1:
        dk = torch.empty((T, 128), dtype=dtype, device=DEV)
        dsa.dsa_index_rope_backward(g[:, 0], pos.to(DEV), freq.to(DEV), dk)
        assert torch.equal(dk, dx[:, 0])
    if dtype == F32:
        dsa.dsa_index_rope_backward(g, pos.to(DEV), freq.to(DEV), g)
        assert torch.equal(g, dx)


def test_index_rope_backward_against_differences():
    """d/dx of sum(g * rotated(x)), the rotation being linear: differences are exact in fp64 up to rounding."""
    dsa, gn = lib(), gen(21)
    freq, pos = R.inv_freq(), torch.tensor([12345], dtype=I32)
    g = normal(gn, 1, 1, 128)
    dx = torch.empty_like(g)
    dsa.dsa_index_rope_backward(g, pos.to(DEV), freq.to(DEV), dx)
    eye = torch.eye(128, dtype=torch.float64)[:, None]
    cols = R.rotate_index(eye, pos.expand(128), freq)
    diff = (cols * R.d(g)).sum((1, 2))
    assert (R.d(dx).view(-1) - diff).abs().max() <= 4 * REL_ROT * float(g.abs().max())


def test_streams_graphs_and_side_by_side_calls():
    """Every operator on a stream of its own, captured and replayed with changed inputs, and two backward calls at
    once with workspaces of their own."""
    dsa, g = lib(), gen(31)
    rows, cols = 64, 4096
    x, res, w = normal(g, rows, cols, dtype=BF), normal(g, rows, cols, dtype=BF), normal(g, cols).to(BF)
    h, out = torch.empty_like(x), torch.empty_like(x)
    codes, scale = torch.empty((rows, cols), dtype=U8, device=DEV), torch.empty((rows, 32), device=DEV)
    dx, dw = torch.empty_like(x), torch.empty(cols, device=DEV)
    ws = torch.empty(dsa.dsa_rmsnorm_backward_workspace_size(rows, cols), dtype=U8, device=DEV)
    freq, pos = R.inv_freq().to(DEV), torch.arange(rows, dtype=I32, device=DEV)
    bt = torch.arange(rows, dtype=I32, device=DEV).view(rows, 1)
    slot = pos % 64
    kvp, k8p, ksp = pools(g, rows, 64)
    kv, kI = normal(g, rows, 576, dtype=BF), normal(g, rows, 128, dtype=BF)
    q, q8, qs = normal(g, rows, 8, 576, dtype=BF), torch.empty((rows, 4, 128), dtype=U8, device=DEV), torch.empty(rows, device=DEV)
    qr, qI, gI = normal(g, rows, 8, 64, dtype=BF), normal(g, rows, 4, 128), normal(g, rows, 4, 128)
    dI = torch.empty_like(gI)

    def step(stream=None):
        dsa.dsa_rmsnorm(x, w, EPS, out=out, residual=res, residual_out=h, codes=codes, scale=scale, block=128, stream=stream)
        dsa.dsa_rmsnorm_backward(out, h, w, EPS, dx, dw, workspace=ws, stream=stream)
        dsa.dsa_cache_append(slot, bt, freq, kv=kv, kv_pool=kvp, kI=kI, k8_pool=k8p, ks_pool=ksp, stream=stream)
        dsa.dsa_rope_queries(pos, freq, q_rope=qr, q=q, qI=qI, q8=q8, q_scale=qs, stream=stream)
        dsa.dsa_index_rope_backward(gI, pos, freq, dI, stream=stream)

    outs = (h, out, codes, scale, dx, dw, kvp, k8p, ksp, q, q8, qs, dI)
    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for k in range(3):
        for t in (x, kv, kI, qr, qI, gI):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))
        step()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        if k == 1:  # the stream argument in place of a replay
            torch.cuda.synchronize()
            step(side)
            side.synchronize()
        else:
            graph.replay()
            torch.cuda.synchronize()
        for a, b, name in zip(outs, want, "h out codes scale dx dw kvp k8p ksp q q8 qs dI".split()):
            if name in ("kvp", "k8p", "ksp"):  # only the written slots come back
                at = (bt.view(-1).long(), slot.long())
                assert torch.equal(a[at], b[at]), name
            elif name == "q":
                assert torch.equal(a[..., 512:], b[..., 512:])
            else:
                assert torch.equal(a, b), name
    # two streams, no workspace given: each call has its own
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    big = [normal(g, 5000, 1024) for _ in range(4)]
    got = [(torch.empty_like(big[0]), torch.empty(1024, device=DEV)) for _ in range(2)]
    torch.cuda.synchronize()
    for s, (a, b), (o, v) in zip((s1, s2), ((big[0], big[1]), (big[2], big[3])), got):
        dsa.dsa_rmsnorm_backward(a, b, w[:1024].float().contiguous(), EPS, o, v, stream=s)
    torch.cuda.synchronize()
    for (a, b), (o, v) in zip(((big[0], big[1]), (big[2], big[3])), got):
        o2, v2 = torch.empty_like(o), torch.empty_like(v)
        dsa.dsa_rmsnorm_backward(a, b, w[:1024].float().contiguous(), EPS, o2, v2)
        assert torch.equal(o, o2) and torch.equal(v, v2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(5000, 40), (4999, 248), (6001, 256), (5003, 1000), (4900, 1024), (700, 1032), (613, 4096),
                                       (640, 6000), (609, 8192), (700, 8200), (650, 16384), (3001, 1001), (700, 4001), (5001, 129)])
def test_many_rows(rows, cols, dtype):
    """Enough rows for the ring of rows in shared memory, of every width class, with and without a tensor that keeps
    them out of it, against fp64 and against the same rows one at a time."""
    dsa, g = lib(), gen(rows + cols)
    x, res, w = normal(g, rows, cols, dtype=dtype), normal(g, rows, cols, dtype=dtype, std=2.0), normal(g, cols).to(dtype)
    h, out = torch.empty_like(x), torch.empty_like(x)
    codes, scale = torch.empty((rows, cols), dtype=U8, device=DEV), torch.empty((rows, -(-cols // 128)), device=DEV)
    dsa.dsa_rmsnorm(x, w, EPS, out=out, residual=res, residual_out=h, codes=codes, scale=scale, block=128)
    pick = sorted({0, 1, 7, 8, rows // 2, rows - 9, rows - 2, rows - 1})
    rh, ry = R.rmsnorm(x[pick], res[pick], w, EPS)
    R.check_close(h[pick], rh, rh.abs() * (R.half_step(dtype) + R.FP32) + 1e-30, "h")
    R.check_close(out[pick], ry, ry.abs() * (R.half_step(dtype) + REL_Y) + 1e-30, "out")
    for b in range(scale.shape[1]):
        cut = slice(b * 128, (b + 1) * 128)
        R.check_fp8(codes[pick][:, cut], scale[pick][:, b], ry[:, cut], REL_Y, 0, f"block {b}")
    row_codes, row_scale = torch.empty((rows, cols), dtype=U8, device=DEV), torch.empty(rows, device=DEV)
    out2 = torch.empty_like(out)
    dsa.dsa_rmsnorm(x, w, EPS, out=out2, codes=row_codes, scale=row_scale)  # no residual, a scale a row
    _, ry = R.rmsnorm(x[pick], None, w, EPS)
    R.check_close(out2[pick], ry, ry.abs() * (R.half_step(dtype) + REL_Y) + 1e-30, "out without residual")
    R.check_fp8(row_codes[pick], row_scale[pick], ry, REL_Y, 0, "row codes")
    r2, x2 = res.clone(), x.clone()
    dsa.dsa_rmsnorm(x2, w, EPS, out=x2, residual=r2, residual_out=r2)  # in place
    assert torch.equal(r2, h) and torch.equal(x2, out)
    # backward
    dy, dres = normal(g, rows, cols, dtype=dtype), normal(g, rows, cols, dtype=dtype)
    for extra in (None, dres):
        dx, dw = torch.empty_like(h), torch.empty(cols, device=DEV)
        dsa.dsa_rmsnorm_backward(dy, h, w, EPS, dx, dw, dres=extra)
        rx, rw, mag, wmag = R.rmsnorm_backward(dy, h, w, extra, EPS)
        R.check_close(dx, rx, rx.abs() * R.half_step(dtype) + 48 * R.FP32 * mag + 1e-30, "dx")
        R.check_close(dw, rw, (rows / 100 + 128) * R.FP32 * wmag + 1e-30, "dweight")
        hh, dw2 = h.clone(), torch.empty_like(dw)
        dsa.dsa_rmsnorm_backward(dy, hh, w, EPS, hh, dw2, dres=extra)
        assert torch.equal(hh, dx) and torch.equal(dw2, dw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [9, 24, 127, 129, 520, 1111, 2049, 8190])
def test_every_misalignment(cols, dtype):
    """Rows at every element offset from 16 bytes, in every tensor: the same values at each, and nothing beside them.
    Rows of whole chunks that all start at 16 bytes deal their columns to the threads otherwise and so sum them in
    another order: there the offsets are held to one another, and to fp64 with the bounds of any order."""
    dsa, g = lib(), gen(cols)
    rows = 3
    x, res, w = normal(g, rows, cols, dtype=dtype), normal(g, rows, cols, dtype=dtype), normal(g, cols).to(dtype)
    want = [torch.empty_like(x), torch.empty_like(x), torch.empty((rows, cols), dtype=U8, device=DEV), torch.empty(rows, device=DEV)]
    dsa.dsa_rmsnorm(x, w, EPS, out=want[0], residual=res, residual_out=want[1], codes=want[2], scale=want[3])
    step = 16 // x.element_size()  # offsets that leave every row at 16 bytes
    two_orders = cols % 8 == 0
    aligned = want
    rh, ry = R.rmsnorm(x, res, w, EPS)

    def shifted(t, off, fill=None):
        """A copy of t that begins `off` elements into a larger buffer, and that buffer."""
        buf = torch.full((t.numel() + 48,), 7, dtype=t.dtype, device=DEV)
        view = buf[off:off + t.numel()].view(t.shape)
        view.copy_(t if fill is None else torch.full_like(t, fill))
        return view, buf

    for off in range(16):
        (xs, _), (rs, _), (ws, _) = shifted(x, off), shifted(res, (off * 3) % 16), shifted(w, (off * 5) % 16)
        outs = [shifted(t, (off * k) % 16, fill=5) for t, k in zip(want, (7, 1, 9, 1))]
        (o, _), (h, _), (c, _), (s, _) = outs
        dsa.dsa_rmsnorm(xs, ws, EPS, out=o, residual=rs, residual_out=h, codes=c, scale=s)
        if two_orders and off == 1:
            assert torch.equal(h, want[1])  # no sum in it
            R.check_close(o, ry, ry.abs() * (R.half_step(dtype) + REL_Y) + 1e-30, "out")
            R.check_fp8(c, s, ry, REL_Y, 0, "codes")
            want = [t.clone() for t in (o, h, c, s)]
        # the codes' rows start at 8 bytes in the aligned form
        for (view, buf), ref, k in zip(outs, aligned if off % max(step, 8) == 0 else want, (7, 1, 9, 1)):
            at = (off * k) % 16
            assert torch.equal(view, ref)
            assert (buf[:at] == 7).all() and (buf[at + ref.numel():] == 7).all()
    dy, dw0, dx0 = normal(g, rows, cols, dtype=dtype), torch.empty(cols, device=DEV), torch.empty_like(x)
    dsa.dsa_rmsnorm_backward(dy, x, w, EPS, dx0, dw0, dres=res)
    dx1, dw1 = dx0, dw0
    for off in range(16):
        dx, buf = shifted(x, (off * 3) % 16, fill=5)
        dw = torch.empty_like(dw0)
        dsa.dsa_rmsnorm_backward(shifted(dy, off)[0], shifted(x, (off * 7) % 16)[0], shifted(w, (off * 5) % 16)[0], EPS, dx, dw,
                                 dres=shifted(res, (off * 9) % 16)[0])
        at = (off * 3) % 16
        if two_orders and off == 1:
            rx, rw, mag, wmag = R.rmsnorm_backward(dy, x, w, res, EPS)
            R.check_close(dx, rx, rx.abs() * R.half_step(dtype) + 48 * R.FP32 * mag + 1e-30, "dx")
            R.check_close(dw, rw, 128 * R.FP32 * wmag + 1e-30, "dweight")
            dx1, dw1 = dx.clone(), dw.clone()
        assert all(torch.equal(a, b) for a, b in zip((dx, dw), (dx0, dw0) if off % step == 0 else (dx1, dw1)))
        assert (buf[:at] == 7).all() and (buf[at + dx.numel():] == 7).all()


def test_quotients_are_those_of_a_division():
    """Codes of the norm's fp32 output against dsa_quantize_fp8, which divides: equal bytes over many magnitudes."""
    dsa, g = lib(), gen(77)
    for k, std in enumerate((1e-35, 1e-20, 1e-3, 1.0, 1e4, 1e18)):
        x = normal(g, 700, 4096)
        w = torch.full((4096,), std, device=DEV)
        out, codes, scale = torch.empty_like(x), torch.empty(x.shape, dtype=U8, device=DEV), torch.empty(700, device=DEV)
        dsa.dsa_rmsnorm(x, w, EPS, out=out, codes=codes, scale=scale, scale_mode=k & 1)
        qc, qs = torch.empty_like(codes), torch.empty_like(scale)
        dsa.dsa_quantize_fp8(out, qc, qs, k & 1)
        assert torch.equal(qc, codes) and torch.equal(qs, scale), std


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(4900, 300), (5003, 1001), (9800, 1033), (9800, 1040), (4900, 520), (4870, 2051), (4900, 2048),
                                       (2500, 4096), (2450, 4001), (700, 6001), (420, 8190), (330, 12001), (310, 16383)])
def test_rows_of_every_ring_shape(rows, cols, dtype):
    """As above, for the widths and counts at which the ring's CTAs change, whole chunks and rows at any address."""
    test_many_rows(rows, cols, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols,pad,off", [(4870, 300, 5, 1), (5003, 1001, 1, 3), (4870, 2049, 0, 7), (700, 6000, 3, 2), (700, 6001, 0, 5),
                                               (640, 4104, 24, 8), (330, 16000, 1, 0)])
def test_strided_rows_through_the_ring(rows, cols, pad, off, dtype):
    """Rows `pad` elements apart that begin `off` elements into their buffer, each tensor at another offset: what one
    call on contiguous rows gives, up to the order of its sums, with nothing written between the rows; in place too."""
    dsa, g = lib(), gen(rows + cols)
    ld = cols + pad

    def strided(t, shift, fill):
        buf = torch.full((rows * ld + 64,), fill, dtype=dtype, device=DEV)
        view = buf[off + shift:off + shift + rows * ld].view(rows, ld)[:, :cols]
        if t is not None:
            view.copy_(t)
        return view, buf

    x, res, w = normal(g, rows, cols, dtype=dtype), normal(g, rows, cols, dtype=dtype), normal(g, cols).to(dtype)
    (xs, _), (rs, rbuf) = strided(x, 0, 9.0), strided(res, 3, 9.0)
    (o, obuf), (h, hbuf) = strided(None, 1, 5.0), strided(None, 2, 5.0)
    codes, scale = torch.empty((rows, cols), dtype=U8, device=DEV), torch.empty((rows, -(-cols // 128)), device=DEV)
    dsa.dsa_rmsnorm(xs, w, EPS, out=o, residual=rs, residual_out=h, codes=codes, scale=scale, block=128)
    pick = sorted({0, 1, 7, 8, rows // 2, rows - 9, rows - 2, rows - 1})
    rh, ry = R.rmsnorm(x[pick], res[pick], w, EPS)
    R.check_close(h[pick], rh, rh.abs() * (R.half_step(dtype) + R.FP32) + 1e-30, "h")
    R.check_close(o[pick], ry, ry.abs() * (R.half_step(dtype) + REL_Y) + 1e-30, "out")
    for b in range(scale.shape[1]):
        cut = slice(b * 128, (b + 1) * 128)
        R.check_fp8(codes[pick][:, cut], scale[pick][:, b], ry[:, cut], REL_Y, 0, f"block {b}")
    for buf, shift in ((obuf, 1), (hbuf, 2)):
        rest = buf.clone()
        rest[off + shift:off + shift + rows * ld].view(rows, ld)[:, :cols] = 5.0
        assert (rest == 5.0).all()
    dsa.dsa_rmsnorm(xs, w, EPS, out=xs, residual=rs, residual_out=rs)
    assert torch.equal(xs, o) and torch.equal(rs, h)
    rest = rbuf.clone()
    rest[off + 3:off + 3 + rows * ld].view(rows, ld)[:, :cols] = 9.0
    assert (rest == 9.0).all()
