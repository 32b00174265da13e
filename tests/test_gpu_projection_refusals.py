"""What the calls of the FP8 product, block quantisation and layer norm say of an argument that is wrong, and sizes that
32 bits do not hold."""
import pytest
import torch

from tests.gpu_util import lib
from tests.test_gpu_projection_calls import DEV, F32, NAMES, U8, calls

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", NAMES)
def test_every_refusal_names_the_argument(name):
    dsa = lib()
    kw, outs = calls()[name]
    for arg, t in kw.items():
        if not isinstance(t, torch.Tensor):
            continue
        wrong = {"host": t.cpu(), "dtype": t.to(torch.float16), "object": t.tolist(), "shape": t.unsqueeze(0).contiguous(),
                 "longer": torch.cat([t, t], -1).contiguous()}
        for kind, w in wrong.items():
            if kind == "longer" and arg in ("x", "h", "a", "b"):
                continue  # the others are measured against it
            with pytest.raises((TypeError, ValueError)) as e:
                getattr(dsa, name)(**{**kw, arg: w})
            assert str(e.value).split(":")[0].split()[0] == arg, (arg, kind, str(e.value))
    torch.cuda.synchronize()
    assert all((t == 0).all() for t in outs)  # nothing was launched


def test_a_sum_over_more_columns_than_the_library_counts_is_refused():
    """Cut to 32 bits, these would be 256 columns."""
    dsa = lib()
    n = (1 << 32) + 256
    codes = torch.zeros((1, n), dtype=U8, device=DEV)
    scale, out = torch.ones((1, n // 128), device=DEV), torch.full((1, 1), 5.0, device=DEV)
    with pytest.raises(dsa.DsaError, match=str(n)):
        dsa.dsa_gemm_fp8(codes, scale, codes, scale, out)
    torch.cuda.synchronize()
    assert out.item() == 5.0
    del codes
    x, w = torch.zeros((1, n), dtype=torch.bfloat16, device=DEV), torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    for f, args in ((dsa.dsa_layernorm, (x, w, None, 1e-6)), (dsa.dsa_rmsnorm, (x, w, 1e-6))):
        with pytest.raises(dsa.DsaError, match=str(n)):
            f(*args, out=x)
    assert dsa.dsa_get_device_status() == 0
