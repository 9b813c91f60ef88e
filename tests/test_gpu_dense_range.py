"""GPU tests of the 16-bit dense layers at the ends of their types' ranges, against plain
64-bit implementations: gradients near binary16's largest numbers.

Tolerances are those of tests/test_gpu_dense.py, in units of u = 2^-24; what a test adds
to them is derived beside it.
"""
import math

import pytest

import quantized_expert_cache_gb300 as qec

torch = pytest.importorskip("torch")
from test_gpu_dense import F16, F32, backward, check_backward, close_norm, gen, layer, rand, slope_ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = qec.moe_layer_init(64, 32, 8, 2, 1, 0, 1, stream=torch.cuda.current_stream().cuda_stream)
    yield c
    torch.cuda.synchronize()
    qec.moe_destroy(c)


# ------------------------------------------------------- large binary16 gradients
@pytest.mark.parametrize("act,peak", [(qec.ACT_SILU, 2.4), (qec.ACT_GELU, 1.414)])
@pytest.mark.parametrize("t,r,c", [(3, 9, 264), (70, 300, 264), (1000, 130, 520), (4100, 40, 128), (1030, 2048, 2056)])
def test_large_binary16_gradients(ctx, t, r, c, act, peak):
    # |dy| up to the largest number, at slopes above 1: dz passes 65504, its gradients do not
    types = (F16, F16, F16)
    s = layer(t, r, c, types, 40)
    g = gen(t, r, c, 41)
    size = 56000 + 9504 * torch.rand(t, r, generator=g, device="cuda")
    size[::3] = 65504
    s["dy"] = torch.where(torch.rand(t, r, generator=g, device="cuda") < 0.5, size, -size).half()
    s["pre"] = (peak + 0.2 * torch.randn(t, r, generator=g, device="cuda")).half()
    s["pre"][:, ::2] = peak
    dz = s["dy"].double() * slope_ref(s["pre"], act)
    assert float(dz.abs().max()) > 70000
    # (weights and rows small enough that the results are finite)
    s["w"] = rand(g, r, c, dtype=F16, scale=0.01 / math.sqrt(r))
    s["x"] = rand(g, t, c, dtype=F16, scale=0.01 / math.sqrt(t))
    for dw_dtype in (F32, F16):
        got = backward(ctx, s, types, act, dw_dtype)
        assert all(torch.isfinite(v).all() for v in got)
        check_backward(s, types, got, act, dw_dtype)
        if dw_dtype == F32 and t >= 64:
            # by norms: 42 u of the sums, 12 u (1 + |z|) of the slopes at |z| of 2.6, 2^-22 of the parts
            close_norm(got[1], dz.t() @ s["x"].double(), F32, "dw", 44 + 4)
