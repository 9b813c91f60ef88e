"""GPU tests of the 16-bit dense layers at the ends of their types' ranges, against plain
64-bit implementations: gradients near binary16's largest numbers, infinities and NaN in
every operand, and the digits that gradients keep whatever their size.

Tolerances are those of tests/test_gpu_dense.py, in units of u = 2^-24; what a test adds
to them is derived beside it.
"""
import math

import pytest

import quantized_expert_cache_gb300 as qec

torch = pytest.importorskip("torch")
from test_gpu_dense import (ACTS, BF16, F16, F32, U, backward, check_backward, close, close_norm,  # noqa: E402
                            forward, gen, layer, rand, slope_ref)

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


# ----------------------------------------------------------------- infinities, NaN
def same_class(got, ref, what):
    """Infinite where the definition is, of its sign; NaN where it is; finite elsewhere."""
    got = got.double()
    ok = torch.where(torch.isfinite(ref), torch.isfinite(got), (got == ref) | (torch.isnan(got) & torch.isnan(ref)))
    assert ok.all(), (what, int((~ok).sum()), got[~ok][:6], ref[~ok][:6])


def nonzero(v):
    return torch.where(v == 0, torch.ones_like(v), v)


@pytest.mark.parametrize("y", [F32, BF16])
@pytest.mark.parametrize("x", [F32, BF16])
@pytest.mark.parametrize("r,c", [(200, 264), (300, 4104)])
@pytest.mark.parametrize("t", [1, 3, 5, 40, 64, 65, 300])
def test_infinite_weights_and_rows(ctx, t, r, c, x, y):
    types = (x, BF16, y)
    s = layer(t, r, c, types, 50)
    s["x"], s["w"] = nonzero(s["x"]), nonzero(s["w"])
    s["x"][:, 2::3] = nonzero(s["x"][:, 2::3].to(BF16).to(x))  # (lower parts of zero)
    inf = float("inf")
    s["w"][3, 7], s["w"][5, 8], s["w"][6, 1] = inf, -inf, float("nan")
    s["w"][8, 2], s["w"][8, 3] = inf, -inf
    s["w"][r - 1, c - 1] = inf
    if t > 2:
        s["x"][1, 5], s["x"][2, 4] = inf, -inf
        s["w"][9, 4] = inf
    got, pre = forward(ctx, s, types, bias=True, pre=True)
    ref = torch.empty(t, r, dtype=torch.float64, device="cuda")
    for i in range(0, t, 25):  # (term by term: no product that the definition has not)
        ref[i:i + 25] = torch.stack([(s["x"][i:i + 25].double() * w.double()).sum(1) for w in s["w"]], 1)
    assert not torch.isfinite(ref).all()
    same_class(pre, ref, "pre")
    same_class(got, ref, "y")


@pytest.mark.parametrize("types,act", [((F32, BF16, F32), qec.ACT_NONE), ((F32, BF16, F32), qec.ACT_SILU),
                                       ((F32, BF16, BF16), qec.ACT_GELU), ((BF16, BF16, F32), qec.ACT_NONE),
                                       ((BF16, BF16, BF16), qec.ACT_SILU), ((BF16, BF16, BF16), qec.ACT_NONE),
                                       ((F16, F16, F16), qec.ACT_SILU)])
@pytest.mark.parametrize("t,r,c", [(3, 72, 136), (40, 72, 136), (300, 200, 72), (1030, 72, 136)])
def test_infinities_in_gradients(ctx, t, r, c, types, act):
    s = layer(t, r, c, types, 51)
    for k in ("x", "w", "dy"):
        s[k] = nonzero(s[k])
    s["pre"] = (s["pre"].abs() + 0.25).to(types[2])  # (slopes above 1/2)
    # (no dz below binary16's smallest step, whose first part would be zero)
    s["dy"] = torch.where(s["dy"].abs() < 1e-3, torch.ones_like(s["dy"]), s["dy"])
    s["dy"][:, ::4] = s["dy"][:, ::4].to(BF16).to(types[2])
    inf = float("inf")
    clean = {k: s[k].clone() for k in ("x", "w", "dy")}

    def run(plant):
        for k in clean:
            s[k] = clean[k].clone()
        for k, at, v in plant:
            s[k][at] = v
        dz = s["dy"].double() * (slope_ref(s["pre"], act) if act else 1.0)
        for dw_dtype in (F32, types[1]):
            dx, dw, db = backward(ctx, s, types, act, dw_dtype)
            x, w = s["x"].double(), s["w"].double()
            for i in range(0, t, 100):
                same_class(dx[i:i + 100], (dz[i:i + 100, :, None] * w[None]).sum(1), "dx")
            same_class(dw, torch.stack([(dz[:, j, None] * x).sum(0) for j in range(r)]), "dw")
            same_class(db, dz.sum(0), "db")

    run([("w", (2, 7), inf), ("w", (r - 1, 8), -inf), ("w", (5, 9), float("nan"))])
    run([("x", (1, 5), inf), ("x", (t - 1, c - 1), -inf)])
    run([("dy", (0, 4), inf), ("dy", (1, 3), -inf), ("dy", (2, 9), float("nan"))])
    run([("dy", (0, 4), inf), ("dy", (1, 4), -inf), ("w", (2, 7), inf), ("x", (2, 6), inf)])


# ---------------------------------------------------- the same digits at every size
@pytest.mark.parametrize("t,r,c", [(64, 256, 128), (1024, 2048, 2048)])
@pytest.mark.parametrize("types", [(BF16, BF16, F32), (F32, BF16, F32)])
def test_16_bit_gradients_of_fp32_ones_at_every_size(ctx, t, r, c, types):
    # differences of neighbouring gradients 1 + j 2^-15 (two bfloat16 numbers to the bit): j 2^-15,
    # j <= 127, is a bfloat16 number too, so the results are exact
    s = layer(t, r, c, types, 60)
    j = torch.randint(0, 128, (t, r), generator=gen(t, r), device="cuda")
    s["dy"] = 1 + j.float() * 2.0 ** -15
    s["w"][:], s["x"][:] = 0, 0
    s["w"][0], s["w"][1], s["x"][0], s["x"][1] = 1, -1, 1, -1
    dx, dw, _ = backward(ctx, s, types, qec.ACT_NONE, BF16)
    dy = s["dy"].double()
    assert torch.equal(dx.double(), (dy[:, 0] - dy[:, 1])[:, None].expand(t, c))
    assert torch.equal(dw.double(), (dy[0] - dy[1])[:, None].expand(r, c))


@pytest.mark.parametrize("t,r,c", [(64, 256, 128), (1024, 2048, 2048)])
@pytest.mark.parametrize("act", [qec.ACT_SILU, qec.ACT_GELU])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_16_bit_gradients_through_slopes_at_every_size(ctx, t, r, c, act, dtype):
    # differences of neighbouring slopes: two of 12 u (1 + |z|) and of the parts' 2^-22 (binary16)
    # or 2^-16 (bfloat16), |z| <= 1.5 and slopes below 1.13; the sum of two terms is exact to 3 u
    types = (dtype, dtype, dtype)
    s = layer(t, r, c, types, 61)
    s["dy"][:] = 1
    s["pre"] = 0.5 + torch.rand(t, r, generator=gen(t, r, 62), device="cuda").to(dtype)
    s["w"][:], s["x"][:] = 0, 0
    s["w"][0], s["w"][1], s["x"][0], s["x"][1] = 1, -1, 1, -1
    dx, dw, _ = backward(ctx, s, types, act, dtype)
    dz = slope_ref(s["pre"], act)
    tol = torch.tensor(2 * (30 * U + (2.0 ** -22 if dtype == F16 else 2.0 ** -16) * 1.13) + 3 * U, device="cuda")
    for got, ref in ((dx, (dz[:, 0] - dz[:, 1])[:, None].expand(t, c)), (dw, (dz[0] - dz[1])[:, None].expand(r, c))):
        close(got, ref, tol.double(), dtype)


# ------------------------------------------------------------- digits of fp32 gradients
@pytest.mark.parametrize("t,r,c", [(5, 8, 64), (64, 130, 264), (1030, 129, 640), (4096, 512, 2048)])
def test_fp32_gradients_keep_their_digits(ctx, t, r, c):
    # one weight: the rows' gradient is dy, all 24 bits of it; one row: the weights' is x times a
    # power of two, or dy times one
    types = (F32, BF16, F32)
    s = layer(t, r, c, types, 70)
    dy, x = s["dy"].clone(), s["x"].clone()
    s["w"][:] = 0
    s["w"][3, 11] = 1
    s["x"][:] = 0
    s["x"][4, 9] = 0.5
    dx, dw, _ = backward(ctx, s, types, qec.ACT_NONE, F32)
    assert torch.equal(dx[:, 11], dy[:, 3]) and not dx[:, :11].any() and not dx[:, 12:].any()
    assert torch.equal(dw[:, 9], dy[4] / 2) and not dw[:, :9].any() and not dw[:, 10:].any()
    s["x"], s["dy"] = x, torch.zeros_like(dy)
    s["dy"][4, 2] = -2
    _, dw, db = backward(ctx, s, types, qec.ACT_NONE, F32)
    assert torch.equal(dw[2], -2 * x[4]) and not dw[:2].any() and not dw[3:].any()
    assert float(db[2]) == -2 and not db[:2].any() and not db[3:].any()


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("t,r,c", [(40, 130, 264), (64, 512, 2048), (1030, 300, 640), (4096, 512, 2048)])
def test_fp32_gradients_of_rows_by_norms(ctx, t, r, c, act):
    # 42 u of the sums, at most 4 u of the additions between (r / 512 of half a step each); the
    # lower parts' sums are 2^-8 of the whole's and take 171 u / 2^8 twice; no pair is left out (a
    # weight is one part); slopes 12 u (1 + |z|), |z| of 1.5 in the mean
    types = (F32, BF16, F32)
    s = layer(t, r, c, types, 71)
    dx, _, _ = backward(ctx, s, types, act, F32, "x")
    dz = s["dy"].double() * (slope_ref(s["pre"], act) if act else 1.0)
    close_norm(dx, dz @ s["w"].double(), F32, "dx", 4 + 2 + (30 if act else 0))


@pytest.mark.parametrize("types", [(BF16, BF16, BF16), (F32, BF16, F32), (F16, F16, F16)])
@pytest.mark.parametrize("act", [qec.ACT_NONE, qec.ACT_GELU])
@pytest.mark.parametrize("t,r", [(1, 33), (200, 136), (2049, 40), (4100, 129), (20000, 64)])
def test_bias_gradients(ctx, t, r, act, types):
    # a warp's chain over every eighth token of a block, eight warps, the blocks in four chains and
    # two joins: additions on the longest way
    s = layer(t, r, 8, types, 72)
    _, _, db = backward(ctx, s, types, act, F32, "b")
    block = 16 if t <= 2048 else ((t + 127) // 128 + 7) // 8 * 8
    chain = block // 8 + 8 + ((t + block - 1) // block + 3) // 4 + 2
    dz = s["dy"].double() * (slope_ref(s["pre"], act) if act else 1.0)
    edz = 12 * U * (1 + s["pre"].double().abs()) * s["dy"].double().abs() if act else torch.zeros_like(dz)
    close(db, dz.sum(0), (chain + (1 if act else 0)) * U * dz.abs().sum(0) + edz.sum(0), F32)
