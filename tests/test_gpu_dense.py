"""GPU tests of moe_dense_forward and moe_dense_backward against plain 64-bit
implementations.

Tolerances, with u = 2^-24 (unit roundoff of binary32) and A = the sum of |products|
of a result:
- up to 2 tokens, or 4 on few weights: a lane's chain of at most K/32 + 8 fused steps and 5 joins:
  (K/32 + 16) u A.
- tensor cores: products of 16-bit operands are exact; for an fp32 result 32
  accumulations between two roundings, each off by at most a step of 2^-23 of what is
  summed, then K/512 + 8 additions rounded to nearest: (64 + K/512 + 8) u A for one
  pair of parts, K counting every pair's steps.  By norms (a partial sum of i of the 32
  terms has sqrt(i/32) of the whole's): 32 (2/3) 2^-23 = 42 u of the result's norm.  A
  16-bit result has 128 accumulations between two: 256 and 171 in place of 64 and 42.
- operands in parts, the layer: fp32 rows whole for an fp32 result (the pairs left out
  are below 3 2^-24 A), to 2^-16 for a 16-bit one (pairs left out: 3 2^-16 A, a parts'
  cut 2^-16).  Gradients likewise, of both operands (6 pairs; 7 2^-24 A for the pairs
  left out and 8 2^-16 A), a binary16 slope to 2^-22 or 2^-36, and a large 16-bit
  gradient's dz rounded to the type: a half step, by A (2^-25 at least in binary16).
- the epilogue: bias, activation and residual a few roundings (expf and erff 2 ulp):
  8 u of each term, |act'| <= 1.13; then half a step of the result's type.
- slopes: 12 u (1 + |z|) of dy.
- db: chains of T/8 + 32 additions: (T/8 + 40) u of the sum of |dz|.
"""
import math

import pytest

import quantized_expert_cache_gb300 as qec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
# (x, w, y)
TYPES = [(BF16, BF16, BF16), (BF16, BF16, F32), (F16, F16, F16), (F16, F16, F32), (F32, BF16, F32), (F32, BF16, BF16)]
ACTS = {qec.ACT_NONE: lambda z: z, qec.ACT_SILU: torch.nn.functional.silu, qec.ACT_GELU: torch.nn.functional.gelu}


@pytest.fixture(scope="module")
def ctx():
    c = qec.moe_layer_init(64, 32, 8, 2, 1, 0, 1, stream=torch.cuda.current_stream().cuda_stream)
    yield c
    torch.cuda.synchronize()
    qec.moe_destroy(c)


def gen(*key):
    return torch.Generator(device="cuda").manual_seed(sum(k * p for k, p in zip(key, (1, 10007, 1000003, 7919))) % (1 << 31))


def rand(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def layer(t, r, c, types, seed=0):
    g = gen(t, r, c, seed)
    x, w, y = types
    return dict(x=rand(g, t, c, dtype=x), w=rand(g, r, c, dtype=w, scale=1 / math.sqrt(c)), bias=rand(g, r),
                res=rand(g, t, r, dtype=y), dy=rand(g, t, r, dtype=y), pre=rand(g, t, r, dtype=y, scale=1.5))


def space(ctx, types, act, t, r, c, which):
    n = qec.moe_dense_workspace(ctx, *types, act, t, r, c)[which]
    # (filled with NaN: what a call reads there it has written)
    return torch.full((max(16, n + 15) // 16 * 8,), float("nan"), dtype=F16, device="cuda").view(torch.uint8)


def half_step(ref, dtype):
    tiny = dict(zip((F32, F16, BF16), (2.0 ** -149, 2.0 ** -24, 2.0 ** -133)))[dtype]
    return ref.abs() * torch.finfo(dtype).eps / 2 + tiny


def close(got, ref, tol, dtype, what=""):
    got = got.double()
    tol = tol + half_step(ref.abs() + tol, dtype)
    err = (got - ref).abs()
    ok = (err <= tol) | ((got == ref) & torch.isinf(ref)) | (torch.isnan(got) & torch.isnan(ref))
    assert ok.all(), (what, int((~ok).sum()), got[~ok][:4], ref[~ok][:4], tol.expand_as(ref)[~ok][:4])


def close_norm(got, ref, dtype, what="", extra=0):
    factor = (42 if dtype == F32 else 171) + extra
    # rounding of the result: at most half a step of each element
    bound = factor * U + (torch.finfo(dtype).eps / 2)
    err = float(torch.linalg.vector_norm(got.double() - ref) / torch.linalg.vector_norm(ref).clamp(min=1e-300))
    assert err <= bound, (what, err, bound)


def sums_tol(a, n_k, parts, few, f32_result):
    """Bound of a product whose absolute sums are a, over n_k of k, in `parts` pairs."""
    if few:
        return (n_k / 32 + 16) * U * a
    tol = ((72 if f32_result else 264) + parts * n_k / 512) * U * a
    if parts > 1:
        tol = tol + (3 * 2.0 ** -24 if f32_result else 4 * 2.0 ** -16) * a
    return tol


def forward(ctx, s, types, act=qec.ACT_NONE, bias=False, res=False, pre=False, stream=None, extra=0):
    t, c = s["x"].shape
    r = s["w"].shape[0]
    y = torch.full((t + extra, r), 7.0, dtype=types[2], device="cuda")
    z = torch.full((t + extra, r), 7.0, dtype=types[2], device="cuda") if pre else None
    qec.moe_dense_forward(ctx, s["x"], s["w"], t, r, c, y, bias=s["bias"] if bias else None, act=act,
                          res=s["res"] if res else None, pre=z, ws=space(ctx, types, act, t, r, c, 0), stream=stream)
    return y, z


def check_forward(s, types, got, act=qec.ACT_NONE, bias=False, res=False, norm=True):
    y, z = got
    x, w = s["x"].double(), s["w"].double()
    t, c = x.shape
    a = x.abs() @ w.abs().t()
    ref = x @ w.t()
    few = t <= 2 or (t <= 4 and s["w"].numel() <= 1 << 22)
    tol = sums_tol(a, c, 1 if types[0] != F32 else 3, few, types[2] == F32)
    if norm and act == qec.ACT_NONE and not bias and not res:
        if not few and c >= 64:
            close_norm(y[:t], ref, types[2], "norm", 0 if types[2] == F32 or types[0] != F32 else 2.0 ** 8 * 3)
    if bias:
        ref = ref + s["bias"].double()
        tol = tol + U * ref.abs()
    if z is not None:
        close(z[:t], ref, tol, types[2], "pre")
    out = ACTS[act](ref)
    tol = 1.13 * tol + (0 if act == qec.ACT_NONE else 8 * U * ref.abs())
    if res:
        out = out + s["res"].double()
        tol = tol + U * (out.abs() + s["res"].double().abs())
    close(y[:t], out, tol, types[2], "y")


# ------------------------------------------------------------------- forward
SHAPES = [(1, 1, 8), (1, 8, 2048), (2, 7, 16), (3, 130, 520), (4, 513, 2880), (4, 5000, 264), (5, 1, 8), (5, 8, 64),
          (6, 9, 72), (7, 127, 512), (8, 128, 2048), (16, 129, 520), (31, 257, 1024), (32, 512, 2048), (33, 2887, 2880),
          (64, 300, 4104), (65, 96, 200), (127, 640, 136), (128, 1000, 1032), (129, 31, 4096), (200, 2880, 328),
          (257, 513, 264), (300, 4096, 512), (1000, 130, 2048), (1, 40, 8192), (2, 1216, 1024), (2, 9000, 136), (3, 4096, 1032),
          (4, 1500, 2048), (63, 1000, 520), (64, 4000, 72), (2100, 1030, 96), (4096, 8, 64)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("t,r,c", SHAPES)
def test_products(ctx, t, r, c, types):
    s = layer(t, r, c, types)
    check_forward(s, types, forward(ctx, s, types))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("bias,res,pre", [(True, False, True), (False, True, False), (True, True, True)])
@pytest.mark.parametrize("t,r,c", [(1, 513, 264), (3, 130, 520), (40, 130, 2048), (600, 1500, 264)])
def test_epilogues(ctx, t, r, c, bias, res, pre, act, types):
    s = layer(t, r, c, types, 1)
    check_forward(s, types, forward(ctx, s, types, act, bias, res, pre), act, bias, res)


def test_residual_in_place_and_rows_behind(ctx):
    types = (BF16, BF16, BF16)
    for t in (3, 50):
        s = layer(t, 130, 136, types, 2)
        want, _ = forward(ctx, s, types, res=True)
        got, z = forward(ctx, s, types, res=True, pre=True, extra=3)
        assert torch.equal(got[:t], want) and (got[t:] == 7).all() and (z[t:] == 7).all()
        y = s["res"].clone()
        qec.moe_dense_forward(ctx, s["x"], s["w"], t, 130, 136, y, res=y)
        assert torch.equal(y, want)


@pytest.mark.parametrize("t", [2, 40, 400])
def test_infinite_nan_and_extreme_values(ctx, t):
    types = (F32, BF16, F32)
    s = layer(t, 200, 264, types, 3)
    s["x"][0, 5] = float("inf")
    s["x"][1, 7] = float("nan")
    s["w"][:, 5] = s["w"][:, 5].abs() + 0.01
    y, _ = forward(ctx, s, types)
    assert (y[0] == float("inf")).all() and torch.isnan(y[1]).all() and torch.isfinite(y[2:]).all()
    # the largest values, which round past bfloat16's range, and small ones
    s = layer(t, 200, 264, types, 4)
    s["w"][:] = 0
    s["w"][:, 0] = 1
    s["x"][0] = 0
    s["x"][0, 0] = torch.finfo(F32).max
    s["x"][1, 0] = 1.2345678e-30
    y, _ = forward(ctx, s, types)
    assert (y[0] == torch.finfo(F32).max).all()
    assert ((y[1].double() - float(s["x"][1, 0])).abs() <= 4 * U * float(s["x"][1, 0])).all()


def test_fp32_rows_keep_their_digits(ctx):
    # one column: the result is the row's value, all 24 bits of it
    types = (F32, BF16, F32)
    s = layer(64, 8, 64, types, 5)
    s["w"][:] = 0
    s["w"][3, 11] = 1
    y, _ = forward(ctx, s, types)
    assert torch.equal(y[:, 3], s["x"][:, 11])


# ------------------------------------------------------------------ gradients
BACK = [(BF16, BF16, BF16), (F16, F16, F16), (F32, BF16, F32), (F32, BF16, BF16), (BF16, BF16, F32)]


def backward(ctx, s, types, act, dw_dtype, want="xwb", stream=None, dy=None):
    t, c = s["x"].shape
    r = s["w"].shape[0]
    dx = torch.full((t, c), 7.0, dtype=types[0], device="cuda") if "x" in want else None
    dw = torch.full((r, c), 7.0, dtype=dw_dtype, device="cuda") if "w" in want else None
    db = torch.full((r,), 7.0, device="cuda") if "b" in want else None
    qec.moe_dense_backward(ctx, s["x"], s["w"], s["dy"] if dy is None else dy, t, r, c, dx, dw, db, act=act,
                           pre=s["pre"] if act else None, ws=space(ctx, types, act, t, r, c, 1), stream=stream)
    return dx, dw, db


def slope_ref(z, act):
    z = z.double().requires_grad_()
    return torch.autograd.grad(ACTS[act](z).sum(), z)[0]


def check_backward(s, types, got, act, dw_dtype):
    dx, dw, db = got
    x, w, dz = s["x"].double(), s["w"].double(), s["dy"].double()
    t, c = x.shape
    r = w.shape[0]
    edz = torch.zeros_like(dz)
    if act:
        z = s["pre"].double()
        edz = 12 * U * (1 + z.abs()) * dz.abs()
        dz = dz * slope_ref(s["pre"], act)
        if types[1] == F16:
            large = s["dy"].numel() * c >= 1 << 32
            edz = edz + dz.abs() * 2.0 ** -22 + (2.0 ** -25 if large else 2.0 ** -36)
    def product(a, n_k, dtype, parts, spread):
        tol = sums_tol(a, n_k, 1, False, dtype == F32) + spread
        if parts > 1:
            tol = tol + a * (7 * 2.0 ** -24 + 6 * n_k / 512 * U if dtype == F32 else 8 * 2.0 ** -16)
            if dtype != F32 and t * r * c >= 1 << 32:
                tol = tol + a * torch.finfo(dtype).eps / 2
        return tol

    z_parts = 3 if types[2] == F32 or act else 1
    if dx is not None:
        close(dx, dz @ w, product(dz.abs() @ w.abs(), r, types[0], z_parts, edz @ w.abs()), types[0], "dx")
    if dw is not None:
        parts = max(z_parts, 3 if types[0] == F32 else 1)
        ref = dz.t() @ x
        close(dw, ref, product(dz.abs().t() @ x.abs(), t, dw_dtype, parts, edz.t() @ x.abs()), dw_dtype, "dw")
        if dw_dtype == F32 and types[1] == BF16 and not act and t >= 64:
            close_norm(dw, ref, dw_dtype, "dw")
    if db is not None:
        close(db, dz.sum(0), (t / 8 + 40) * U * dz.abs().sum(0) + edz.sum(0), F32, "db")


@pytest.mark.parametrize("types", BACK)
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("t,r,c", [(1, 1, 8), (1, 130, 264), (3, 8, 64), (5, 513, 72), (33, 7, 520), (64, 64, 64),
                                   (65, 130, 2048), (127, 128, 136), (200, 520, 264), (500, 1000, 96), (1030, 129, 640),
                                   (1000, 33, 8), (4100, 40, 128),
                                   (2050, 1100, 2048)])
def test_gradients(ctx, t, r, c, act, types):
    s = layer(t, r, c, types, 6)
    for dw_dtype in (F32, types[1]):
        check_backward(s, types, backward(ctx, s, types, act, dw_dtype), act, dw_dtype)


@pytest.mark.parametrize("types", BACK)
def test_gradients_one_by_one(ctx, types):
    s = layer(70, 137, 136, types, 7)
    for act in (qec.ACT_NONE, qec.ACT_SILU):
        want = backward(ctx, s, types, act, F32)
        for w in ("x", "w", "b", "xb", "wb"):
            got = backward(ctx, s, types, act, F32, w)
            # (the products' order of summation goes by both: their bits may differ)
            if got[2] is not None:
                assert torch.equal(got[2], want[2])
            check_backward(s, types, got, act, F32)
    # operands that a gradient does not read
    t, r, c = 70, 137, 136
    xd, wd = (dict(zip((F32, F16, BF16), (0, 1, 2)))[d] for d in types[:2])
    ws = space(ctx, types, 0, t, r, c, 1)
    dx, dw = torch.empty(t, c, dtype=types[0], device="cuda"), torch.empty(r, c, device="cuda")
    qec.moe_dense_backward(ctx, None, s["w"], s["dy"], t, r, c, dx=dx, ws=ws, x_dtype=xd)
    qec.moe_dense_backward(ctx, s["x"], None, s["dy"], t, r, c, dw=dw, ws=ws, w_dtype=wd)
    check_backward(s, types, (dx, dw, None), qec.ACT_NONE, F32)


def test_gradients_without_tokens(ctx):
    dw, db = torch.full((9, 16), 7.0, device="cuda"), torch.full((9,), 7.0, device="cuda")
    qec.moe_dense_backward(ctx, None, None, None, 0, 9, 16, None, dw, db, x_dtype=2, w_dtype=2, y_dtype=2)
    assert (dw == 0).all() and (db == 0).all()
    qec.moe_dense_forward(ctx, None, None, 0, 9, 16, None, x_dtype=2, w_dtype=2, y_dtype=2)


def test_gradients_off_the_boundary(ctx):
    # dy and pre at addresses of their elements only
    types = (BF16, BF16, BF16)
    s = layer(40, 128, 64, types, 8)
    for name in ("dy", "pre"):
        flat = torch.empty(40 * 128 + 3, dtype=BF16, device="cuda")
        flat[3:].copy_(s[name].reshape(-1))
        s[name] = flat[3:].view(40, 128)
    for act in ACTS:
        check_backward(s, types, backward(ctx, s, types, act, F32), act, F32)


@pytest.mark.parametrize("t,r,c", [(3, 9, 2112), (70, 300, 264), (1000, 130, 520)])
def test_small_binary16_gradients_keep_their_digits(ctx, t, r, c):
    # dy far below 1, as without a loss scale: the second part of dz must not sink
    types = (F16, F16, F16)
    s = layer(t, r, c, types, 30)
    s["dy"] = (s["dy"].float() * 1e-3).half()
    for act in (qec.ACT_SILU, qec.ACT_GELU):
        got = backward(ctx, s, types, act, F32)
        check_backward(s, types, got, act, F32)
        dz = s["dy"].double() * slope_ref(s["pre"], act)
        # by norms: 42 u of the sums, 12 u (1 + |z|) of the slopes at |z| of 1.5, 2^-22 of the parts
        close_norm(got[1], dz.t() @ s["x"].double(), F32, "dw", 30 + 4)


def test_gradients_against_differences(ctx):
    # f = sum(act(x W^T + b) * dy) along directions of x, W and b: central differences in 64 bits, whose
    # error is below 1e-7 of the absolute parts at h = 1e-4
    types = (F32, BF16, F32)
    t, r, c = 40, 72, 136
    s = layer(t, r, c, types, 9)
    for act in ACTS:
        y, pre = forward(ctx, s, types, act, bias=True, pre=True)
        s["pre"] = pre
        dx, dw, db = (v.double() for v in backward(ctx, s, types, act, F32))
        base = [s["x"].double(), s["w"].double(), s["bias"].double()]

        def f(x, w, b):
            return (ACTS[act](x @ w.t() + b) * s["dy"].double()).sum()

        for i, d in enumerate((dx, dw, db)):
            v = rand(gen(i, act), *d.shape).double()
            h = 1e-4
            up, down = list(base), list(base)
            up[i], down[i] = base[i] + h * v, base[i] - h * v
            slope = float((f(*up) - f(*down)) / (2 * h))
            # fp32 gradients of fp32-rounded sums: 200 u of the absolute parts
            assert abs(slope - float((d * v).sum())) <= 1.3e-5 * float((d.abs() * v.abs()).sum())


# ------------------------------------------------------- streams, graphs, sizes
@pytest.mark.parametrize("t", [2, 77])
def test_other_streams_graphs_and_the_same_bits(ctx, t):
    types, act = (F32, BF16, F32), qec.ACT_SILU
    r, c = 300, 520
    a, b = layer(t, r, c, types, 10), layer(t, r, c, types, 11)
    b["w"] = a["w"]

    def both(s, stream=None):
        y, pre = forward(ctx, s, types, act, True, True, True, stream)
        s = dict(s, pre=pre)
        return (y, pre) + backward(ctx, s, types, act, F32, stream=stream)

    want = [both(a), both(b)]
    torch.cuda.synchronize()
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(both(a), want[0]))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = both(a, st)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want[0]))
    hold = {k: v.clone() for k, v in a.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            out = both(hold, st)
    for s, w in ((a, want[0]), (b, want[1]), (a, want[0])):
        for k in hold:
            hold[k].copy_(s[k])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, w))


def test_results_of_more_than_2_31_elements(ctx):
    types = (BF16, BF16, BF16)
    t, r, c = 40000, 65536, 64
    g = gen(12)
    x, w = rand(g, t, c, dtype=BF16), rand(g, r, c, dtype=BF16, scale=0.1)
    y = torch.empty(t, r, dtype=BF16, device="cuda")
    qec.moe_dense_forward(ctx, x, w, t, r, c, y)
    rows = [0, 1, 32767, 32768, t - 1]
    ref = x[rows].double() @ w.double().t()
    a = x[rows].double().abs() @ w.double().abs().t()
    close(y[rows], ref, sums_tol(a, c, 1, False, False), BF16)
    dx = torch.empty_like(x)
    ws = space(ctx, types, 0, t, r, c, 1)
    qec.moe_dense_backward(ctx, None, w, y, t, r, c, dx=dx, ws=ws, x_dtype=qec.BF16)
    dz = y[rows].double()
    close(dx[rows], dz @ w.double(), sums_tol(dz.abs() @ w.double().abs(), r, 1, False, False), BF16)


def test_no_wait_expired(ctx):
    qec.miss_drain(ctx)


def test_refusals(ctx):
    x, w, y = (torch.empty(s, dtype=BF16, device="cuda") for s in ((5, 16), (9, 16), (5, 9)))
    with pytest.raises(ValueError):
        qec.moe_dense_forward(ctx, x, w, 5, 9, 16, y, bias=torch.empty(9, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError):
        qec.moe_dense_forward(ctx, x, w, 5, 9, 16, y, res=torch.empty(5, 9, device="cuda"))
    for bad in (dict(w=w.float()), dict(w=w.half()), dict(x=x.half()), dict(y=y.half())):
        a = dict(dict(x=x, w=w, y=y), **bad)
        with pytest.raises(qec.MoeError):
            qec.moe_dense_forward(ctx, a["x"], a["w"], 5, 9, 16, a["y"])
    with pytest.raises(qec.MoeError):
        qec.moe_dense_forward(ctx, x, w, 5, 9, 12, y)
    with pytest.raises(qec.MoeError, match="workspace"):
        qec.moe_dense_forward(ctx, x.float(), w, 5, 9, 16, y)
    with pytest.raises(qec.MoeError, match="workspace"):
        qec.moe_dense_backward(ctx, x, w, y, 5, 9, 16, x.clone())
    with pytest.raises(qec.MoeError):
        qec.moe_dense_forward(ctx, x, w, 5, 9, 16, y, act=3)


def test_two_streams_at_once(ctx):
    # calls in flight together, each with its own workspace: split tiles, pairs and parts
    types = (F32, BF16, F32)
    shapes = [(70, 700, 1032), (300, 520, 2048)]
    layers = [layer(t, r, c, types, 20 + i) for i, (t, r, c) in enumerate(shapes)]

    def run(s, stream):
        t, c = s["x"].shape
        r = s["w"].shape[0]
        y, dx, dw, db = (torch.empty(n, device="cuda") for n in ((t, r), (t, c), (r, c), (r,)))
        ws = [space(ctx, types, qec.ACT_NONE, t, r, c, i) for i in (0, 1)]

        def go():
            qec.moe_dense_forward(ctx, s["x"], s["w"], t, r, c, y, ws=ws[0], stream=stream)
            qec.moe_dense_backward(ctx, s["x"], s["w"], s["dy"], t, r, c, dx, dw, db, ws=ws[1], stream=stream)
        return go, (y, dx, dw, db)

    streams = [torch.cuda.Stream() for _ in layers]
    calls = [run(s, st) for s, st in zip(layers, streams)]
    torch.cuda.synchronize()
    want = []
    for go, out in calls:
        go()
        torch.cuda.synchronize()
        want.append([o.clone() for o in out])
    for _ in range(20):
        for _, out in calls:
            for o in out:
                o.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for go, _ in calls:
                go()
        torch.cuda.synchronize()
        for (_, out), w in zip(calls, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w))
    qec.miss_drain(ctx)
