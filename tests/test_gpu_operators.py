"""GPU tests of the operators around the routed experts (moe_rms_norm,
moe_linear_forward, moe_router_loss) against plain 64-bit implementations.

Tolerances, with u = 2^-24 (unit roundoff of binary32):
- norm: the sum of squares is a tree of at most 32 + 32 + 10 additions a chain,
  its relative error halves in the square root; the rest is 6 roundings:
  |y - ref| <= (40 + 6) u |ref|, and for the 16-bit sums and the codes the bits
  of a restatement (codes of the y that was written).
- linear: operands exact to 2^-22 and at most 6 accumulations a block of 32
  columns, rounded or truncated (2^-23 each) against the sum of |products|:
  |err| <= (6 nb + 16) 2^-23 sum |w x|; and, the accumulations between two
  roundings to fp32 being at most 64: norm(err) <= 5e-6 norm(ref).
- router: p = exp(z - top) / sum errs by (|z - top| + E/32 + 24) u, every other
  step by a few u: |dz - ref| <= (max|z - top| + E/32 + 64) u (the terms'
  absolute sum); losses likewise, relative.
"""
import numpy as np
import pytest

import quantized_expert_cache_gb300 as qec
import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ctxs():
    made = {}

    def get(max_tokens=64, experts=8, k=2, renorm=1):
        key = (max_tokens, experts, k, renorm)
        if key not in made:
            made[key] = qec.moe_layer_init(64, 32, experts, k, 1, 0, max_tokens, renorm_topk=renorm,
                                           stream=torch.cuda.current_stream().cuda_stream)
        return made[key]

    yield get
    torch.cuda.synchronize()
    for c in made.values():
        qec.moe_destroy(c)


def quantize32(y):
    """Codes and scales of fp32 rows, steps in binary32 (numpy)."""
    b = y.reshape(-1, 32)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        d = (np.abs(b).max(1) / np.float32(127)).astype(np.float16)
        f = d.astype(np.float32)[:, None]
        q = np.where(f > 0, np.clip(np.rint(b / np.where(f > 0, f, 1)), -127, 127), 0)
    return q.astype(np.int8).reshape(y.shape), d.reshape(y.shape[0], -1)


# ------------------------------------------------------------------- norm
def norm_ref(x, res, w, eps):
    s = x.double() + (res.double() if res is not None else 0)
    return s / torch.sqrt((s * s).mean(1, keepdim=True) + eps) * w.double()


def run_norm(ctx, x, res, w, codes=True, eps=1e-5, with_sum=True, with_y=True, stream=None):
    t, n = x.shape
    out_sum = torch.full_like(x, 7) if with_sum else None
    y = torch.full((t, n), 7.0, device="cuda") if with_y else None
    q = torch.full((t, n), 7, dtype=torch.int8, device="cuda") if codes else None
    d = torch.full((t, max(1, n // 32)), 7.0, dtype=torch.float16, device="cuda") if codes else None
    qec.moe_rms_norm(ctx, x, res, w, t, n, eps, out_sum, y, q, d, stream=stream)
    return out_sum, y, q, d


def check_norm(x, res, w, got, eps=1e-5):
    out_sum, y, q, d = got
    s32 = x.float() + (res.float() if res is not None else 0)
    if out_sum is not None:
        assert torch.equal(out_sum, s32.to(x.dtype))
    ref = norm_ref(x, res, w, eps)
    if y is not None:
        err = (y.double() - ref).abs()
        assert (err <= 46 * U * ref.abs() + 1e-38).all(), float((err / ref.abs().clamp(min=1e-30)).max() / U)
    if q is not None and y is not None:
        q0, d0 = quantize32(y.cpu().numpy())
        assert np.array_equal(q.cpu().numpy(), q0)
        assert np.array_equal(d.cpu().numpy().view(np.uint16), d0.view(np.uint16))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,width,codes", [
    (1, 2048, True), (3, 2880, True), (33, 256, True), (9, 32, True), (5, 96, True), (2, 4128, True), (2, 8192, True),
    (1, 16384, True), (2, 40000, True), (7, 1, False), (5, 17, False), (3, 1001, False), (2, 2047, False),
    (2, 4099, False), (1, 33333, False), (1000, 160, True), (300, 2048, True)])
def test_norm_shapes(ctxs, tokens, width, codes, dtype):
    g = torch.Generator(device="cuda").manual_seed(tokens * 10007 + width)
    x = torch.randn(tokens, width, generator=g, device="cuda").to(dtype)
    res = (3 * torch.randn(tokens, width, generator=g, device="cuda")).to(dtype)
    w = 1 + 0.3 * torch.randn(width, generator=g, device="cuda")
    check_norm(x, res, w, run_norm(ctxs(), x, res, w, codes))
    check_norm(x, None, w, run_norm(ctxs(), x, None, w, codes, with_sum=False))


def test_norm_no_tokens_and_single_outputs(ctxs):
    ctx = ctxs()
    w = torch.ones(64, device="cuda")
    qec.moe_rms_norm(ctx, None, None, None, 0, 64, 1e-5, None, None)
    x = torch.randn(4, 64, device="cuda")
    for kw in (dict(with_y=False), dict(codes=False), dict(with_sum=False)):
        check_norm(x, x, w, run_norm(ctx, x, x, w, **kw))
    _, _, q, d = run_norm(ctx, x, x, w, with_y=False, with_sum=False)
    _, y, _, _ = run_norm(ctx, x, x, w)
    q0, d0 = quantize32(y.cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), q0) and np.array_equal(d.cpu().numpy(), d0)


def test_norm_in_place(ctxs):
    for width in (2048, 40000):
        x, res, w = torch.randn(3, width, device="cuda"), torch.randn(3, width, device="cuda"), torch.ones(
            width, device="cuda")
        want = run_norm(ctxs(), x, res, w, codes=False)
        r2, y2 = res.clone(), x.clone()
        qec.moe_rms_norm(ctxs(), y2, r2, w, 3, width, 1e-5, r2, y2)
        assert torch.equal(r2, want[0]) and torch.equal(y2, want[1])


@pytest.mark.parametrize("off", [1, 2, 3])
def test_norm_unaligned_rows(ctxs, off):
    n = 320
    flat = torch.randn(3 * n + off, device="cuda")
    x = flat[off:].view(3, n)
    w = torch.randn(n + off, device="cuda")[off:]
    check_norm(x, x, w, run_norm(ctxs(), x, x, w))
    y = torch.empty(3 * n + off, device="cuda")[off:].view(3, n)
    qec.moe_rms_norm(ctxs(), x, None, w, 3, n, 1e-5, None, y)
    check_norm(x, None, w, (None, y, None, None))


def test_norm_zero_infinite_and_nan_rows(ctxs):
    x = torch.randn(6, 128, device="cuda")
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, 7] = float("nan")
    x[3] *= 1e30       # the sum of squares overflows: y = 0
    x[4] *= 1e-30      # below eps
    w = torch.ones(128, device="cuda")
    s, y, q, d = run_norm(ctxs(), x, None, w)
    check_norm(x[4:], None, w, (s[4:], y[4:], q[4:], d[4:]))
    assert (y[0] == 0).all() and (q[0] == 0).all() and (d[0] == 0).all()
    assert torch.isnan(y[1, 5]) and (y[1, :5] == 0).all()
    assert torch.isnan(y[2]).all() and torch.isnan(d[2]).all()
    assert (y[3] == 0).all() and (q[3] == 0).all()


def test_norm_other_stream_and_graph(ctxs):
    ctx = ctxs()
    st = torch.cuda.Stream()
    x, w = torch.randn(16, 2048, device="cuda"), torch.ones(2048, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        got = run_norm(ctx, x, x, w, stream=st)
    st.synchronize()
    check_norm(x, x, w, got)
    y = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qec.moe_rms_norm(ctx, x, None, w, 16, 2048, 1e-5, None, y, stream=torch.cuda.current_stream())
    x.mul_(2).add_(1)
    g.replay()
    torch.cuda.synchronize()
    check_norm(x, None, w, (None, y, None, None))


def test_norm_refusals(ctxs):
    ctx = ctxs()
    x, w = torch.randn(2, 48, device="cuda"), torch.ones(48, device="cuda")
    q, d = torch.empty(2, 48, dtype=torch.int8, device="cuda"), torch.empty(2, 2, dtype=torch.float16, device="cuda")

    def bad(*a, **kw):
        with pytest.raises(qec.MoeError) as e:
            qec.moe_rms_norm(ctx, *a, **kw)
        assert e.value.code == -1
    bad(x, None, w, 2, 48, 1e-5, None, None, q, d)       # width not in whole blocks
    bad(x, None, w, 2, 32, 1e-5, None, x, q, None)       # codes without scales
    bad(x, None, w, 2, 48, 1e-5, None, None)             # no output
    bad(x, None, None, 2, 48, 1e-5, None, x)
    bad(None, None, w, 2, 48, 1e-5, None, x)
    bad(x, None, w, -1, 48, 1e-5, None, x)
    bad(x, None, w, 2, 0, 1e-5, None, x)
    bad(x, None, w, 2, 48, -1.0, None, x)
    bad(x, None, w, 2, 48, float("nan"), None, x)
    bad(x, None, w, 2, 48, 1e-5, None, x, dtype=3)
    with pytest.raises(ValueError):
        qec.moe_rms_norm(ctx, x, x.half(), w, 2, 48, 1e-5, None, x)


def test_norm_codes_are_the_forwards_codes():
    # the codes a forward makes of y are the ones the norm wrote
    H, F, E, k, T = 256, 512, 8, 2, 3
    ctx = qec.moe_layer_init(H, F, E, k, 1, E, T, stream=torch.cuda.current_stream().cuda_stream)
    wl = synth.WORKLOADS["tiny"]
    for kind in range(3):
        rows, cols = wl.tensor_shapes[kind]
        qec.register_expert_tensor(ctx, 0, kind, wl.expert_tensor(0, kind), rows, cols, E, None, E)
    x, w = torch.randn(T, H, device="cuda"), 1 + 0.1 * torch.randn(H, device="cuda")
    _, y, q, d = run_norm(ctx, x, x, w)
    idx, cw, out = (torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda"),
                    torch.empty(T, H, device="cuda"))
    qec.moe_ffn_forward_routed(ctx, 0, y, torch.randn(T, E, device="cuda"), T, idx, cw, out)
    xq, xd = np.empty((T, H), np.int8), np.empty((T, H // 32), np.uint16)
    qec.moe_debug_read(ctx, 0, xq)
    qec.moe_debug_read(ctx, 1, xd)
    assert np.array_equal(xq, q.cpu().numpy()) and np.array_equal(xd, d.cpu().numpy().view(np.uint16))
    qec.moe_destroy(ctx)


# ----------------------------------------------------------------- linear
def decode(w, fmt):
    """Canonical bytes [rows][n][18 or 144] -> fp64 weights, element by element of the format's definition."""
    rows, n, _ = w.shape
    if fmt == qec.FMT_Q4_0:
        d = w[:, :, :2].copy().view(np.float16).astype(np.float64)
        q = np.concatenate([w[:, :, 2:] & 15, w[:, :, 2:] >> 4], 2).astype(np.float64) - 8
        return (d * q).reshape(rows, -1)
    d = w[:, :, 0:2].copy().view(np.float16).astype(np.float64)
    m = w[:, :, 2:4].copy().view(np.float16).astype(np.float64)
    b = w[:, :, 4:16].astype(np.int64)
    out = np.empty((rows, n, 8, 32))
    for j in range(8):
        if j < 4:
            s6, m6 = b[:, :, j] & 63, b[:, :, j + 4] & 63
        else:
            s6 = (b[:, :, j + 4] & 15) | ((b[:, :, j - 4] >> 6) << 4)
            m6 = (b[:, :, j + 4] >> 4) | ((b[:, :, j] >> 6) << 4)
        c = w[:, :, 16 + 32 * (j // 2):48 + 32 * (j // 2)]
        out[:, :, j] = d * s6[..., None] * ((c >> (4 * (j % 2))) & 15) - m * m6[..., None]
    return out.reshape(rows, -1)


def make_weights(rows, cols, fmt, seed):
    if fmt == qec.FMT_Q4_0:
        return synth.q4_blocks(seed, rows * cols // 32).reshape(rows, cols // 32, 18)
    return synth.q4k_blocks(seed, rows * cols // 256).reshape(rows, cols // 256, 144)


def check_linear(w, fmt, q, d, y):
    wf = decode(w, fmt)
    x = (q.astype(np.float64).reshape(q.shape[0], -1, 32) * d.astype(np.float64)[..., None]).reshape(q.shape)
    ref, mag = x @ wf.T, np.abs(x) @ np.abs(wf).T
    y = y.cpu().numpy().astype(np.float64)
    err = np.abs(y - ref)
    tol = (6 * (x.shape[1] // 32) + 16) * 2.0 ** -23 * mag
    assert (err <= tol).all(), float((err / tol.clip(1e-300)).max())
    assert np.linalg.norm(err) <= 5e-6 * np.linalg.norm(ref)


SHAPES = [(1, 512, 2048), (1, 33, 64), (1, 1, 256), (2, 2880, 2880), (3, 1000, 512), (4, 129, 2080), (5, 64, 32),
          (7, 2050, 1152), (8, 300, 4096), (9, 257, 2304), (16, 640, 1024), (17, 1, 2048), (31, 200, 288),
          (32, 1280, 2048), (33, 77, 1536), (64, 2880, 2880), (100, 65, 320), (1, 24, 65536), (6, 24, 16384),
          (130, 384, 1280), (257, 130, 2048), (512, 1000, 512),
          # more tiles than SMs: a CTA walks several
          (20, 20000, 288), (40, 20001, 256), (300, 8100, 544)]


@pytest.mark.parametrize("fmt", [qec.FMT_Q4_0, qec.FMT_Q4_K])
@pytest.mark.parametrize("tokens,rows,cols", SHAPES)
def test_linear_shapes(ctxs, tokens, rows, cols, fmt):
    if fmt == qec.FMT_Q4_K and cols % 256:
        cols = (cols + 255) // 256 * 256
    ctx = ctxs(max_tokens=512)
    w = make_weights(rows, cols, fmt, rows + cols)
    lid = qec.moe_linear_register(ctx, w, fmt, rows, cols)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn(tokens, cols, generator=g, device="cuda") * torch.exp(
        torch.randn(cols, generator=g, device="cuda"))
    x[tokens // 2, :32] = 0  # an all-zero block
    q, d = quantize32(x.cpu().numpy())
    y = torch.full((tokens + 1, rows), 7.0, device="cuda")
    qec.moe_linear_forward(ctx, lid, x, tokens, y)
    check_linear(w, fmt, q, d, y[:tokens])
    assert (y[tokens:] == 7).all()
    # from codes: the same bits
    y2 = torch.full((tokens, rows), 7.0, device="cuda")
    qec.moe_linear_forward(ctx, lid, None, tokens, y2, q=torch.from_numpy(q).cuda(), d=torch.from_numpy(d).cuda())
    assert torch.equal(y2, y[:tokens])


@pytest.mark.parametrize("tokens", [1, 4, 40])
def test_linear_extreme_codes_and_scales(ctxs, tokens):
    # every weight code and the largest activation codes, scales over the range of binary16
    ctx = ctxs(max_tokens=512)
    rows, cols = 64, 512
    w = make_weights(rows, cols, qec.FMT_Q4_0, 3)
    dd = np.geomspace(6e-8, 8000, rows * cols // 32).astype(np.float16).reshape(rows, cols // 32, 1)
    w[:, :, :2] = dd.view(np.uint8)
    lid = qec.moe_linear_register(ctx, w, qec.FMT_Q4_0, rows, cols)
    q = np.resize(np.array([127, -127, 0, 1, -1, 64], np.int8), (tokens, cols))
    d = np.geomspace(6e-8, 60000, tokens * (cols // 32)).astype(np.float16).reshape(tokens, -1)
    y = torch.empty(tokens, rows, device="cuda")
    qec.moe_linear_forward(ctx, lid, None, tokens, y, q=torch.from_numpy(q).cuda(), d=torch.from_numpy(d).cuda())
    check_linear(w, qec.FMT_Q4_0, q, d, y)


@pytest.mark.parametrize("tokens", [1, 12, 70])
def test_linear_nan_stays_in_its_token(ctxs, tokens):
    ctx = ctxs(max_tokens=512)
    w = make_weights(96, 256, qec.FMT_Q4_0, 9)
    lid = qec.moe_linear_register(ctx, w, qec.FMT_Q4_0, 96, 256)
    x = torch.randn(tokens, 256, device="cuda")
    y0, y1 = torch.empty(tokens, 96, device="cuda"), torch.empty(tokens, 96, device="cuda")
    qec.moe_linear_forward(ctx, lid, x, tokens, y0)
    x[tokens - 1, 3] = float("nan")
    qec.moe_linear_forward(ctx, lid, x, tokens, y1)
    assert torch.isnan(y1[-1]).all()
    assert torch.equal(y1[:-1], y0[:-1])


def test_linear_graph_and_no_tokens(ctxs):
    ctx = qec.moe_layer_init(64, 32, 8, 2, 1, 0, 64, stream=(st := torch.cuda.Stream()).cuda_stream)
    w = make_weights(200, 512, qec.FMT_Q4_0, 4)
    lid = qec.moe_linear_register(ctx, w, qec.FMT_Q4_0, 200, 512)
    qec.moe_linear_forward(ctx, lid, None, 0, None)
    for tokens in (1, 48):
        x, y = torch.randn(tokens, 512, device="cuda"), torch.zeros(tokens, 200, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            qec.moe_linear_forward(ctx, lid, x, tokens, y)
        x.mul_(-3)
        torch.cuda.synchronize()
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        q, d = quantize32(x.cpu().numpy())
        check_linear(w, qec.FMT_Q4_0, q, d, y)
    qec.moe_destroy(ctx)


def test_linear_refusals(ctxs):
    ctx = ctxs(max_tokens=64)
    w = make_weights(8, 256, qec.FMT_Q4_0, 1)

    def bad(f, *a, **kw):
        with pytest.raises(qec.MoeError) as e:
            f(ctx, *a, **kw)
        assert e.value.code == -1
    bad(qec.moe_linear_register, w, qec.FMT_Q8_0, 8, 256)
    bad(qec.moe_linear_register, w, qec.FMT_Q4_0, 8, 250)
    bad(qec.moe_linear_register, w, qec.FMT_Q4_K, 8, 224)
    bad(qec.moe_linear_register, w, qec.FMT_Q4_0, 0, 256)
    bad(qec.moe_linear_register, w, qec.FMT_Q4_0, 8, 65536 + 32)
    bad(qec.moe_linear_register, None, qec.FMT_Q4_0, 8, 256)
    lid = qec.moe_linear_register(ctx, w, qec.FMT_Q4_0, 8, 256)
    x, y = torch.randn(64, 256, device="cuda"), torch.empty(64, 8, device="cuda")
    q, d = torch.zeros(64, 256, dtype=torch.int8, device="cuda"), torch.zeros(64, 8, dtype=torch.float16, device="cuda")
    f = qec.moe_linear_forward
    bad(f, lid + 1, x, 1, y)
    bad(f, -1, x, 1, y)
    bad(f, lid, x, 65, y)                       # above max_tokens
    bad(f, lid, x, -1, y)
    bad(f, lid, x, 1, None)
    bad(f, lid, None, 1, y)
    bad(f, lid, None, 1, y, q=q)                # codes without scales
    bad(f, lid, x, 1, y, q=q, d=d)              # both inputs
    bad(f, lid, x.view(-1)[1:], 1, y)           # not 16-byte aligned
    bad(f, lid, x, 1, y, stream=torch.cuda.Stream())


# ----------------------------------------------------------------- router
def router_ref(z, idx, mask, gw, a, b, renorm):
    """Losses, counts and gradient in fp64 numpy."""
    T, E = z.shape
    k = idx.shape[1]
    on = np.ones(T, bool) if mask is None else mask != 0
    n = int(on.sum())
    counts = np.bincount(idx[on].reshape(-1), minlength=E)
    loss, dz, mag = np.zeros(2), np.zeros((T, E)), np.zeros((T, E))
    f = counts / (n * k) if n else np.zeros(E)
    for t in np.flatnonzero(on):
        top = z[t].max()
        if top == -np.inf:
            continue
        e = np.exp(z[t] - top)
        p, lse = e / e.sum(), top + np.log(e.sum())
        dot = (p * f).sum()
        loss += [a * E * dot / n, b * lse * lse / n]
        dz[t] = p * (a * E * (f - dot) + 2 * b * lse) / n
        mag[t] = p * (abs(a) * E * (f + dot) + 2 * abs(b * lse)) / n
        if gw is not None:
            if renorm:
                zs = z[t, idx[t]]
                w = np.exp(zs - zs.max()) if zs.max() > -np.inf else np.zeros(k)
                w = w / w.sum() if w.sum() > 0 else w
                g, m = w * (gw[t] - (w * gw[t]).sum()), w * (abs(gw[t]) + abs(w * gw[t]).sum())
            else:
                ps = p[idx[t]]
                g, m = ps * gw[t], ps * abs(gw[t])
                dz[t] -= p * g.sum()
                mag[t] += p * m.sum()
            np.add.at(dz[t], idx[t], g)
            np.add.at(mag[t], idx[t], m)
    return loss, counts, dz, mag


def run_router(ctx, z, idx, mask, gw, a, b, grad=True):
    T, E = z.shape
    loss = torch.full((2,), 7.0, device="cuda")
    counts = torch.full((E,), 7, dtype=torch.int32, device="cuda")
    dz = torch.full((T, E), 7.0, device="cuda") if grad else None
    qec.moe_router_loss(ctx, z, idx, mask, gw, T, E, idx.shape[1], a, b, loss, counts, dz)
    return loss, counts, dz


def check_router(z, idx, mask, gw, a, b, renorm, got):
    zn = z.cpu().numpy().astype(np.float64)
    ref = router_ref(zn, idx.cpu().numpy(), None if mask is None else mask.cpu().numpy(),
                     None if gw is None else gw.cpu().numpy().astype(np.float64), a, b, renorm)
    loss, counts, dz = got
    assert np.array_equal(counts.cpu().numpy(), ref[1])
    fin = np.where(np.isfinite(zn), zn, np.nan)
    spread = float(np.nanmax(fin) - np.nanmin(fin)) if np.isfinite(zn).any() else 0.0
    rel = (spread + z.shape[1] / 32 + 64) * U
    assert (np.abs(loss.cpu().numpy() - ref[0]) <= rel * np.abs(ref[0]) + 1e-38).all(), (loss, ref[0])
    if dz is not None:
        err = np.abs(dz.cpu().numpy() - ref[2])
        assert (err <= rel * ref[3] + 1e-37).all(), float((err / (rel * ref[3]).clip(1e-300)).max())


def router_inputs(T, E, k, seed, scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = scale * torch.randn(T, E, generator=g, device="cuda") - 1.1 * torch.log(
        torch.arange(E, device="cuda").float() + 1)
    idx = torch.topk(z, k, dim=1).indices.to(torch.int32)
    mask = (torch.rand(T, generator=g, device="cuda") < 0.7).to(torch.uint8)
    gw = torch.randn(T, k, generator=g, device="cuda")
    return z.contiguous(), idx.contiguous(), mask, gw


@pytest.mark.parametrize("renorm", [1, 0])
@pytest.mark.parametrize("T,E,k", [(1, 512, 8), (1, 1, 1), (2, 8, 2), (5, 33, 8), (8, 128, 4), (31, 60, 32),
                                   (64, 512, 8), (3, 1000, 6), (2, 1028, 5), (2, 4096, 8), (3, 4095, 32), (700, 257, 3),
                                   (5000, 128, 4)])
def test_router_shapes(ctxs, T, E, k, renorm):
    ctx = ctxs(1, E, k, renorm)
    z, idx, mask, gw = router_inputs(T, E, k, T + E)
    for m, g in ((None, gw), (mask, gw), (mask, None)):
        check_router(z, idx, m, g, 0.01, 0.001, renorm, run_router(ctx, z, idx, m, g, 0.01, 0.001))
    check_router(z, idx, mask, None, 0.5, 0.0, renorm, run_router(ctx, z, idx, mask, None, 0.5, 0.0, grad=False))


def test_router_gradient_against_differences(ctxs):
    # central differences of the fp64 losses and of sum(gw * routing weights), the counts held
    T, E, k, a, b, h = 4, 12, 3, 0.3, 0.05, 1e-5
    z, idx, mask, gw = router_inputs(T, E, k, 5)
    mask[:] = torch.tensor([1, 0, 1, 1])
    for renorm in (1, 0):
        ctx = ctxs(1, E, k, renorm)
        _, _, dz = run_router(ctx, z, idx, mask, gw, a, b)
        zn, ix, mk, g = (v.cpu().numpy().astype(np.float64) for v in (z, idx, mask, gw))
        ix = ix.astype(int)

        def total(zz):
            on = mk != 0
            f = np.bincount(ix[on].reshape(-1), minlength=E) / (on.sum() * k)
            p = np.exp(zz) / np.exp(zz).sum(1, keepdims=True)
            lse = np.log(np.exp(zz).sum(1))
            w = np.take_along_axis(p, ix, 1)
            if renorm:
                w = w / w.sum(1, keepdims=True)
            return (a * E * (p @ f)[on].mean() + b * (lse[on] ** 2).mean() + (g * w)[on].sum())
        num = np.zeros((T, E))
        for t in range(T):
            for e in range(E):
                zp, zm = zn.copy(), zn.copy()
                zp[t, e] += h
                zm[t, e] -= h
                num[t, e] = (total(zp) - total(zm)) / (2 * h)
        # differences: third-derivative error h^2 ~ 1e-10 and cancellation 1e-16 / h ~ 1e-11, each times O(10); fp32: 100 u
        assert np.abs(num - dz.cpu().numpy()).max() < 1e-8 + 100 * U * np.abs(num).max()


def test_router_masks_and_infinities(ctxs):
    ctx = ctxs(1, 64, 4)
    z, idx, mask, gw = router_inputs(9, 64, 4, 1)
    mask[:] = 0
    loss, counts, dz = run_router(ctx, z, idx, mask, gw, 0.1, 0.1)
    assert (loss == 0).all() and (counts == 0).all() and (dz == 0).all()
    mask[4] = 200  # any non-zero value keeps a token
    check_router(z, idx, mask, gw, 0.1, 0.1, 1, run_router(ctx, z, idx, mask, gw, 0.1, 0.1))
    # experts a token cannot take, rows of nothing else, masks of the type's lowest value
    z[0, 10:] = -float("inf")
    z[1] = -float("inf")
    z[2, :63] = -float("inf")
    z[3, 5:] = torch.finfo(torch.float32).min
    check_router(z, idx, None, gw, 0.1, 0.0, 1, run_router(ctx, z, idx, None, gw, 0.1, 0.0))
    got = run_router(ctx, z, idx, None, None, 0.1, 0.1)
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[2]).all()
    assert (got[2][1] == 0).all()
    # values in a masked row do not matter
    z2 = z.clone()
    z2[5] = float("nan")
    m = torch.ones(9, dtype=torch.uint8, device="cuda")
    m[5] = 0
    a, b = run_router(ctx, z, idx, m, gw, 0.1, 0.1), run_router(ctx, z2, idx, m, gw, 0.1, 0.1)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    # NaN in a row that counts reaches the losses and that row's gradient
    for row in (z2[5], None):
        if row is None:
            z2[5] = 0
            z2[5, 7] = float("nan")
        loss, _, dz = run_router(ctx, z2, idx, None, None, 0.1, 0.1)
        assert torch.isnan(loss).all() and torch.isnan(dz[5]).all() and torch.isfinite(dz[6]).all()


def test_router_repeats_and_no_tokens(ctxs):
    ctx = ctxs(1, 512, 8)
    z, idx, mask, gw = router_inputs(3000, 512, 8, 3)
    first = run_router(ctx, z, idx, mask, gw, 0.01, 0.001)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(first, run_router(ctx, z, idx, mask, gw, 0.01, 0.001)))
    loss, counts = torch.full((2,), 7.0, device="cuda"), torch.full((512,), 7, dtype=torch.int32, device="cuda")
    qec.moe_router_loss(ctx, None, None, None, None, 0, 512, 8, 0.1, 0.1, loss, counts, None)
    assert (loss == 0).all() and (counts == 0).all()


def test_router_repeated_and_bad_ids(ctxs):
    ctx = ctxs(1, 16, 3)
    z, idx, _, gw = router_inputs(5, 16, 3, 2)
    idx[:, 1] = idx[:, 0]  # route_topk writes distinct ids; repeated ones still add up
    for T in (5, 1):
        check_router(z[:T], idx[:T], None, gw[:T], 0.1, 0.1, 1, run_router(ctx, z[:T], idx[:T], None, gw[:T], 0.1, 0.1))
    bad = idx.clone()
    bad[2, 0], bad[3, 1] = 16, -5
    as0 = idx.clone()
    as0[2, 0], as0[3, 1] = 0, 0
    check_router(z, as0, None, gw, 0.1, 0.1, 1, run_router(ctx, z, bad, None, gw, 0.1, 0.1))
    with pytest.raises(qec.MoeError) as e:
        qec.miss_drain(ctx)
    assert e.value.code == -8
    qec.miss_drain(ctx)


def test_router_refusals(ctxs):
    ctx = ctxs(1, 16, 3)
    z, idx, mask, gw = router_inputs(5, 16, 3, 2)
    loss, counts = torch.empty(2, device="cuda"), torch.empty(16, dtype=torch.int32, device="cuda")

    def bad(*a, **kw):
        with pytest.raises(qec.MoeError) as e:
            qec.moe_router_loss(ctx, *a, **kw)
        assert e.value.code == -1
    bad(z, idx, None, None, 5, 15, 3, 0.1, 0.1, loss, counts)
    bad(z, idx, None, None, 5, 16, 2, 0.1, 0.1, loss, counts)
    bad(z, idx, None, None, -1, 16, 3, 0.1, 0.1, loss, counts)
    bad(None, idx, None, None, 5, 16, 3, 0.1, 0.1, loss, counts)
    bad(z, None, None, None, 5, 16, 3, 0.1, 0.1, loss, counts)
    bad(z, idx, None, None, 5, 16, 3, 0.1, 0.1, None, counts)
    bad(z, idx, None, None, 5, 16, 3, 0.1, 0.1, loss, None)
    bad(z, idx, None, None, 5, 16, 3, 0.1, 0.1, loss, counts, z)  # in place
    bad(z, idx, None, None, 5, 16, 3, 0.1, 0.1, loss, counts, stream=torch.cuda.Stream())
