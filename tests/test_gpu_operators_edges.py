"""GPU tests of the operators around the routed experts where they can go
wrong: registration beside other streams, weights and activations over the whole
range of their formats, batches that leave the tensor cores, layers registered
between a graph's capture and its replay.

Tolerances are those of the operators' own tests.  Linear, element by element:
|err| <= (6 nb + 16) 2^-23 sum |w x| of nb blocks of 32 columns (operands to 2^-22,
at most 6 accumulations a block).
"""
import numpy as np
import pytest

import quantized_expert_cache_gb300 as qec
from test_gpu_operators import check_linear, check_norm, decode, make_weights, run_norm

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def context(max_tokens=64, experts=8, k=2, stream=None):
    st = torch.cuda.current_stream() if stream is None else stream
    return qec.moe_layer_init(64, 32, experts, k, 1, 0, max_tokens, stream=st.cuda_stream)


def elementwise(w, fmt, q, d, y):
    """Every |err| against the bound, where the reference is finite; the reference."""
    x = (q.astype(np.float64).reshape(q.shape[0], -1, 32) * d.astype(np.float64)[..., None]).reshape(q.shape)
    wf = decode(w, fmt)
    with np.errstate(invalid="ignore", over="ignore"):
        ref, mag = x @ wf.T, np.abs(x) @ np.abs(wf).T
        err = np.abs(y.cpu().numpy().astype(np.float64) - ref)
    tol = (6 * (x.shape[1] // 32) + 16) * 2.0 ** -23 * mag
    on = np.isfinite(ref)
    assert (err[on] <= tol[on]).all(), float((err[on] / tol[on].clip(1e-300)).max())
    return ref


def test_registration_on_a_side_stream():
    # the same blocks registered on a stream of their own and on the default one: the same bits
    rows, cols = 8192, 8192
    w = make_weights(rows, cols, qec.FMT_Q4_0, 11)
    x = torch.randn(40, cols, device="cuda")
    out = []
    for st in (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
        ctx = context(stream=st)
        lid = qec.moe_linear_register(ctx, w, qec.FMT_Q4_0, rows, cols)
        torch.cuda.synchronize()
        for n in (1, 40):
            y = torch.full((n, rows), 7.0, device="cuda")
            torch.cuda.synchronize()
            qec.moe_linear_forward(ctx, lid, x, n, y)
            torch.cuda.synchronize()
            out.append(y)
        qec.moe_destroy(ctx)
    for y in out[2:]:
        assert torch.equal(y, out[0 if y.shape[0] == 1 else 1])


@pytest.mark.parametrize("tokens", [1, 5, 40, 130])
def test_linear_q4k_rows_over_the_whole_scale_range(tokens):
    # every row has its own magnitude, from the smallest to the largest binary16 scales
    rows, cols = 300, 512
    ctx = context(max_tokens=130)
    w = make_weights(rows, cols, qec.FMT_Q4_K, 21)
    top = np.geomspace(1e-6, 60000, rows)[np.random.default_rng(5).permutation(rows)][:, None]
    f = np.random.default_rng(4).uniform(0.25, 1.0, (2, rows, cols // 256))
    w[:, :, 0:2] = (top * f[0]).astype(np.float16)[..., None].view(np.uint8)
    w[:, :, 2:4] = (top * f[1]).astype(np.float16)[..., None].view(np.uint8)
    lid = qec.moe_linear_register(ctx, w, qec.FMT_Q4_K, rows, cols)
    rng = np.random.default_rng(tokens)
    q = rng.integers(-127, 128, (tokens, cols)).astype(np.int8)
    d = rng.uniform(0.001, 0.01, (tokens, cols // 32)).astype(np.float16)
    y = torch.empty(tokens, rows, device="cuda")
    qec.moe_linear_forward(ctx, lid, None, tokens, y, q=torch.from_numpy(q).cuda(), d=torch.from_numpy(d).cuda())
    elementwise(w, qec.FMT_Q4_K, q, d, y)
    qec.moe_destroy(ctx)


@pytest.mark.parametrize("fmt", [qec.FMT_Q4_0, qec.FMT_Q4_K])
@pytest.mark.parametrize("tokens", [1, 5, 40, 130])
def test_linear_small_activations_beside_a_block_that_the_weights_ignore(tokens, fmt):
    # the first block is 2^22 times the others, and its weights are zero
    rows, cols = 140, 512
    ctx = context(max_tokens=130)
    w = make_weights(rows, cols, fmt, 22)
    first = 1  # blocks of the weights' format that hold the first 32 (256) columns
    w[:, :first, :4 if fmt == qec.FMT_Q4_K else 2] = 0
    lid = qec.moe_linear_register(ctx, w, fmt, rows, cols)
    rng = np.random.default_rng(tokens)
    q = rng.integers(-127, 128, (tokens, cols)).astype(np.int8)
    d = (rng.uniform(1, 2, (tokens, cols // 32)) * 2.0 ** -14).astype(np.float16)
    d[:, 0] = 256.0
    y = torch.empty(tokens, rows, device="cuda")
    qec.moe_linear_forward(ctx, lid, None, tokens, y, q=torch.from_numpy(q).cuda(), d=torch.from_numpy(d).cuda())
    elementwise(w, fmt, q, d, y)
    qec.moe_destroy(ctx)


@pytest.mark.parametrize("tokens", [1, 5, 40, 130])
def test_linear_weights_beyond_binary16(tokens):
    # 8 d above 65504, infinite and NaN scales: batches too take the exact block dots
    rows, cols = 70, 2080
    ctx = context(max_tokens=130)
    w = make_weights(rows, cols, qec.FMT_Q4_0, 23)
    dd = np.geomspace(1e-6, 60000, rows * cols // 32).astype(np.float16).reshape(rows, cols // 32, 1)
    w[:, :, :2] = dd.view(np.uint8)
    rng = np.random.default_rng(tokens)
    x = torch.from_numpy(rng.standard_normal((tokens, cols)).astype(np.float32)).cuda()
    q, d = (a.numpy() for a in codes_of(x))
    y = torch.empty(tokens, rows, device="cuda")
    lid = qec.moe_linear_register(ctx, w, qec.FMT_Q4_0, rows, cols)
    qec.moe_linear_forward(ctx, lid, x, tokens, y)
    elementwise(w, qec.FMT_Q4_0, q, d, y)
    w[3, 5, :2] = np.array([np.inf], np.float16).view(np.uint8)
    w[9, 0, :2] = np.array([np.nan], np.float16).view(np.uint8)
    lid = qec.moe_linear_register(ctx, w, qec.FMT_Q4_0, rows, cols)
    y2 = torch.empty(tokens, rows, device="cuda")
    qec.moe_linear_forward(ctx, lid, x, tokens, y2)
    assert not torch.isfinite(y2[:, 3]).any() and torch.isnan(y2[:, 9]).all()
    keep = [r for r in range(rows) if r not in (3, 9)]
    assert torch.equal(y2[:, keep], y[:, keep])
    qec.moe_destroy(ctx)


def codes_of(x):
    """int8 codes and binary16 scales of fp32 rows, each step in binary32."""
    from test_gpu_operators import quantize32
    q, d = quantize32(x.cpu().numpy())
    return torch.from_numpy(q), torch.from_numpy(d)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,width", [(1, 2048), (5, 96), (300, 2048), (700, 160), (3, 1001), (3, 40000)])
def test_norm_sums_in_place(tokens, width, dtype):
    ctx = context()
    g = torch.Generator(device="cuda").manual_seed(width)
    x, res = (torch.randn(tokens, width, generator=g, device="cuda").to(dtype) for _ in range(2))
    w = 1 + 0.3 * torch.randn(width, generator=g, device="cuda")
    want = run_norm(ctx, x, res, w, codes=width % 32 == 0)
    check_norm(x, res, w, want)
    for into in (0, 1):
        a = [x.clone(), res.clone()]
        y = torch.empty(tokens, width, device="cuda")
        qec.moe_rms_norm(ctx, a[0], a[1], w, tokens, width, 1e-5, a[into], y)
        assert torch.equal(a[into], want[0]) and torch.equal(y, want[1])
        assert torch.equal(a[1 - into], (x, res)[1 - into])
    if dtype == torch.float32:
        for into in (0, 1):
            a = [x.clone(), res.clone()]
            qec.moe_rms_norm(ctx, a[0], a[1], w, tokens, width, 1e-5, a[1 - into], a[into])
            assert torch.equal(a[1 - into], want[0]) and torch.equal(a[into], want[1])
    qec.moe_destroy(ctx)


def test_norm_of_the_widest_row():
    # 2^31 - 1 elements: the index steps past the end need the 32nd bit
    n = 2 ** 31 - 1
    ctx = context()
    at = torch.cat([torch.arange(0, n, n // 60, device="cuda"), torch.arange(n - 3, n, device="cuda")]).unique()
    x = torch.zeros(1, n, dtype=torch.bfloat16, device="cuda")
    x[0, at] = 1
    y = torch.full((1, n), 7.0, device="cuda")
    qec.moe_rms_norm(ctx, x, None, torch.full((n,), 0.5, device="cuda"), 1, n, 1e-9, None, y)
    torch.cuda.synchronize()
    r = 0.5 / np.sqrt(at.numel() / n + 1e-9)  # sums of ones are exact; the rest is 6 roundings
    assert (abs(y[0, at].double() - r) <= 6 * 2.0 ** -24 * r).all()
    y[0, at] = 0
    assert int(torch.count_nonzero(y)) == 0
    qec.moe_destroy(ctx)


@pytest.mark.parametrize("fmt", [qec.FMT_Q4_0, qec.FMT_Q4_K])
@pytest.mark.parametrize("tokens,rows,cols", [(1030, 130, 1280), (4096, 200, 512), (12289, 33, 256)])
def test_linear_prompts(tokens, rows, cols, fmt):
    # prompts of the workloads' lengths: many token tiles, the last one ragged
    ctx = context(max_tokens=tokens)
    w = make_weights(rows, cols, fmt, tokens)
    lid = qec.moe_linear_register(ctx, w, fmt, rows, cols)
    x = torch.randn(tokens, cols, generator=torch.Generator(device="cuda").manual_seed(tokens), device="cuda")
    q, d = (a.numpy() for a in codes_of(x))
    y = torch.full((tokens + 1, rows), 7.0, device="cuda")
    qec.moe_linear_forward(ctx, lid, x, tokens, y)
    check_linear(w, fmt, q, d, y[:tokens])
    assert (y[tokens:] == 7).all()
    qec.moe_destroy(ctx)


def test_linear_more_token_groups_than_a_grid_has_rows():
    # four tokens a pass: more than 65535 passes
    tokens = 4 * 65535 + 5
    ctx = context(max_tokens=tokens)
    w = make_weights(3, 32, qec.FMT_Q4_0, 24)
    w[:, :, :2] = np.full((3, 1, 1), 10000.0, np.float16).view(np.uint8)
    lid = qec.moe_linear_register(ctx, w, qec.FMT_Q4_0, 3, 32)
    rng = np.random.default_rng(3)
    q = rng.integers(-127, 128, (tokens, 32)).astype(np.int8)
    d = rng.uniform(0.001, 0.01, (tokens, 1)).astype(np.float16)
    y = torch.full((tokens + 1, 3), 7.0, device="cuda")
    qec.moe_linear_forward(ctx, lid, None, tokens, y, q=torch.from_numpy(q).cuda(), d=torch.from_numpy(d).cuda())
    elementwise(w, qec.FMT_Q4_0, q, d, y[:tokens])
    assert (y[tokens:] == 7).all()
    qec.moe_destroy(ctx)


def test_linear_layer_keeps_its_workspace():
    # a wider layer is registered after a batch of the first was captured: the graph and direct calls
    # of both layers still give the bits of a context that holds one layer
    st = torch.cuda.Stream()
    shapes = ((200, 512), (130, 4096))
    ws = [make_weights(r, c, qec.FMT_Q4_0, c) for r, c in shapes]
    xs = [torch.randn(40, c, device="cuda") for _, c in shapes]
    want = []
    for w, x, (r, c) in zip(ws, xs, shapes):
        ctx = context(stream=st)
        lid = qec.moe_linear_register(ctx, w, qec.FMT_Q4_0, r, c)
        y = torch.empty(40, r, device="cuda")
        torch.cuda.synchronize()
        qec.moe_linear_forward(ctx, lid, x, 40, y)
        torch.cuda.synchronize()
        want.append(y)
        qec.moe_destroy(ctx)
    ctx = context(stream=st)
    ids = [qec.moe_linear_register(ctx, ws[0], qec.FMT_Q4_0, *shapes[0])]
    yg = torch.zeros(40, shapes[0][0], device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        qec.moe_linear_forward(ctx, ids[0], xs[0], 40, yg)
    ids.append(qec.moe_linear_register(ctx, ws[1], qec.FMT_Q4_0, *shapes[1]))
    ys = [torch.zeros(40, r, device="cuda") for r, _ in shapes]
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for i in (1, 0):
            qec.moe_linear_forward(ctx, ids[i], xs[i], 40, ys[i])
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ys[0], want[0]) and torch.equal(ys[1], want[1]) and torch.equal(yg, want[0])
    qec.moe_destroy(ctx)


def test_linear_registration_without_memory_leaves_no_error():
    # an allocation that cannot be had is reported once: the next calls do not meet it again
    ctx = context()
    w = make_weights(40, 256, qec.FMT_Q4_0, 25)
    with pytest.raises(qec.MoeError) as e:
        qec.moe_linear_register(ctx, w, qec.FMT_Q4_0, 1 << 26, 65536)  # 2.4 TB: refused before w is read
    assert e.value.code == -2
    lid = qec.moe_linear_register(ctx, w, qec.FMT_Q4_0, 40, 256)
    y = torch.empty(1, 40, device="cuda")
    qec.moe_linear_forward(ctx, lid, torch.randn(1, 256, device="cuda"), 1, y)
    torch.cuda.synchronize()
    qec.moe_destroy(ctx)


# ---- offsets that pass 32 bits: the first and the last rows of results of more than 2^31 elements
def test_norm_offsets_beyond_32_bits():
    tokens, width = 540000, 4096
    ctx = context()
    w = 1 + 0.3 * torch.randn(width, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    x = torch.zeros(tokens, width, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, 262143, 524287, 524288, 524289, tokens - 1], device="cuda")
    x[at] = torch.randn(len(at), width, generator=torch.Generator(device="cuda").manual_seed(2),
                        device="cuda").bfloat16()
    y = torch.full((tokens, width), 7.0, device="cuda")
    q = torch.full((tokens, width), 7, dtype=torch.int8, device="cuda")
    d = torch.full((tokens, width // 32), 7.0, dtype=torch.float16, device="cuda")
    qec.moe_rms_norm(ctx, x, None, w, tokens, width, 1e-5, None, y, q, d)
    torch.cuda.synchronize()
    check_norm(x[at], None, w, (None, y[at], q[at], d[at]))
    y[at], q[at], d[at] = 0, 0, 0
    assert not y.any() and not q.any() and not d.any()
    qec.moe_destroy(ctx)


@pytest.mark.parametrize("large", [False, True])  # weights within binary16 and beyond: tensor cores, dp4a
def test_linear_offsets_beyond_32_bits(large):
    tokens, rows, cols = 33000, 65537, 32
    ctx = context(max_tokens=tokens)
    w = make_weights(rows, cols, qec.FMT_Q4_0, 31)
    if large:
        w[0, 0, :2] = np.array([10000.0], np.float16).view(np.uint8)
    lid = qec.moe_linear_register(ctx, w, qec.FMT_Q4_0, rows, cols)
    rng = np.random.default_rng(1)
    q = rng.integers(-127, 128, (tokens, cols)).astype(np.int8)
    d = rng.uniform(0.001, 0.01, (tokens, 1)).astype(np.float16)
    y = torch.full((tokens, rows), float("inf"), device="cuda")
    qec.moe_linear_forward(ctx, lid, None, tokens, y, q=torch.from_numpy(q).cuda(), d=torch.from_numpy(d).cuda())
    torch.cuda.synchronize()
    at = np.array([0, 1, 16383, 32766, 32767, 32768, tokens - 1])
    elementwise(w, qec.FMT_Q4_0, q[at], d[at], y[torch.from_numpy(at).cuda()])
    assert torch.isfinite(y.amax()) and torch.isfinite(y.amin())  # every element was written
    qec.moe_destroy(ctx)


def test_router_offsets_beyond_32_bits():
    T, E, k, a, b = 530000, 4096, 2, 0.01, 0.001
    ctx = context(max_tokens=1, experts=E, k=k)
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.randn(T, E, generator=g, device="cuda")
    idx = torch.randint(0, E // 2, (T, k), generator=g, device="cuda", dtype=torch.int32)
    idx[:, 1] += E // 2
    gw = torch.randn(T, k, generator=g, device="cuda")
    loss, counts = torch.empty(2, device="cuda"), torch.empty(E, dtype=torch.int32, device="cuda")
    dz = torch.full((T, E), float("inf"), device="cuda")
    qec.moe_router_loss(ctx, z, idx, None, gw, T, E, k, a, b, loss, counts, dz)
    torch.cuda.synchronize()
    ref_counts = torch.bincount(idx.reshape(-1).long(), minlength=E)
    assert torch.equal(counts.long(), ref_counts)
    f = ref_counts.double() / (T * k)
    at = torch.tensor([0, 1, 262144, 524287, 524288, T - 1], device="cuda")
    zz = z[at].double()
    p, lse = torch.softmax(zz, 1), torch.logsumexp(zz, 1, keepdim=True)
    dot = (p * f).sum(1, keepdim=True)
    ref = p * (a * E * (f - dot) + 2 * b * lse) / T
    mag = p * (a * E * (f + dot) + 2 * b * lse.abs()) / T
    ids, gd = idx[at].long(), gw[at].double()
    pw = torch.softmax(zz.gather(1, ids), 1)
    mean = (pw * gd).sum(1, keepdim=True)
    ref.scatter_add_(1, ids, pw * (gd - mean))
    mag.scatter_add_(1, ids, pw * (gd.abs() + (pw * gd).abs().sum(1, keepdim=True)))
    spread = float(zz.max() - zz.min())
    assert ((dz[at].double() - ref).abs() <= (spread + E / 32 + 64) * 2.0 ** -24 * mag + 1e-37).all()
    assert torch.isfinite(dz.amax()) and torch.isfinite(dz.amin())
    # the losses, against the mean over all rows in 64 bits
    total = torch.zeros(2, dtype=torch.float64, device="cuda")
    for r in range(0, T, 20000):
        zz = z[r:r + 20000].double()
        total[0] += (torch.softmax(zz, 1) @ f).sum() * a * E / T
        total[1] += torch.logsumexp(zz, 1).square().sum() * b / T
    rel = (12 + E / 32 + 64 + T / (608 * 8)) * 2.0 ** -24  # a warp adds up its rows one by one
    assert ((loss.double() - total).abs() <= rel * total).all()
    qec.moe_destroy(ctx)
