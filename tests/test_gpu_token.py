"""GPU tests of moe_token_logprobs and moe_token_logprobs_grad against plain
64-bit implementations.

Tolerances, with u = 2^-24 (unit roundoff of binary32), d_j = scale (max x - x_j),
e_j = exp(-d_j), R = the sum of e_j without one largest element, S = 1 + R:
- e_j: three roundings in its exponent, ex2's 2 ulp: relative (3 d_j + 4) u; sums
  over a lane's at most V/256 elements, then 16 joins (each with its own e_j):
  |dR| <= u (3 sum e d + R (V/256 + 40)) + 2^-126 V: a term below binary32's
  smallest normal number, 2^-126, is taken as 0 (ex2 flushes it), and there are
  fewer than V of them, each below 2^-126.  log S = log1p(R):
  |d log S| <= |dR| / S + 4 u log S.
- logp_j = -d_j - log S: 3 u d_j + |d log S| + u |logp_j|.
- H = log S + sum e d / S: with D1 = sum e d / S and D2 = sum e d^2 / S,
  |dH| <= |d log S| + u (3 D2 + D1 (V/256 + 48)) + D1 |dR| / S + 2 u H.
- gradient, from the stats and entropies given: log p_j to u (3 d_j + 2 |log p_j|),
  p_j = 2^(log2e log p_j) to (3 d_j + 3 |log p_j| + 8) u of itself, the products a
  few roundings more; then half a step of the output's type.
Alternatives are whole numbers and have to be equal.
"""
import math

import numpy as np
import pytest

import quantized_expert_cache_gb300 as qec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def ctx():
    c = qec.moe_layer_init(64, 32, 8, 2, 1, 0, 1, stream=torch.cuda.current_stream().cuda_stream)
    yield c
    torch.cuda.synchronize()
    qec.moe_destroy(c)


def logits_of(tokens, vocab, dtype, seed=0, spread=3.0, off=0):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 31 * vocab + tokens)
    flat = torch.empty(tokens * vocab + off, dtype=dtype, device="cuda")
    x = flat[off:].view(tokens, vocab)
    x.copy_(torch.randn(tokens, vocab, generator=g, device="cuda") * spread)
    targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    return x, targets


def forward(ctx, x, targets, n_top=0, scale=1.0, stream=None, extra=0):
    t, v = x.shape
    out = dict(logp=torch.full((t + extra,), 7.0, device="cuda") if targets is not None else None,
               entropy=torch.full((t + extra,), 7.0, device="cuda"),
               top_idx=torch.full((t + extra, n_top), 7, dtype=torch.int32, device="cuda"),
               top_logp=torch.full((t + extra, n_top), 7.0, device="cuda"),
               stats=torch.full((t + extra, 2), 7.0, device="cuda"))
    qec.moe_token_logprobs(ctx, x, targets, t, v, out["logp"], out["entropy"], n_top,
                           out["top_idx"] if n_top else None, out["top_logp"] if n_top else None, out["stats"],
                           scale=scale, stream=stream)
    return out


class Ref:
    """The definition in 64 bits and the bounds above, of rows with a finite largest logit and no NaN."""

    def __init__(self, x, scale):
        x64 = x.double()
        self.v = x.shape[1]
        self.top = x64.max(1, keepdim=True).values
        self.d = (self.top - x64) * scale
        e = torch.exp(-self.d)
        first = torch.zeros_like(e).scatter_(1, x64.max(1, keepdim=True).indices, 1.0)
        rest = (e * (1 - first)).sum(1, keepdim=True)
        ed = torch.where(e > 0, e * self.d, 0.0)
        s = 1 + rest
        d1, d2 = ed.sum(1, keepdim=True) / s, torch.where(e > 0, ed * self.d, 0.0).sum(1, keepdim=True) / s
        chain = self.v / 256 + 40
        d_rest = U * (3 * ed.sum(1, keepdim=True) + rest * chain) + self.v * 2.0 ** -126
        self.log_sum = torch.log1p(rest)
        self.t_log_sum = d_rest / s + 4 * U * self.log_sum + 1e-37
        self.entropy = self.log_sum + d1
        self.t_entropy = (self.t_log_sum + U * (3 * d2 + d1 * (chain + 8)) + d1 * d_rest / s + 2 * U * self.entropy)

    def logp(self, idx):
        d = self.d.gather(1, idx)
        lp = -d - self.log_sum
        return lp, torch.where(torch.isinf(d), 0.0, 3 * U * d + self.t_log_sum + U * lp.abs())


def close(got, want, tol):
    got, want = got.double().reshape(want.shape), want.double()
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    ok = same | ((got - want).abs() <= tol)
    assert ok.all(), (got[~ok][:4], want[~ok][:4], torch.broadcast_to(tol, ok.shape)[~ok][:4], int((~ok).sum()))


def check(x, targets, got, n_top=0, scale=1.0):
    t, v = x.shape
    step = max(1, (1 << 24) // v)
    for i in range(0, t, step):
        n = slice(i, min(t, i + step))
        ref = Ref(x[n], scale)
        assert torch.equal(got["stats"][n, :1].double(), ref.top)
        close(got["stats"][n, 1:], ref.log_sum, ref.t_log_sum)
        close(got["entropy"][n], ref.entropy, ref.t_entropy)
        if targets is not None:
            tgt = targets[n].long()[:, None]
            lp, tol = ref.logp(tgt.clamp(min=0))
            close(got["logp"][n], torch.where(tgt >= 0, lp, 0.0), tol)
        if n_top:
            idx = torch.sort(x[n].float() + 0.0, dim=1, descending=True, stable=True).indices[:, :n_top]
            assert torch.equal(got["top_idx"][n].long(), idx)
            lp, tol = ref.logp(idx)
            close(got["top_logp"][n], lp, tol)


# ------------------------------------------------------------------- forward
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,vocab,n_top", [
    (1, 1, 1), (3, 2, 2), (2, 7, 7), (5, 31, 20), (4, 33, 32), (1, 128, 8), (3, 1000, 20), (7, 1025, 1), (2, 4097, 32),
    (1, 32003, 5), (33, 32003, 20), (1, 65536, 8), (9, 65537, 32), (2, 100003, 20), (160, 50001, 5), (700, 8192, 3),
    (1300, 513, 8), (1, 262147, 20), (2, 3000001, 32), (64, 131072, 0)])
def test_shapes(ctx, tokens, vocab, n_top, dtype):
    x, targets = logits_of(tokens, vocab, dtype)
    check(x, targets, forward(ctx, x, targets, n_top), n_top)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("off", [1, 2, 3, 5, 7])
@pytest.mark.parametrize("tokens,vocab", [(3, 1000), (2, 70003)])
def test_rows_off_the_boundary(ctx, tokens, vocab, off, dtype):
    x, targets = logits_of(tokens, vocab, dtype, off=off)
    check(x, targets, forward(ctx, x, targets, 20), 20)


@pytest.mark.parametrize("scale", [0.25, 0.7, 1.25, 8.0])
def test_temperatures(ctx, scale):
    for vocab in (777, 65536):
        x, targets = logits_of(6, vocab, torch.float32, seed=2)
        check(x, targets, forward(ctx, x, targets, 5, scale), 5, scale)


def test_likely_tokens_keep_their_digits(ctx):
    # one token far above the rest: log p and the entropy are tiny and right to their last digits; a
    # common offset of the row changes nothing
    x, _ = logits_of(8, 40000, torch.float32, seed=3, spread=1.0)
    where = torch.arange(8, device="cuda") * 4999
    x[torch.arange(8), where] += torch.tensor([14.0, 18, 22, 26, 30, 40, 60, 90], device="cuda")
    x[4:] = torch.round(x[4:] * 64) / 64 + 4096.0
    targets = where.to(torch.int32)
    got = forward(ctx, x, targets, 8)
    check(x, targets, got, 8)
    assert -1e-11 < float(got["logp"][5]) < 0 and 0 < float(got["entropy"][5]) < 1e-10


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [50, 1000, 32003, 100003])
def test_ties_go_to_the_lowest_index(ctx, vocab, dtype):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = torch.zeros(6, vocab, device="cuda")
    x[1] = torch.randint(-1, 2, (vocab,), generator=g, device="cuda").float()
    x[2] = torch.randint(-3, 3, (vocab,), generator=g, device="cuda").float() * 0.5
    x[3] = torch.where(torch.rand(vocab, generator=g, device="cuda") < 0.5, 0.0, -0.0)
    x[4] = torch.arange(vocab, device="cuda") / vocab           # rising
    x[5] = -torch.arange(vocab, device="cuda") / vocab          # falling
    x = x.to(dtype)
    targets = torch.full((6,), vocab - 1, dtype=torch.int32, device="cuda")
    n_top = 32
    check(x, targets, forward(ctx, x, targets, n_top), n_top)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [40, 5000, 100003])
def test_masked_rows(ctx, vocab, dtype):
    low = -float("inf")
    x, targets = logits_of(7, vocab, dtype, seed=4)
    keep = x.clone()
    x[0, 1:] = low                     # one token left
    x[1, : vocab - 3] = low            # three, at the end
    x[2, ::2] = low
    x[3] = low                         # none
    x[4] = torch.finfo(dtype).min      # the type's lowest value is a logit like another
    x[5, : vocab // 2] = torch.finfo(dtype).min
    targets = torch.tensor([0, vocab - 1, 0, 3, 5, vocab - 1, 9], dtype=torch.int32, device="cuda")
    got = forward(ctx, x, targets, 20)
    rows = [0, 1, 2, 4, 5, 6]
    check(x[rows], targets[rows], {k: v[rows] for k, v in got.items()}, 20)
    assert float(got["logp"][2]) == low and torch.equal(x[6], keep[6])
    assert float(got["logp"][3]) == low and float(got["entropy"][3]) == 0
    assert got["stats"][3].tolist() == [low, 0.0]
    assert got["top_idx"][3].tolist() == list(range(20)) and (got["top_logp"][3] == low).all()


@pytest.mark.parametrize("vocab", [40, 40000])
def test_infinite_and_nan_rows(ctx, vocab):
    x, targets = logits_of(6, vocab, torch.float32, seed=5)
    x[0, 11] = float("nan")
    x[1] = float("nan")
    x[2, 13] = float("inf")
    x[3, 17] = -float("nan")
    x[4] = float("inf")
    got = forward(ctx, x, targets, 8)
    for k in ("logp", "entropy", "top_logp"):
        v = got[k].view(6, -1)[:5]
        assert torch.isnan(v[:, 0]).all(), k
    assert (got["top_idx"] >= 0).all() and (got["top_idx"] < vocab).all()
    check(x[5:], targets[5:], {k: v[5:] for k, v in got.items()}, 8)
    # and their gradients
    g = torch.ones(6, device="cuda")
    dx = torch.empty_like(x)
    qec.moe_token_logprobs_grad(ctx, x, targets, 6, vocab, got["stats"], got["entropy"], g, g, dx)
    assert torch.isnan(dx[:5]).any(1).all() and torch.isfinite(dx[5]).all()


def test_outputs_one_by_one_and_rows_behind(ctx):
    x, targets = logits_of(5, 3001, torch.float32, seed=6)
    want = forward(ctx, x, targets, 4)
    got = forward(ctx, x, targets, 4, extra=2)
    for k in want:
        assert torch.equal(got[k][:5], want[k]) and (got[k][5:] == 7).all(), k
    for k in ("logp", "entropy", "stats"):
        one = {n: None for n in ("logp", "entropy", "stats")}
        one[k] = torch.full_like(want[k], 7)
        qec.moe_token_logprobs(ctx, x, targets, 5, 3001, one["logp"], one["entropy"], stats=one["stats"])
        assert torch.equal(one[k], want[k]), k
    idx, lp = torch.empty(5, 4, dtype=torch.int32, device="cuda"), torch.empty(5, 4, device="cuda")
    qec.moe_token_logprobs(ctx, x, None, 5, 3001, None, None, 4, idx, lp)
    assert torch.equal(idx, want["top_idx"]) and torch.equal(lp, want["top_logp"])
    qec.moe_token_logprobs(ctx, None, None, 0, 3001, None, dtype=qec.F32)


def test_targets_without_a_token(ctx):
    x, targets = logits_of(6, 501, torch.float32, seed=7)
    targets[1], targets[4] = -1, -100
    got = forward(ctx, x, targets)
    check(x, targets, got)
    assert float(got["logp"][1]) == 0 and float(got["logp"][4]) == 0
    qec.miss_drain(ctx)  # nothing to report
    targets[2] = 501
    again = forward(ctx, x, targets)
    assert float(again["logp"][2]) == 0
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(again["logp"][keep], got["logp"][keep])
    with pytest.raises(qec.MoeError, match="target id") as err:
        qec.miss_drain(ctx)
    assert err.value.code == -8
    dx = torch.empty_like(x)
    qec.moe_token_logprobs_grad(ctx, x, targets, 6, 501, got["stats"], None, torch.ones(6, device="cuda"), None, dx)
    assert (dx[[1, 2, 4]] == 0).all()
    with pytest.raises(qec.MoeError, match="target id"):
        qec.miss_drain(ctx)
    qec.miss_drain(ctx)


# ------------------------------------------------------------------ gradient
def grad(ctx, x, targets, got, g, gh, scale=1.0, into=None, stream=None):
    dx = torch.full_like(x, 7) if into is None else into
    qec.moe_token_logprobs_grad(ctx, x, targets, x.shape[0], x.shape[1], got["stats"],
                                got["entropy"] if gh is not None else None, g, gh, dx, scale=scale, stream=stream)
    return dx


def check_grad(x, targets, got, g, gh, dx, scale=1.0):
    t, v = x.shape
    step = max(1, (1 << 24) // v)
    for i in range(0, t, step):
        n = slice(i, min(t, i + step))
        st = got["stats"][n].double()
        d = (st[:, :1] - x[n].double()) * scale
        lp = -d - st[:, 1:]
        p = torch.exp(lp)
        gt = torch.zeros(lp.shape[0], 1, dtype=torch.float64, device="cuda")
        hit = torch.zeros_like(lp)
        if g is not None:
            tgt = targets[n].long()[:, None]
            gt = torch.where(tgt >= 0, g[n].double()[:, None], 0.0)
            hit.scatter_(1, tgt.clamp(min=0), (tgt >= 0).double())
        live = p > 0
        lpz, dz = torch.where(live, lp, 0.0), torch.where(live, d, 0.0)
        g2 = torch.zeros_like(gt) if gh is None else gh[n].double()[:, None]
        h = torch.zeros_like(gt) if gh is None else got["entropy"][n].double()[:, None]
        ref = scale * (gt * (hit - p) - g2 * p * (lpz + h))
        rel = (3 * dz + 3 * lpz.abs() + 14) * U
        tol = scale * (p * (gt.abs() + g2.abs() * (lpz + h).abs()) * rel
                       + p * g2.abs() * (3 * dz + 2 * lpz.abs() + h) * U + gt.abs() * hit * (1 - p).abs() * 4 * U)
        tol = tol + (ref.abs() + tol) * torch.finfo(x.dtype).eps / 2 + torch.finfo(x.dtype).smallest_normal * (
            torch.finfo(x.dtype).eps if x.dtype == torch.float16 else 1.0)
        close(dx[n], ref, tol)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,vocab,off", [(1, 1, 0), (3, 7, 0), (2, 33, 1), (5, 1000, 0), (4, 4095, 3),
                                              (33, 32003, 0), (2, 100003, 5), (300, 513, 0), (1, 262147, 0)])
def test_gradients(ctx, tokens, vocab, off, dtype):
    x, targets = logits_of(tokens, vocab, dtype, seed=8, off=off)
    targets[tokens // 2] = -1
    gen = torch.Generator(device="cuda").manual_seed(vocab)
    g, gh = torch.randn(tokens, generator=gen, device="cuda"), torch.randn(tokens, generator=gen, device="cuda")
    for scale in (1.0, 0.7):
        got = forward(ctx, x, targets, scale=scale)
        for a, b in ((g, gh), (g, None), (None, gh)):
            dx = grad(ctx, x, targets if a is not None else None, got, a, b, scale)
            check_grad(x, targets, got, a, b, dx, scale)
    # aligned otherwise than the logits
    flat = torch.full((tokens * vocab + 1,), 7.0, dtype=dtype, device="cuda")
    assert torch.equal(grad(ctx, x, targets, got, g, None, 0.7, into=flat[1:].view(tokens, vocab)),
                       grad(ctx, x, targets, got, g, None, 0.7))
    assert float(flat[0]) == 7
    # and in the logits' own place
    want = grad(ctx, x, targets, got, g, gh, 0.7)
    assert torch.equal(grad(ctx, x, targets, got, g, gh, 0.7, into=x), want) and torch.equal(x, want)


def test_gradient_of_likely_and_masked_tokens(ctx):
    x, _ = logits_of(4, 5000, torch.float32, seed=9, spread=1.0)
    x[0, 100] += 40
    x[1, 100] += 18
    x[2, ::3] = -float("inf")
    x[3] = -float("inf")
    targets = torch.tensor([100, 100, 1, 2], dtype=torch.int32, device="cuda")
    got = forward(ctx, x, targets)
    g, gh = torch.full((4,), 2.0, device="cuda"), torch.full((4,), 1e30, device="cuda")
    dx = grad(ctx, x, targets, got, g, None)
    check_grad(x[:3], targets[:3], {k: v[:3] for k, v in got.items()}, g[:3], None, dx[:3])
    assert 0 < float(dx[0, 100]) < 1e-10 and (dx[3] == 0).all() and (dx[2, ::3] == 0).all()
    assert (grad(ctx, x, targets, got, g, gh)[2, ::3] == 0).all()


def test_gradient_against_differences(ctx):
    # along a direction v: (f(x + h v) - f(x - h v)) / 2h in 64 bits, whose error is h^2 |f'''| / 6 and
    # rounding 1e-16 f / h: below 1e-7 of |v| at h = 1e-4
    x, targets = logits_of(5, 801, torch.float32, seed=10)
    g, gh = torch.randn(5, device="cuda"), torch.randn(5, device="cuda")
    got = forward(ctx, x, targets, scale=1.25)
    dx = grad(ctx, x, targets, got, g, gh, 1.25).double()

    def f(z):
        lp = torch.log_softmax(z * 1.25, 1)
        return ((lp.gather(1, targets.long()[:, None]).squeeze(1) * g.double()).sum()
                + (torch.special.entr(lp.exp()).sum(1) * gh.double()).sum())

    for seed in range(6):
        v = torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").double()
        h = 1e-4
        slope = float((f(x.double() + h * v) - f(x.double() - h * v)) / (2 * h))
        # fp32 gradients: 60 u of the sum of their absolute parts
        assert abs(slope - float((dx * v).sum())) <= 1e-6 * float((dx.abs() * v.abs()).sum() + 1)


# ------------------------------------------------------- streams, graphs, sizes
def test_other_streams_and_graphs(ctx):
    x, targets = logits_of(9, 33001, torch.bfloat16, seed=11)
    y, other = logits_of(9, 33001, torch.bfloat16, seed=12)
    g = torch.randn(9, device="cuda")
    want = [(forward(ctx, z, t, 8), grad(ctx, z, t, forward(ctx, z, t), g, None)) for z, t in ((x, targets), (y, other))]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = forward(ctx, x, targets, 8, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[0][0][k]) for k in got)
    zin, tin, dx = x.clone(), targets.clone(), torch.empty_like(x)
    out = {k: torch.empty_like(v) for k, v in got.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            qec.moe_token_logprobs(ctx, zin, tin, 9, 33001, out["logp"], out["entropy"], 8, out["top_idx"],
                                   out["top_logp"], out["stats"], stream=s)
            qec.moe_token_logprobs_grad(ctx, zin, tin, 9, 33001, out["stats"], None, g, None, dx, stream=s)
    for z, t, (f, d) in ((x, targets, want[0]), (y, other, want[1]), (x, targets, want[0])):
        zin.copy_(z)
        tin.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], f[k]) for k in out) and torch.equal(dx, d)


@pytest.mark.parametrize("tokens,vocab", [(3, 65536), (700, 32003)])
def test_the_same_inputs_give_the_same_bits(ctx, tokens, vocab):
    x, targets = logits_of(tokens, vocab, torch.float32, seed=13)
    want = forward(ctx, x, targets, 20)
    for _ in range(4):
        got = forward(ctx, x, targets, 20)
        assert all(torch.equal(got[k], want[k]) for k in got)


def test_more_than_2_31_elements(ctx):
    tokens, vocab = 33000, 65537
    x = torch.zeros(tokens, vocab, dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, 32767, 32768, tokens - 1]
    g = torch.Generator(device="cuda").manual_seed(14)
    for r in rows:
        x[r] = torch.randn(vocab, generator=g, device="cuda").bfloat16()
    targets = torch.full((tokens,), vocab - 1, dtype=torch.int32, device="cuda")
    got = forward(ctx, x, targets, 5)
    check(x[rows], targets[rows], {k: v[rows] for k, v in got.items()}, 5)
    assert torch.allclose(got["logp"][5], torch.tensor(-math.log(vocab), device="cuda"), rtol=1e-5)
    w = torch.ones(tokens, device="cuda")
    dx = grad(ctx, x, targets, got, w, None, into=x.clone())
    check_grad(x[rows], targets[rows], {k: v[rows] for k, v in got.items()}, w[rows], None, dx[rows])


def test_refusals(ctx):
    x, targets = logits_of(3, 100, torch.float32)
    out = torch.empty(3, device="cuda")
    with pytest.raises(ValueError):
        qec.moe_token_logprobs(ctx, x, targets.long(), 3, 100, out)
    with pytest.raises(ValueError):
        qec.moe_token_logprobs(ctx, x.double(), targets, 3, 100, out)
    with pytest.raises(ValueError):
        qec.moe_token_logprobs(ctx, x.t(), targets, 100, 3, out)
    with pytest.raises(ValueError):
        qec.moe_token_logprobs_grad(ctx, x, targets, 3, 100, out, None, out, None, x.half())
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(n_top=33), dict(n_top=-1), dict(n_top=2)):
        with pytest.raises(qec.MoeError):
            qec.moe_token_logprobs(ctx, x, targets, 3, 100, out, **bad)
    with pytest.raises(qec.MoeError):
        qec.moe_token_logprobs(ctx, x, None, 3, 100, out)
    assert np.isfinite(x.cpu().numpy()).all()
