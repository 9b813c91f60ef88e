"""GPU tests of moe_token_logprobs and its gradient at the ends of the scale's range, where
every value has a closed form."""
import math

import pytest

import quantized_expert_cache_gb300 as qec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = qec.moe_layer_init(64, 32, 8, 2, 1, 0, 1, stream=torch.cuda.current_stream().cuda_stream)
    yield c
    torch.cuda.synchronize()
    qec.moe_destroy(c)


def run(ctx, x, targets, scale):
    t, v = x.shape
    logp, entropy, stats = (torch.full(s, 7.0, device="cuda") for s in ((t,), (t,), (t, 2)))
    idx, top = torch.full((t, 2), 7, dtype=torch.int32, device="cuda"), torch.full((t, 2), 7.0, device="cuda")
    qec.moe_token_logprobs(ctx, x, targets, t, v, logp, entropy, 2, idx, top, stats, scale=scale)
    dx = torch.full_like(x, 7.0)
    one = torch.ones(t, device="cuda")
    qec.moe_token_logprobs_grad(ctx, x, targets, t, v, stats, entropy, one, one, dx, scale=scale)
    return logp, entropy, idx, top, dx


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("vocab", [40, 5000, 70003])
def test_the_largest_scale_takes_the_largest_logit(ctx, vocab, dtype):
    # all but the largest are at probability 0, also next to logits of the type's lowest value
    t = 3
    x = torch.rand(t, vocab, generator=torch.Generator(device="cuda").manual_seed(vocab), device="cuda").to(dtype)
    best = [0, vocab // 2, vocab - 1]
    for row, i in enumerate(best):
        x[row, i] = 2
    x[1, 1:5] = torch.finfo(dtype).min
    targets = torch.tensor([best[0], best[1], 3], dtype=torch.int32, device="cuda")
    logp, entropy, idx, top, dx = run(ctx, x, targets, 2.0 ** 127)
    assert logp[0] == 0 and logp[1] == 0
    assert (entropy == 0).all() and idx[:, 0].tolist() == best
    assert (top[:, 0] == 0).all()
    # the others' are 2^127 times a difference rounded once, where fp32 holds that
    for got, ref in ((logp[2], x[2, 3]), *((top[i, 1], x[i, idx[i, 1]]) for i in range(t))):
        ref = (float(ref) - 2) * 2.0 ** 127
        assert float(got) == -math.inf if ref <= -(2.0 ** 128) else abs(float(got) - ref) <= abs(ref) * 2.0 ** -24
    assert not dx[:2].any()


@pytest.mark.parametrize("vocab", [40, 5000, 70003])
def test_the_smallest_scale_takes_all_alike(ctx, vocab):
    t = 3
    x = torch.randn(t, vocab, generator=torch.Generator(device="cuda").manual_seed(vocab), device="cuda")
    targets = torch.tensor([0, 1, vocab - 1], dtype=torch.int32, device="cuda")
    logp, entropy, idx, top, dx = run(ctx, x, targets, 2.0 ** -149)
    # terms of 1 but for a step of 2^-24 each, sums of V/256 + 40 additions, log1p's 2 ulp (4 u)
    tol = 2.0 ** -24 * (4 + vocab / 256 + 40 + 4 * math.log(vocab))
    for v in (logp, top):
        assert float((v.double() + math.log(vocab)).abs().max()) <= tol
    assert float((entropy.double() - math.log(vocab)).abs().max()) <= tol
    assert torch.equal(idx.long(), torch.topk(x, 2, 1).indices)
    assert float(dx.abs().max()) <= 2.0 ** -148


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** 120])
def test_gradients_that_are_no_numbers(ctx, scale, dtype):
    # NaN and infinities of the outputs' gradients spread over their rows, also to logits at
    # probability 0 (0 times them); a row of nothing but -infinity stays at zero
    t, v = 6, 1000
    x = torch.randn(t, v, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").to(dtype)
    x[:, ::7] = -math.inf
    x[4] = -math.inf
    x[:4, 1] = 8
    targets = torch.tensor([1, 2, 3, 1, 1, 1], dtype=torch.int32, device="cuda")
    logp, entropy, stats = (torch.empty(s, device="cuda") for s in ((t,), (t,), (t, 2)))
    qec.moe_token_logprobs(ctx, x, targets, t, v, logp, entropy, stats=stats, scale=scale)
    nan = float("nan")
    g = torch.tensor([nan, 1.0, math.inf, 1.0, nan, 1.0], device="cuda")
    gh = torch.tensor([1.0, nan, 1.0, 1.0, 1.0, 1.0], device="cuda")
    dx = torch.full_like(x, 7.0)
    qec.moe_token_logprobs_grad(ctx, x, targets, t, v, stats, entropy, g, gh, dx, scale=scale)
    assert torch.isnan(dx[:2]).all() and not torch.isfinite(dx[2]).any() and torch.isnan(dx[2, ::7]).all()
    assert not dx[4].any()
    assert not dx[3, ::7].any() and not dx[5, ::7].any()
    assert torch.isfinite(dx[3]).all()
