"""GPU test of the operators as a tuner of a router and an output head uses them
together: norm, the router as a 16-bit dense layer, top-k, the router's losses with
their gradient, the head, the targets' log probabilities with their gradient, and both
layers' gradients down to the normed rows.  One captured graph holds the whole step;
its results are held against automatic differentiation of the definitions in 64 bits.

Tolerances: every value passes at most eight operators, each within 1e-5 of its 2-norm
where its results are fp32 (the operators' own tests hold them closer), 2^-8 where they
are bfloat16 and so is what they read."""
import pytest

import quantized_expert_cache_gb300 as qec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
EPS, BALANCE, ZLOSS, H_COEF = 1e-6, 0.01, 0.001, 0.02


class Step:
    def __init__(self, tokens, hidden, experts, k, vocab, seed, stream):
        self.T, self.H, self.E, self.k, self.V, self.stream = tokens, hidden, experts, k, vocab, stream
        self.ctx = qec.moe_layer_init(hidden, 32, experts, k, 1, 0, tokens, stream=stream.cuda_stream)
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        empty = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.x, self.norm = rand(tokens, hidden), 1 + 0.1 * rand(hidden)
        self.router, self.bias = (rand(experts, hidden) / hidden ** 0.5).bfloat16(), 0.1 * rand(experts)
        self.head = (rand(vocab, hidden) / hidden ** 0.5).bfloat16()
        self.targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda", dtype=torch.int32)
        self.targets[::5] = -1
        self.g_logp, self.g_h = -1.0 / tokens * torch.ones(tokens, device="cuda"), torch.full(
            (tokens,), -H_COEF / tokens, device="cuda")
        self.y = empty(tokens, hidden)
        self.z, self.dz = empty(tokens, experts), empty(tokens, experts)
        self.idx, self.w = empty(tokens, k, dtype=torch.int32), empty(tokens, k)
        self.loss, self.counts = empty(2), empty(experts, dtype=torch.int32)
        self.logits = empty(tokens, vocab)
        self.logp, self.entropy, self.stats = empty(tokens), empty(tokens), empty(tokens, 2)
        self.dx_r, self.dx_h = empty(tokens, hidden), empty(tokens, hidden)
        self.dw_r, self.db_r, self.dw_h = empty(experts, hidden), empty(experts), empty(vocab, hidden)
        need = [qec.moe_dense_workspace(self.ctx, self.y, self.router, self.z, 0, tokens, r, hidden)
                for r in (experts, vocab)]
        self.ws = empty(max(max(n) for n in need) + 16, dtype=torch.uint8)

    def run(self):
        c, t, s = self.ctx, self.T, self.stream
        qec.moe_rms_norm(c, self.x, None, self.norm, t, self.H, EPS, None, self.y, stream=s)
        qec.moe_dense_forward(c, self.y, self.router, t, self.E, self.H, self.z, bias=self.bias, ws=self.ws, stream=s)
        qec.route_topk(c, self.z, t, self.E, self.k, self.idx, self.w, stream=s)
        qec.moe_router_loss(c, self.z, self.idx, None, None, t, self.E, self.k, BALANCE, ZLOSS, self.loss, self.counts,
                            self.dz, stream=s)
        qec.moe_dense_forward(c, self.y, self.head, t, self.V, self.H, self.logits, ws=self.ws, stream=s)
        qec.moe_token_logprobs(c, self.logits, self.targets, t, self.V, self.logp, self.entropy, stats=self.stats,
                               stream=s)
        # the logits' own place holds their gradient
        qec.moe_token_logprobs_grad(c, self.logits, self.targets, t, self.V, self.stats, self.entropy, self.g_logp,
                                    self.g_h, self.logits, stream=s)
        qec.moe_dense_backward(c, self.y, self.router, self.dz, t, self.E, self.H, self.dx_r, self.dw_r, self.db_r,
                               ws=self.ws, stream=s)
        qec.moe_dense_backward(c, self.y, self.head, self.logits, t, self.V, self.H, self.dx_h, self.dw_h, ws=self.ws,
                               stream=s)

    def want(self):
        """The same in 64 bits, by automatic differentiation."""
        x, w = self.x.double(), self.norm.double()
        y = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * w
        yr, yh = y.clone().requires_grad_(), y.clone().requires_grad_()
        router, head = self.router.double().requires_grad_(), self.head.double().requires_grad_()
        bias = self.bias.double().requires_grad_()
        z = yr @ router.t() + bias
        p, lse = torch.softmax(z, 1), torch.logsumexp(z, 1)
        counts = torch.bincount(torch.topk(z, self.k, 1).indices.reshape(-1), minlength=self.E).double()
        loss = (BALANCE * self.E * (p.mean(0) * counts / (self.T * self.k)).sum(), ZLOSS * (lse * lse).mean())
        (loss[0] + loss[1]).backward()
        lp = torch.log_softmax(yh @ head.t(), 1)
        tgt = self.targets.long()
        logp = torch.where(tgt >= 0, lp.gather(1, tgt.clamp(min=0)[:, None]).squeeze(1), 0.0)
        entropy = torch.special.entr(lp.exp()).sum(1)
        ((logp * self.g_logp.double()).sum() + (entropy * self.g_h.double()).sum()).backward()
        return dict(z=z, loss=torch.stack(loss), counts=counts, logp=logp, entropy=entropy, dx_r=yr.grad,
                    dw_r=router.grad, db_r=bias.grad, dx_h=yh.grad, dw_h=head.grad)

    def check(self):
        torch.cuda.synchronize()
        for name, ref in self.want().items():
            got, ref = getattr(self, name).double(), ref.detach()
            if name == "counts":
                assert torch.equal(got, ref)
                continue
            err = torch.linalg.vector_norm(got - ref) / torch.linalg.vector_norm(ref)
            assert float(err) <= 8e-5, (name, float(err))
        qec.miss_drain(self.ctx)  # (no wait expired, no id out of range)


@pytest.mark.parametrize("tokens,hidden,experts,k,vocab", [(3, 64, 8, 2, 501), (33, 256, 8, 2, 1000),
                                                           (200, 2048, 512, 8, 5003), (1000, 576, 129, 4, 777)])
def test_a_tuning_step(tokens, hidden, experts, k, vocab):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step = Step(tokens, hidden, experts, k, vocab, tokens, s)
        step.run()
    step.check()
    first = {n: getattr(step, n).clone() for n in ("z", "logp", "dx_r", "dw_r", "db_r", "dx_h", "dw_h")}
    # captured once, replayed on new rows and on the old ones
    graph, old = torch.cuda.CUDAGraph(), step.x.clone()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            step.run()
        step.x.copy_(torch.randn(tokens, hidden, generator=torch.Generator(device="cuda").manual_seed(7), device="cuda"))
        graph.replay()
    step.check()
    with torch.cuda.stream(s):
        step.x.copy_(old)
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(getattr(step, n), v) for n, v in first.items())
    qec.moe_destroy(step.ctx)


def test_the_example_answers_with_log_probabilities(capsys):
    import os
    import sys

    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    from decoder_stack import DecoderStack

    stack = DecoderStack(slots=8)
    x = torch.randn(5, stack.H, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    logits = stack.step(x).clone()
    tokens = torch.tensor([4, 0, 999, -1, 17], dtype=torch.int32, device="cuda")
    logp, entropy, idx, alternatives = stack.answer(tokens, 6)
    lp = torch.log_softmax(logits.double(), 1)
    want = lp.gather(1, tokens.long().clamp(min=0)[:, None]).squeeze(1) * (tokens >= 0)
    top = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :6]
    assert torch.equal(idx.long(), top)
    # fp32 sums over 1000 logits: (1000 / 256 + 60) 2^-24 of values up to 20
    for got, ref in ((logp, want), (entropy, torch.special.entr(lp.exp()).sum(1)), (alternatives, lp.gather(1, top))):
        assert ((got.double() - ref).abs() <= 1e-4 * (ref.abs() + 1)).all()
    stack.close()


FIRST = """
import torch
import quantized_expert_cache_gb300 as qec
t, r, c = 100, 520, 264
st = torch.cuda.Stream()
ctx = qec.moe_layer_init(64, 32, 8, 2, 1, 0, 1, stream=st.cuda_stream)
g = torch.Generator(device="cuda").manual_seed(1)
x, w = torch.randn(t, c, generator=g, device="cuda"), (torch.randn(r, c, generator=g, device="cuda") / 16).bfloat16()
y, dx, dw, db = (torch.empty(n, device="cuda") for n in ((t, r), (t, c), (r, c), (r,)))
logp, stats = torch.empty(t, device="cuda"), torch.empty(t, 2, device="cuda")
targets = torch.arange(t, dtype=torch.int32, device="cuda")
ws = torch.empty(max(qec.moe_dense_workspace(ctx, x, w, y, 0, t, r, c)), dtype=torch.uint8, device="cuda")
one = torch.ones(t, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.stream(st):
    with torch.cuda.graph(graph, stream=st):
        qec.moe_dense_forward(ctx, x, w, t, r, c, y, ws=ws, stream=st)
        qec.moe_token_logprobs(ctx, y, targets, t, r, logp, None, 0, None, None, stats, stream=st)
        qec.moe_token_logprobs_grad(ctx, y, targets, t, r, stats, None, one, None, y, stream=st)
        qec.moe_dense_backward(ctx, x, w, y, t, r, c, dx, dw, db, ws=ws, stream=st)
    graph.replay()
torch.cuda.synchronize()
xd, wd = x.double().requires_grad_(), w.double().requires_grad_()
lp = torch.log_softmax(xd @ wd.t(), 1).gather(1, targets.long()[:, None]).squeeze(1)
lp.sum().backward()
for got, ref in ((logp, lp), (dx, xd.grad), (dw, wd.grad)):
    assert float(torch.linalg.vector_norm(got.double() - ref) / torch.linalg.vector_norm(ref)) <= 8e-5
qec.moe_destroy(ctx)
print("first in a graph")
"""


def test_a_process_may_capture_its_first_calls():
    # nothing that a call sets up on first use may break a capture
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "first in a graph" in done.stdout, done.stderr[-2000:]
