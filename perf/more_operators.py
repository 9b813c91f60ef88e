"""Cases of the operators around the vocabulary and the 16-bit dense layers: log
probabilities of given tokens with entropy and top alternatives, their gradient
to the logits, the product with bias, activation and residual, and its gradients.

listed() gives the measured cases and draw() more of the same ranges; run()
makes one pass, in plain torch operations (own = False) or through the library
(own = True); exact() is the same result from the definition in 64 bits.
Shapes are those of the repository's workloads (hidden 2048 with 512 experts;
hidden 2880; prompts of 4096 tokens; decode batches of 1, 8 and 32) next to
generic ones.
"""
import math
import weakref

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decoded token: its log probability and eight alternatives for the answer
        dict(name="logprobs_t1", op="logprobs", tokens=1, vocab=65536, dtype="f32", top=8, scale=1.0, masked=False),
        # a decode batch with a grammar's mask on an odd vocabulary, 16-bit logits, a temperature
        dict(name="logprobs_t32_bf16", op="logprobs", tokens=32, vocab=100003, dtype="bf16", top=20, scale=1.25,
             masked=True),
        # a 4096-token prompt scored with five alternatives a position
        dict(name="logprobs_t4096", op="logprobs", tokens=4096, vocab=65536, dtype="f32", top=5, scale=1.0,
             masked=False),
        # the gradient of a short answer's log probabilities, padded, odd vocabulary
        dict(name="logprobs_grad_t33", op="logprobs_grad", tokens=33, vocab=32003, dtype="f32", scale=1.0,
             entropy=False),
        # a 4096-token training step with an entropy term on 16-bit logits
        dict(name="logprobs_grad_t4096_bf16", op="logprobs_grad", tokens=4096, vocab=65536, dtype="bf16", scale=1.0,
             entropy=True),
        # one token's router logits: fp32 rows of the norm, 512 experts, a bias for balance
        dict(name="dense_router_t1", op="dense", tokens=1, rows=512, cols=2048, x="f32", w="bf16", y="f32",
             bias=True, act="none", res=False, pre=False),
        # a decode batch's output head, fp32 logits
        dict(name="dense_head_t8", op="dense", tokens=8, rows=65536, cols=2048, x="bf16", w="bf16", y="f32",
             bias=False, act="none", res=False, pre=False),
        # a ragged batch of speculated tokens: odd rows, bias, activation and residual
        dict(name="dense_odd_t33", op="dense", tokens=33, rows=2887, cols=2880, x="f16", w="f16", y="f16",
             bias=True, act="gelu", res=True, pre=False),
        # a 4096-token prompt through a wide layer, what its gradient needs kept
        dict(name="dense_prompt_t4096", op="dense", tokens=4096, rows=8192, cols=2048, x="bf16", w="bf16", y="bf16",
             bias=True, act="silu", res=False, pre=True),
        # a router's training step: fp32 rows and the router loss's fp32 gradient
        dict(name="dense_grad_router_t4096", op="dense_grad", tokens=4096, rows=512, cols=2048, x="f32", w="bf16",
             y="f32", act="none", dw="f32"),
        # a ragged batch through an activation
        dict(name="dense_grad_t1000_f16", op="dense_grad", tokens=1000, rows=2880, cols=2880, x="f16", w="f16",
             y="f16", act="gelu", dw="f16"),
        # a 4096-token training step of a square layer, fp32 weight gradients
        dict(name="dense_grad_t4096", op="dense_grad", tokens=4096, rows=4096, cols=4096, x="bf16", w="bf16",
             y="bf16", act="none", dw="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs_grad", "dense", "dense_grad"])
    if op.startswith("logprobs"):
        vocab = _log(rng, 33, 200000)
        c = dict(op=op, tokens=_log(rng, 1, min(4096, 4096 * 65536 // 2 // vocab)), vocab=vocab,
                 dtype=rng.choice(["f32", "f32", "bf16", "f16"]), scale=rng.choice([1.0, 1.0, 0.7, 1.25]))
        if op == "logprobs":
            return dict(c, top=rng.choice([0, 1, 5, 8, 20, 32]), masked=rng.random() < 0.3)
        return dict(c, entropy=rng.random() < 0.5)
    w = rng.choice(["bf16", "bf16", "f16"])
    x = rng.choice(["f32", "bf16"]) if w == "bf16" else "f16"
    cols = _log(rng, 8, 512) * 8 if rng.random() < 0.8 else _log(rng, 8, 1024) * 8
    tokens = _log(rng, 1, 4096)
    rows = _log(rng, 8, min(65536, 2 ** 35 // (tokens * cols), 2 ** 27 // cols))
    act = rng.choice(["none", "none", "silu", "gelu"])
    if op == "dense":
        return dict(op=op, tokens=tokens, rows=rows, cols=cols, x=x, w=w, y=rng.choice(["f32", w]),
                    bias=rng.random() < 0.6, act=act, res=rng.random() < 0.4, pre=rng.random() < 0.3)
    return dict(op=op, tokens=tokens, rows=rows, cols=cols, x=x, w=w,
                y=rng.choice(["f32", "bf16"]) if w == "bf16" else "f16", act=act, dw=rng.choice(["f32", w]))


def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    t = case["tokens"]
    if case["op"] == "logprobs":
        n = t * case["vocab"]
        return dict(bytes=n * _size(case["dtype"]) + t * (4 + 4 + 4 + 8 + 8 * case["top"]), flops=6 * n)
    if case["op"] == "logprobs_grad":
        n = t * case["vocab"]
        return dict(bytes=2 * n * _size(case["dtype"]) + t * (4 + 4 + 8 + (8 if case["entropy"] else 0)), flops=6 * n)
    r, c = case["rows"], case["cols"]
    x, w, y = _size(case["x"]), _size(case["w"]), _size(case["y"])
    if case["op"] == "dense":
        moved = t * c * x + r * c * w + (4 * r if case["bias"] else 0)
        moved += t * r * y * (1 + (1 if case["res"] else 0) + (1 if case["pre"] else 0))
        return dict(bytes=moved, flops=2 * t * r * c)
    moved = 2 * t * c * x + r * c * (w + _size(case["dw"])) + 4 * r + t * r * y * (1 if case["act"] == "none" else 2)
    return dict(bytes=moved, flops=4 * t * r * c)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
class _Context:
    """A library context that goes with the state that holds it."""

    def __init__(self):
        import quantized_expert_cache_gb300 as qec

        self.qec = qec
        self.ctx = qec.moe_layer_init(64, 32, 8, 1, 1, 0, 1, stream=torch.cuda.current_stream().cuda_stream)
        weakref.finalize(self, qec.moe_destroy, self.ctx)


def _empty(dtype, *shape):
    return torch.empty(*shape, dtype=DTYPES.get(dtype, dtype), device="cuda")


def _logits(g, case):
    """A language model's: a popular head of the vocabulary, and a few likely tokens in each row."""
    t, v = case["tokens"], case["vocab"]
    pop = -0.7 * torch.log(torch.randperm(v, generator=g, device="cuda").float() + 1)
    z = torch.randn(t, v, generator=g, device="cuda").mul_(1.5).add_(pop)
    likely = torch.randint(0, v, (t, 4), generator=g, device="cuda")
    z.scatter_add_(1, likely, 4 + 3 * torch.randn(t, 4, generator=g, device="cuda"))
    targets = torch.where(torch.rand(t, generator=g, device="cuda") < 0.7, likely[:, 0],
                          torch.randint(0, v, (t,), generator=g, device="cuda")).to(torch.int32)
    if t > 1:  # padding carries no target
        targets[torch.rand(t, generator=g, device="cuda") < 0.1] = -1
    if case.get("masked"):
        off = torch.rand(t, v, generator=g, device="cuda") < 0.4
        off.scatter_(1, likely, False)
        off.scatter_(1, targets.long().clamp(min=0)[:, None], False)
        z.masked_fill_(off, float("-inf"))
    return z.to(DTYPES[case["dtype"]]), targets


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    t = case["tokens"]
    if own:
        s["c"] = _Context()
    if case["op"].startswith("logprobs"):
        v = case["vocab"]
        s["logits"], s["targets"] = _logits(g, case)
        if case["op"] == "logprobs":
            if own:
                s["logp"], s["entropy"], s["stats"] = _empty("f32", t), _empty("f32", t), _empty("f32", t, 2)
                s["top_idx"], s["top_logp"] = _empty(torch.int32, t, case["top"]), _empty("f32", t, case["top"])
            return s
        # what the forward pass kept: the row's largest logit and the log of the sum relative to it, the entropy
        s["stats"], s["entropy"] = _empty("f32", t, 2), _empty("f32", t)
        for i in range(0, t, 256):
            z = s["logits"][i:i + 256].float()
            m = z.amax(1, keepdim=True)
            z = (z - m) * case["scale"]
            e = torch.exp(z)
            tot = e.sum(1, keepdim=True)
            s["stats"][i:i + 256] = torch.cat([m, torch.log(tot)], 1)
            s["entropy"][i:i + 256] = (torch.log(tot) - (e * z).sum(1, keepdim=True) / tot).squeeze(1)
        # advantages over the tokens of the batch
        s["g_logp"] = torch.randn(t, generator=g, device="cuda") / t
        s["g_entropy"] = torch.full((t,), -0.01 / t, device="cuda") if case["entropy"] else None
        if own:
            s["dlogits"] = _empty(case["dtype"], t, v)
        return s
    r, c = case["rows"], case["cols"]
    x, w, y = DTYPES[case["x"]], DTYPES[case["w"]], DTYPES[case["y"]]
    # a few channels of a layer's input are larger than the rest
    s["x"] = (torch.randn(t, c, generator=g, device="cuda") * torch.exp(
        0.5 * torch.randn(c, generator=g, device="cuda"))).to(x)
    s["w"] = (torch.randn(r, c, generator=g, device="cuda") / math.sqrt(c)).to(w)
    if case["op"] == "dense":
        s["bias"] = 0.3 * torch.randn(r, generator=g, device="cuda") if case["bias"] else None
        s["res"] = torch.randn(t, r, generator=g, device="cuda").to(y) if case["res"] else None
        if own:
            s["y"] = _empty(y, t, r)
            s["pre"] = _empty(y, t, r) if case["pre"] else None
    else:
        s["pre"] = None if case["act"] == "none" else (
            1.2 * torch.randn(t, r, generator=g, device="cuda")).to(y)
        s["dy"] = (torch.randn(t, r, generator=g, device="cuda") * (1e-3 if case["y"] == "f32" else 1e-2)).to(y)
        if own:
            s["dx"], s["dw"], s["db"] = _empty(x, t, c), _empty(case["dw"], r, c), _empty("f32", r)
    if own:
        q = s["c"].qec
        need = q.moe_dense_workspace(s["c"].ctx, s["x"], s["w"], y, _act(q, case), t, r, c)
        s["ws"] = _empty(torch.uint8, max(1, need[0 if case["op"] == "dense" else 1]))
    return s


def _act(qec, case):
    return dict(none=qec.ACT_NONE, silu=qec.ACT_SILU, gelu=qec.ACT_GELU)[case["act"]]


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if own:
        return _OWN[case["op"]](s, case, s["c"].qec, s["c"].ctx)
    return _PLAIN[case["op"]](s, case)


def _own_logprobs(s, case, q, ctx):
    top = case["top"]
    q.moe_token_logprobs(ctx, s["logits"], s["targets"], case["tokens"], case["vocab"], s["logp"], s["entropy"],
                         top, s["top_idx"] if top else None, s["top_logp"] if top else None, s["stats"],
                         scale=case["scale"])
    return dict(logp=s["logp"], entropy=s["entropy"], top_idx=s["top_idx"], top_logp=s["top_logp"], stats=s["stats"])


def _own_logprobs_grad(s, case, q, ctx):
    q.moe_token_logprobs_grad(ctx, s["logits"], s["targets"], case["tokens"], case["vocab"], s["stats"], s["entropy"],
                              s["g_logp"], s["g_entropy"], s["dlogits"], scale=case["scale"])
    return s["dlogits"]


def _own_dense(s, case, q, ctx):
    q.moe_dense_forward(ctx, s["x"], s["w"], case["tokens"], case["rows"], case["cols"], s["y"], bias=s["bias"],
                        act=_act(q, case), res=s["res"], pre=s["pre"], ws=s["ws"])
    return dict(y=s["y"], pre=s["pre"])


def _own_dense_grad(s, case, q, ctx):
    q.moe_dense_backward(ctx, s["x"], s["w"], s["dy"], case["tokens"], case["rows"], case["cols"], s["dx"], s["dw"],
                         s["db"], act=_act(q, case), pre=s["pre"], ws=s["ws"])
    return dict(dx=s["dx"], dw=s["dw"], db=s["db"])


def _top(logits, k):
    """The k largest of each row, ties to the lowest index: one whole-number key orders both."""
    bits = (logits.float() + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() << 32
    key |= torch.arange(logits.shape[1] - 1, -1, -1, device=logits.device)
    best = torch.topk(key, k, dim=1).values
    return logits.shape[1] - 1 - (best & 0xFFFFFFFF)


def _plain_logprobs(s, case):
    z = s["logits"].float()
    m = z.amax(1, keepdim=True)
    z = (z - m) * case["scale"]
    e = torch.exp(z)
    tot = e.sum(1, keepdim=True)
    log_tot = torch.log(tot)
    tgt = s["targets"].long()[:, None]
    logp = torch.where(tgt >= 0, z.gather(1, tgt.clamp(min=0)) - log_tot, 0.0)
    entropy = log_tot - torch.where(e > 0, e * z, 0.0).sum(1, keepdim=True) / tot
    idx = _top(s["logits"], case["top"])
    return dict(logp=logp.squeeze(1), entropy=entropy.squeeze(1), top_idx=idx.to(torch.int32),
                top_logp=z.gather(1, idx) - log_tot, stats=torch.cat([m, log_tot], 1))


def _plain_logprobs_grad(s, case):
    logp = (s["logits"].float() - s["stats"][:, :1]) * case["scale"] - s["stats"][:, 1:]
    p = torch.exp(logp)
    tgt = s["targets"].long()[:, None]
    gt = torch.where(tgt >= 0, s["g_logp"][:, None], 0.0)
    if case["entropy"]:
        d = -p * (gt + s["g_entropy"][:, None] * (logp + s["entropy"][:, None]))
    else:
        d = -p * gt
    d = d.scatter_add(1, tgt.clamp(min=0), gt)
    return (d * case["scale"]).to(s["logits"].dtype)


def _plain_act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _plain_dense(s, case):
    z = s["x"].float() @ s["w"].float().t()
    if case["bias"]:
        z = z + s["bias"]
    y = _plain_act(z, case["act"])
    if case["res"]:
        y = y + s["res"].float()
    dt = DTYPES[case["y"]]
    return dict(y=y.to(dt), pre=z.to(dt) if case["pre"] else None)


def _plain_slope(z, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))


def _plain_dense_grad(s, case):
    dz = s["dy"].float()
    if case["act"] != "none":
        dz = dz * _plain_slope(s["pre"].float(), case["act"])
    return dict(dx=(dz @ s["w"].float()).to(s["x"].dtype), dw=(dz.t() @ s["x"].float()).to(DTYPES[case["dw"]]),
                db=dz.sum(0))


_OWN = dict(logprobs=_own_logprobs, logprobs_grad=_own_logprobs_grad, dense=_own_dense, dense_grad=_own_dense_grad)
_PLAIN = dict(logprobs=_plain_logprobs, logprobs_grad=_plain_logprobs_grad, dense=_plain_dense,
              dense_grad=_plain_dense_grad)


# --------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "logprobs":
        parts = [_exact_logprobs(s["logits"][i:i + 256], s["targets"][i:i + 256].long(), case)
                 for i in range(0, case["tokens"], 256)]
        return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if case["op"] == "logprobs_grad":
        out = torch.empty(case["tokens"], case["vocab"], dtype=torch.float64)
        for i in range(0, case["tokens"], 256):
            n = slice(i, i + 256)
            out[n] = _exact_logprobs_grad(s["logits"][n], s["targets"][n].long(), s["g_logp"][n],
                                          s["g_entropy"][n] if case["entropy"] else None, case).cpu()
        return out
    x, w = s["x"].double(), s["w"].double()
    if case["op"] == "dense":
        z = torch.matmul(x, w.mT)
        if s["bias"] is not None:
            z += s["bias"].double()
        y = dict(none=lambda v: v, silu=torch.nn.functional.silu, gelu=torch.nn.functional.gelu)[case["act"]](z)
        if s["res"] is not None:
            y = y + s["res"].double()
        return dict(y=y, pre=z if case["pre"] else None)
    dz = s["dy"].double()
    if case["act"] != "none":
        z = s["pre"].double().requires_grad_()
        y = (torch.nn.functional.silu if case["act"] == "silu" else torch.nn.functional.gelu)(z)
        dz, = torch.autograd.grad(y, z, dz)
    return dict(dx=torch.matmul(dz, w), dw=torch.matmul(dz.mT, x), db=dz.sum(0))


def _exact_logprobs(logits, tgt, case):
    z = logits.double() * case["scale"]
    lp = torch.log_softmax(z, 1)
    m = logits.double().max(1).values
    logp = lp[torch.arange(len(tgt), device=z.device), tgt.clamp(min=0)] * (tgt >= 0)
    idx = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :case["top"]]
    return dict(logp=logp, entropy=torch.special.entr(lp.exp()).sum(1), top_idx=idx.to(torch.int32),
                top_logp=lp.gather(1, idx), stats=torch.stack([m, torch.logsumexp(z, 1) - m * case["scale"]], 1))


def _exact_logprobs_grad(logits, tgt, g_logp, g_entropy, case):
    """By automatic differentiation of the definition."""
    z = logits.double().requires_grad_()
    lp = torch.log_softmax(z * case["scale"], 1)
    total = (lp[torch.arange(len(tgt), device=z.device), tgt.clamp(min=0)] * (tgt >= 0) * g_logp.double()).sum()
    if g_entropy is not None:
        total = total - ((lp.exp() * lp).sum(1) * g_entropy.double()).sum()
    return torch.autograd.grad(total, z)[0]
