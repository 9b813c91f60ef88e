"""Cases of the operators around the routed experts: the residual addition
with its root-mean-square norm and int8 output, the 4-bit linear layer, and
the router's balance loss with its gradient.

listed() gives the measured cases and draw() more of the same ranges; run()
makes one pass, in plain torch operations (own = False) or through the
library (own = True); exact() is the same result from the definition in 64
bits.  Shapes are those of the repository's workloads (hidden 2048 with 512
experts and top-8; hidden 2880 with 128 experts and top-4; prompts of 4096 and
12288 tokens; decode batches of 1, 8 and 32) next to generic ones.
"""
import math
import weakref

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
BALANCE, ZLOSS = 0.01, 0.001


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decoded token between two layers: residual sum, norm, codes for the next product
        dict(name="norm_decode_1", op="norm", tokens=1, width=2048, dtype="f32", residual=True, codes=True),
        # a decode batch of the large-expert shape with a half-precision residual stream
        dict(name="norm_batch_32_bf16", op="norm", tokens=32, width=2880, dtype="bf16", residual=True, codes=True),
        # a 4096-token prompt: the experts take the normed rows in fp32
        dict(name="norm_prompt_4096", op="norm", tokens=4096, width=2048, dtype="f32", residual=True, codes=False),
        # the longest prompt pass of the large-expert shape, sums, rows and codes
        dict(name="norm_prompt_12288", op="norm", tokens=12288, width=2880, dtype="f32", residual=True, codes=True),
        # one token against a layer's 512 router or projection rows
        dict(name="linear_rows512_t1", op="linear", tokens=1, rows=512, cols=2048, fmt="q4_0", codes=False),
        # one token's output head: the largest read of a decode step outside the experts
        dict(name="linear_head_t1", op="linear", tokens=1, rows=65536, cols=2048, fmt="q4_0", codes=False),
        # a decode batch of 8 through a square projection of the large-expert shape
        dict(name="linear_square_t8", op="linear", tokens=8, rows=2880, cols=2880, fmt="q4_0", codes=True),
        # a ragged batch (speculated tokens) with super-block weights
        dict(name="linear_q4k_t33", op="linear", tokens=33, rows=8192, cols=2048, fmt="q4_k", codes=True),
        # a 512-token prompt chunk through a wide projection
        dict(name="linear_chunk_t512", op="linear", tokens=512, rows=4096, cols=4096, fmt="q4_0", codes=False),
        # the smallest training step of a router
        dict(name="router_loss_t8", op="router", tokens=8, experts=128, k=4, mask=False, gw=True),
        # a 4096-token micro-batch of the 512-expert shape: all three gradients
        dict(name="router_loss_t4096", op="router", tokens=4096, experts=512, k=8, mask=False, gw=True),
        # a padded 12288-token batch
        dict(name="router_loss_t12288_pad", op="router", tokens=12288, experts=512, k=8, mask=True, gw=True),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n - 1 if n == 3072 else max(lo, min(hi, n))


def _blocks(rng, lo, hi, step):
    n = _log(rng, lo // step, hi // step) * step
    return n - step if n == 3072 else n


def draw(rng):
    op = rng.choice(["norm", "linear", "router"])
    if op == "norm":
        codes = rng.random() < 0.6
        width = _blocks(rng, 32, 8192, 32) if codes else _log(rng, 17, 8192)
        return dict(op="norm", tokens=_log(rng, 1, max(1, min(12288, 12288 * 2880 // width))), width=width,
                    dtype=rng.choice(["f32", "f32", "bf16", "f16"]), residual=rng.random() < 0.75, codes=codes)
    if op == "linear":
        fmt = rng.choice(["q4_0", "q4_0", "q4_k"])
        cols = _blocks(rng, 256, 8192, 256 if fmt == "q4_k" else 32)
        tokens = _log(rng, 1, 512)
        rows = _log(rng, 33, max(33, min(65536, 65536 * 2048 // cols, 512 * 4096 * 4096 // (tokens * cols))))
        return dict(op="linear", tokens=tokens, rows=rows, cols=cols, fmt=fmt, codes=rng.random() < 0.5)
    experts = _log(rng, 8, 512)
    return dict(op="router", tokens=_log(rng, 1, 12288), experts=experts, k=rng.randint(1, min(8, experts)),
                mask=rng.random() < 0.5, gw=rng.random() < 0.7)


def work(case):
    if case["op"] == "norm":
        n, el = case["tokens"] * case["width"], 4 if case["dtype"] == "f32" else 2
        moved = n * (el * (3 if case["residual"] else 1) + 4) + 4 * case["width"]
        moved += n + n // 16 if case["codes"] else 0
        return dict(bytes=moved, flops=(6 if case["codes"] else 4) * n)
    if case["op"] == "linear":
        t, r, c = case["tokens"], case["rows"], case["cols"]
        act = c + c // 16 if case["codes"] else 4 * c
        return dict(bytes=r * c * 18 // 32 + t * act + 4 * t * r, flops=2 * t * r * c)
    t, e, k = case["tokens"], case["experts"], case["k"]
    return dict(bytes=8 * t * e + 4 * t * k * (2 if case["gw"] else 1) + (t if case["mask"] else 0) + 4 * e + 8,
                flops=10 * t * e)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _q4_0(g, rows, cols):
    """Canonical blocks [rows][cols/32][18]: binary16 d, then 16 code bytes."""
    nb = cols // 32
    d = (torch.rand(rows, nb, 1, generator=g, device="cuda") * 0.015 + 0.005).half()
    codes = torch.randint(0, 256, (rows, nb, 16), generator=g, device="cuda", dtype=torch.uint8)
    return torch.cat([d.view(torch.uint8), codes], 2)


def _q4_k(g, rows, cols):
    """Canonical super-blocks [rows][cols/256][144]: d, dmin, 12 scale bytes, 128 code bytes."""
    ns = cols // 256
    d = torch.rand(rows, ns, 1, generator=g, device="cuda") * 1.07e-4 + 6.25e-5
    m = torch.rand(rows, ns, 1, generator=g, device="cuda") * 1.9e-3 + 6e-4
    rest = torch.randint(0, 256, (rows, ns, 140), generator=g, device="cuda", dtype=torch.uint8)
    return torch.cat([torch.cat([d, m], 2).half().view(torch.uint8), rest], 2)


def _quantize(x):
    """int8 codes and binary16 scales of blocks of 32: d = amax/127, q = rint(x/d)."""
    b = x.float().reshape(x.shape[0], -1, 32)
    d = (b.abs().amax(2, keepdim=True) / torch.full((1,), 127.0, device=x.device)).half()
    f = d.float()
    q = torch.where(f > 0, (b / torch.where(f > 0, f, torch.ones_like(f))).round().clamp(-127, 127), 0.0)
    return q.to(torch.int8).reshape(x.shape), d.squeeze(2)


class _Context:
    """A library context that goes with the state that holds it."""

    def __init__(self, max_tokens, experts=8, k=1):
        import quantized_expert_cache_gb300 as qec

        self.qec = qec
        self.ctx = qec.moe_layer_init(64, 32, experts, k, 1, 0, max_tokens,
                                      stream=torch.cuda.current_stream().cuda_stream)
        weakref.finalize(self, qec.moe_destroy, self.ctx)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    t = case["tokens"]
    if case["op"] == "norm":
        n, dt = case["width"], DTYPES[case["dtype"]]
        # a few channels carry most of a residual stream's energy
        scale = torch.exp(torch.randn(n, generator=g, device="cuda"))
        s["x"] = (torch.randn(t, n, generator=g, device="cuda") * 0.5).to(dt)
        s["res"] = (torch.randn(t, n, generator=g, device="cuda") * scale).to(dt) if case["residual"] else None
        s["weight"] = 1.0 + 0.2 * torch.randn(n, generator=g, device="cuda")
        if own:
            s["c"] = _Context(1)
            s["sum"] = torch.empty(t, n, dtype=dt, device="cuda") if case["residual"] else None
            s["y"] = torch.empty(t, n, device="cuda")
            if case["codes"]:
                s["q"] = torch.empty(t, n, dtype=torch.int8, device="cuda")
                s["d"] = torch.empty(t, n // 32, dtype=torch.float16, device="cuda")
                s["values"] = torch.empty(t, n // 32, 32, dtype=torch.float16, device="cuda")
                s["q32"], s["d1"] = s["q"].view(t, n // 32, 32), s["d"].view(t, n // 32, 1)
        return s
    if case["op"] == "linear":
        rows, cols = case["rows"], case["cols"]
        s["w"] = (_q4_k if case["fmt"] == "q4_k" else _q4_0)(g, rows, cols)
        s["x"] = torch.randn(t, cols, generator=g, device="cuda") * torch.exp(
            0.5 * torch.randn(cols, generator=g, device="cuda"))
        s["q"], s["d"] = _quantize(s["x"])
        if own:
            s["c"] = _Context(t)
            qec = s["c"].qec
            s["id"] = qec.moe_linear_register(s["c"].ctx, s["w"].cpu().numpy(),
                                              qec.FMT_Q4_K if case["fmt"] == "q4_k" else qec.FMT_Q4_0, rows, cols)
            s["y"] = torch.empty(t, rows, device="cuda")
        return s
    e, k = case["experts"], case["k"]
    # popularity falls off with an expert's rank, as in a trained router
    pop = -1.1 * torch.log(torch.randperm(e, generator=g, device="cuda").float() + 1)
    s["logits"] = pop + torch.randn(t, e, generator=g, device="cuda") * 1.3
    s["idx"] = torch.topk(s["logits"], k, dim=1).indices.to(torch.int32)
    s["mask"] = (torch.rand(t, generator=g, device="cuda") < 0.8).to(torch.uint8) if case["mask"] else None
    s["gw"] = torch.randn(t, k, generator=g, device="cuda") / t if case["gw"] else None
    if own:
        s["c"] = _Context(1, e, k)
        s["loss"] = torch.empty(2, device="cuda")
        s["counts"] = torch.empty(e, dtype=torch.int32, device="cuda")
        s["dlogits"] = torch.empty(t, e, device="cuda")
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if own:
        return {"norm": _own_norm, "linear": _own_linear, "router": _own_router}[case["op"]](s, case)
    return {"norm": _plain_norm, "linear": _plain_linear, "router": _plain_router}[case["op"]](s, case)


def _own_norm(s, case):
    c = s["c"]
    codes = case["codes"]
    c.qec.moe_rms_norm(c.ctx, s["x"], s["res"], s["weight"], case["tokens"], case["width"], EPS, s["sum"], s["y"],
                       s["q"] if codes else None, s["d"] if codes else None)
    out = dict(sum=s["sum"], y=s["y"])
    if codes:
        # the codes as the values they stand for
        out["codes"] = torch.mul(s["q32"], s["d1"], out=s["values"])
    return out


def _plain_norm(s, case):
    v = s["x"].float()
    out = {}
    if case["residual"]:
        v = v + s["res"].float()
        out["sum"] = v.to(s["x"].dtype)
    else:
        out["sum"] = None
    y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * s["weight"]
    out["y"] = y
    if case["codes"]:
        q, d = _quantize(y)
        out["codes"] = q.view(case["tokens"], -1, 32) * d.unsqueeze(2)
    return out


def _own_linear(s, case):
    c = s["c"]
    if case["codes"]:
        c.qec.moe_linear_forward(c.ctx, s["id"], None, case["tokens"], s["y"], q=s["q"], d=s["d"])
    else:
        c.qec.moe_linear_forward(c.ctx, s["id"], s["x"], case["tokens"], s["y"])
    return s["y"]


def _weights(w, fmt, dtype):
    """Canonical bytes -> the weights [rows][cols] in dtype."""
    rows, n, _ = w.shape
    if fmt == "q4_0":
        d = w[:, :, :2].contiguous().view(torch.float16).to(dtype)
        b = w[:, :, 2:]
        q = torch.cat([b & 15, b >> 4], 2).to(dtype) - 8
        return (d * q).reshape(rows, n * 32)
    dm = w[:, :, :4].contiguous().view(torch.float16).to(dtype)
    a, b, h = w[:, :, 4:8], w[:, :, 8:12], w[:, :, 12:16]
    sc = torch.cat([a & 63, (h & 15) | ((a >> 6) << 4)], 2).to(dtype)
    mn = torch.cat([b & 63, (h >> 4) | ((b >> 6) << 4)], 2).to(dtype)
    c = w[:, :, 16:].reshape(rows, n, 4, 1, 32)
    q = torch.cat([c & 15, c >> 4], 3).reshape(rows, n, 8, 32).to(dtype)
    scale, low = (dm[:, :, 0:1] * sc).unsqueeze(3), (dm[:, :, 1:2] * mn).unsqueeze(3)
    return (scale * q - low).reshape(rows, n * 256)


def _plain_linear(s, case):
    q, d = (s["q"], s["d"]) if case["codes"] else _quantize(s["x"])
    x = (q.float().view(case["tokens"], -1, 32) * d.float().unsqueeze(2)).reshape(case["tokens"], -1)
    return x @ _weights(s["w"], case["fmt"], torch.float32).t()


def _own_router(s, case):
    c = s["c"]
    c.qec.moe_router_loss(c.ctx, s["logits"], s["idx"], s["mask"], s["gw"], case["tokens"], case["experts"],
                          case["k"], BALANCE, ZLOSS, s["loss"], s["counts"], s["dlogits"])
    return dict(loss=s["loss"], counts=s["counts"], dlogits=s["dlogits"])


def _plain_router(s, case):
    z, idx = s["logits"], s["idx"].long()
    t, e, k = case["tokens"], case["experts"], case["k"]
    m = s["mask"].float() if case["mask"] else torch.ones(t, device=z.device)
    n = m.sum().clamp(min=1.0)
    counts = torch.zeros(e, device=z.device).index_add_(0, idx.reshape(-1), m.repeat_interleave(k))
    top = z.amax(1, keepdim=True)
    ex = torch.exp(z - top)
    tot = ex.sum(1, keepdim=True)
    p, lse = ex / tot, (top + torch.log(tot))
    f = counts / (n * k)
    dot = (p * f).sum(1, keepdim=True)
    m1 = m.unsqueeze(1)
    loss = torch.stack([BALANCE * e * (dot * m1).sum() / n, ZLOSS * (lse * lse * m1).sum() / n])
    dz = m1 / n * p * (BALANCE * e * (f - dot) + 2 * ZLOSS * lse)
    if case["gw"]:
        zs = z.gather(1, idx)
        es = torch.exp(zs - zs.amax(1, keepdim=True))
        w = es / es.sum(1, keepdim=True)
        gs = w * (s["gw"] - (w * s["gw"]).sum(1, keepdim=True)) * m1
        dz = dz.scatter_add(1, idx, gs)
    return dict(loss=loss, counts=counts.to(torch.int32), dlogits=dz)


# --------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# --------------------------------------------------------------------------
def _np_quantize(y32):
    """The format's rounding steps are part of its definition: binary32 amax/127 to binary16, then binary32 x/d."""
    b = y32.reshape(-1, 32)
    d = (np.abs(b).max(1) / np.float32(127)).astype(np.float16)
    f = d.astype(np.float32)
    q = np.zeros_like(b)
    on = f > 0
    q[on] = np.clip(np.rint(b[on] / f[on, None]), -127, 127)
    return q, d


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    t = case["tokens"]
    if case["op"] == "norm":
        v = s["x"].double()
        out = dict(sum=None)
        if case["residual"]:
            v = v + s["res"].double()
            out["sum"] = v
        ms = torch.linalg.vector_norm(v, dim=1, keepdim=True) ** 2 / case["width"]
        y = v / torch.sqrt(ms + EPS) * s["weight"].double()
        out["y"] = y
        if case["codes"]:
            q, d = _np_quantize(y.float().cpu().numpy())
            out["codes"] = torch.from_numpy((q * d[:, None].astype(np.float64)).reshape(t, -1, 32))
        return out
    if case["op"] == "linear":
        if case["codes"]:
            x = s["q"].double().view(t, -1, 32) * s["d"].double().unsqueeze(2)
        else:
            q, d = _np_quantize(s["x"].cpu().numpy())
            x = torch.from_numpy(q * d[:, None].astype(np.float64)).cuda()
        x = x.reshape(t, -1)
        rows = max(1, (1 << 25) // case["cols"])
        parts = [x @ _weights(s["w"][r:r + rows], case["fmt"], torch.float64).t()
                 for r in range(0, case["rows"], rows)]
        return torch.cat(parts, 1)
    z, idx, e, k = s["logits"].double(), s["idx"].long(), case["experts"], case["k"]
    keep = torch.ones(t, dtype=torch.bool, device=z.device) if s["mask"] is None else s["mask"].bool()
    n = int(keep.sum())
    counts = torch.bincount(idx[keep].reshape(-1), minlength=e)
    dz = torch.zeros_like(z)
    if n == 0:
        return dict(loss=torch.zeros(2, dtype=torch.float64), counts=None, dlogits=dz)
    f = counts.double() / (n * k)
    p, lse = torch.softmax(z, 1), torch.logsumexp(z, 1)
    dot = p @ f
    loss = torch.stack([BALANCE * e * dot[keep].mean(), ZLOSS * lse[keep].square().mean()])
    dz = p * (BALANCE * e * (f[None] - dot[:, None]) + 2 * ZLOSS * lse[:, None]) / n
    if case["gw"]:
        w = torch.softmax(z.gather(1, idx), 1)
        gw = s["gw"].double()
        dz.scatter_add_(1, idx, w * (gw - (w * gw).sum(1, keepdim=True)))
    dz[~keep] = 0
    return dict(loss=loss, counts=None, dlogits=dz)
