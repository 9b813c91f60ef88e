"""The C entry points of the token log probabilities and the 16-bit dense layers,
built for the host over a stand-in for the CUDA runtime
(`tests/host/operators_host.cpp`): what is refused before any launch, which launches a
call makes and on which stream."""
import ctypes
import os
import shutil
import subprocess

import pytest

import quantized_expert_cache_gb300 as qec
from test_host_format_path import CSRC, ROOT, _cuda_include

HOST = os.path.join(ROOT, "tests", "host")
SRC = os.path.join(HOST, "operators_host.cpp")
OUT = os.path.join(HOST, "_build", "liboperators_host.so")
STREAM, OTHER = 0x1000, 0x2000
A = 1 << 42  # buffers far from one another unless a test moves them
NAMES = ("moe_layer_init", "moe_destroy", "moe_last_error", "moe_token_logprobs", "moe_token_logprobs_grad",
         "moe_dense_forward", "moe_dense_backward", "moe_dense_workspace")
F32, F16, BF16 = qec.F32, qec.F16, qec.BF16


@pytest.fixture(scope="module")
def lib():
    inc = _cuda_include()
    if inc is None or shutil.which("g++") is None:
        pytest.skip("needs g++ and the CUDA headers")
    deps = [SRC, os.path.join(HOST, "api_host.cpp"), os.path.join(ROOT, "include", "moe_cache.h")]
    deps += [os.path.join(CSRC, h) for h in os.listdir(CSRC)
             if h.endswith((".h", ".cuh")) or h in ("moe_cache.cu", "operators.cu")]
    if not os.path.exists(OUT) or any(os.path.getmtime(d) > os.path.getmtime(OUT) for d in deps):
        os.makedirs(os.path.dirname(OUT), exist_ok=True)
        tmp = OUT + f".{os.getpid()}.tmp"
        subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-fvisibility-inlines-hidden",
                        "-Wl,-Bsymbolic", "-Wno-unknown-pragmas", "-Wno-class-memaccess", "-Wno-subobject-linkage",
                        "-I" + inc, "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, "-I" + HOST, SRC, "-o", tmp,
                        "-lpthread"], check=True)
        os.replace(tmp, OUT)
    made = ctypes.CDLL(OUT)
    for name in NAMES:
        f = getattr(made, name)
        f.restype, f.argtypes = qec.SIGNATURES[name]
    made.host_log.restype = ctypes.c_char_p
    made.host_fail_launch.argtypes = [ctypes.c_char_p]
    return made


@pytest.fixture()
def ctx(lib):
    cfg = qec.moe_cfg(64, 32, 8, 2, 1, 0, 64, 64, 0, 1, 10000, 0, qec.FMT_Q4_0, 0)
    out = ctypes.c_void_p()
    assert lib.moe_layer_init(ctypes.byref(cfg), STREAM, ctypes.byref(out)) == 0
    lib.host_clear()
    yield out.value
    lib.moe_destroy(out.value)


def log(lib):
    rows = [line.split() for line in lib.host_log().decode().splitlines()]
    return [(r[0], int(r[1], 16)) for r in rows]


class Call:
    """A call with its usual arguments, any of them changed by name."""

    def __init__(self, lib, ctx, name, order, buffers, **fixed):
        self.lib, self.ctx, self.fn, self.order = lib, ctx, getattr(lib, name), order
        self.args = dict({n: (i + 1) * A for i, n in enumerate(buffers)}, stream=None, **fixed)

    def __call__(self, **change):
        a = dict(self.args, **change)
        assert set(a) == set(self.args), change
        self.lib.host_clear()
        return self.fn(self.ctx, *(a[n] for n in self.order))

    def takes(self, launches=None, **change):
        assert self(**change) == 0, (change, self.lib.moe_last_error(self.ctx))
        made = log(self.lib)
        assert made, change
        if launches is not None:
            assert [m[0] for m in made] == launches
        return made

    def refuses(self, **change):
        assert self(**change) == -1, change
        assert not log(self.lib)


def logprobs(lib, ctx, **fixed):
    return Call(lib, ctx, "moe_token_logprobs",
                ("logits", "dtype", "targets", "tokens", "vocab", "scale", "n_top", "logp", "entropy", "top_idx",
                 "top_logp", "stats", "stream"),
                ("logits", "targets", "logp", "entropy", "top_idx", "top_logp", "stats"),
                **dict(dict(dtype=F32, tokens=3, vocab=100, scale=1.0, n_top=5), **fixed))


def grad(lib, ctx, **fixed):
    return Call(lib, ctx, "moe_token_logprobs_grad",
                ("logits", "dtype", "targets", "tokens", "vocab", "scale", "stats", "entropy", "g_logp", "g_entropy",
                 "dlogits", "stream"),
                ("logits", "targets", "stats", "entropy", "g_logp", "g_entropy", "dlogits"),
                **dict(dict(dtype=F32, tokens=3, vocab=100, scale=1.0), **fixed))


def forward(lib, ctx, **fixed):
    return Call(lib, ctx, "moe_dense_forward",
                ("x", "xd", "w", "wd", "bias", "act", "res", "tokens", "rows", "cols", "y", "yd", "pre", "ws",
                 "ws_bytes", "stream"),
                ("x", "w", "bias", "res", "y", "pre", "ws"),
                **dict(dict(xd=BF16, wd=BF16, yd=BF16, act=1, tokens=9, rows=33, cols=64, ws_bytes=1 << 30), **fixed))


def backward(lib, ctx, **fixed):
    return Call(lib, ctx, "moe_dense_backward",
                ("x", "xd", "w", "wd", "dy", "yd", "pre", "act", "tokens", "rows", "cols", "dx", "dw", "dwd", "db",
                 "ws", "ws_bytes", "stream"),
                ("x", "w", "dy", "pre", "dx", "dw", "db", "ws"),
                **dict(dict(xd=BF16, wd=BF16, yd=BF16, dwd=F32, act=1, tokens=9, rows=33, cols=64, ws_bytes=1 << 30),
                       **fixed))


def overlaps(call, outs, sizes, same=(), **fixed):
    """Every output against every other buffer: side by side is taken, a shared byte refused."""
    base = 64 * A
    gap = lambda n: (n + 255) // 256 * 256  # noqa: E731
    for o in outs:
        for i in sizes:
            if i == o:
                continue
            call.takes(**fixed, **{i: base, o: base + gap(sizes[i])})
            call.takes(**fixed, **{i: base, o: base - gap(sizes[o])})
            for at in ((sizes[i] - 1) // 16 * 16, -((sizes[o] - 1) // 16 * 16)):
                if at:
                    call.refuses(**fixed, **{i: base, o: base + at})
            (call.takes if (o, i) in same else call.refuses)(**fixed, **{i: base, o: base})


# ------------------------------------------------------------ token log probabilities
def test_logprobs_sizes(lib, ctx):
    c = logprobs(lib, ctx)
    c.takes(["token_logprobs"])
    for bad in (dict(dtype=3), dict(dtype=-1), dict(tokens=-1), dict(vocab=0), dict(vocab=(1 << 30) + 1),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(n_top=-1),
                dict(n_top=33), dict(n_top=6, vocab=5)):
        c.refuses(**bad)
        if "n_top" not in bad and "tokens" not in bad:
            grad(lib, ctx).refuses(**bad)
    c.takes(n_top=5, vocab=5)
    c.takes(n_top=32)
    assert c(tokens=0, logits=None) == 0 and not log(lib)
    assert grad(lib, ctx)(tokens=0, logits=None) == 0 and not log(lib)


def test_logprobs_needs_its_pointers(lib, ctx):
    c = logprobs(lib, ctx)
    for bad in (dict(logits=None), dict(targets=None), dict(top_idx=None), dict(top_logp=None),
                dict(logp=None, entropy=None, stats=None, n_top=0)):
        c.refuses(**bad)
    c.takes(targets=None, logp=None)
    c.takes(top_idx=None, top_logp=None, n_top=0)
    for one in ("logp", "entropy", "stats"):
        c.takes(n_top=0, **{n: None for n in ("logp", "entropy", "stats") if n != one})
    g = grad(lib, ctx)
    g.takes(["token_grad"])
    for bad in (dict(logits=None), dict(stats=None), dict(dlogits=None), dict(targets=None), dict(entropy=None),
                dict(g_logp=None, g_entropy=None)):
        g.refuses(**bad)
    g.takes(g_entropy=None, entropy=None)
    g.takes(g_logp=None, targets=None)


def test_logprobs_addresses(lib, ctx):
    c, g = logprobs(lib, ctx), grad(lib, ctx)
    for dtype, size in ((F32, 4), (F16, 2), (BF16, 2)):
        for off in range(1, size):
            c.refuses(dtype=dtype, logits=A + off)
            g.refuses(dtype=dtype, logits=A + off)
            g.refuses(dtype=dtype, dlogits=9 * A + off)
        c.takes(dtype=dtype, logits=A + size)
        g.takes(dtype=dtype, logits=A + size)
    for name in ("targets", "logp", "entropy", "top_idx", "top_logp", "stats"):
        c.refuses(**{name: 9 * A + 2})
        c.takes(**{name: 9 * A + 4})
    for name in ("targets", "stats", "entropy", "g_logp", "g_entropy"):
        g.refuses(**{name: 9 * A + 2})


def test_logprobs_buffers_that_meet(lib, ctx):
    sizes = dict(logits=9600, targets=96, logp=96, entropy=96, top_idx=480, top_logp=480, stats=192)
    overlaps(logprobs(lib, ctx, tokens=24), ("logp", "entropy", "top_idx", "top_logp", "stats"), sizes)
    sizes = dict(logits=9600, targets=96, stats=192, entropy=96, g_logp=96, g_entropy=96, dlogits=9600)
    overlaps(grad(lib, ctx, tokens=24), ("dlogits",), sizes, {("dlogits", "logits")})
    overlaps(grad(lib, ctx, tokens=24, dtype=BF16), ("dlogits",), dict(sizes, logits=4800, dlogits=4800),
             {("dlogits", "logits")})


# ------------------------------------------------------------------------ dense layers
@pytest.mark.parametrize("make", [forward, backward])
def test_dense_types_and_sizes(lib, ctx, make):
    c = make(lib, ctx)
    good = [(BF16, BF16, BF16), (BF16, BF16, F32), (F16, F16, F16), (F32, BF16, F32), (F32, BF16, BF16)]
    for x in (-1, F32, F16, BF16, 3):
        for w in (-1, F32, F16, BF16, 3):
            for y in (-1, F32, F16, BF16, 3):
                ok = (x, w, y) in good or (make is forward and (x, w, y) == (F16, F16, F32))
                # (a weight gradient of the weights' type)
                (c.takes if ok else c.refuses)(xd=x, wd=w, yd=y)
    for bad in (dict(act=3), dict(act=-1), dict(tokens=-1), dict(tokens=(1 << 26) + 1), dict(rows=0),
                dict(rows=(1 << 26) + 1), dict(cols=0), dict(cols=4), dict(cols=60), dict(cols=(1 << 26) + 8),
                dict(rows=1 << 20, cols=1 << 19), dict(tokens=1 << 20, rows=1 << 19), dict(tokens=1 << 20, cols=1 << 19)):
        c.refuses(**bad)
    if make is backward:
        for dwd in (-1, F16, 3):
            c.refuses(dwd=dwd)
        c.takes(dwd=F16, dw=None)
        c.takes(dwd=BF16)


def test_dense_forward_launches(lib, ctx):
    c = forward(lib, ctx)
    for tokens in (1, 4):
        c.takes(["dense_few"], tokens=tokens)
        c.takes(["dense_few"], tokens=tokens, xd=F32, ws=None, ws_bytes=0)
    c.takes(["dense_gemm"], tokens=5, ws=None, ws_bytes=0)
    c.takes(["dense_split", "dense_gemm"], tokens=5, xd=F32)
    assert c(tokens=0, x=None, w=None, y=None) == 0 and not log(lib)
    for s, want in ((None, STREAM), (OTHER, OTHER)):
        assert all(m[1] == want for m in c.takes(tokens=5, xd=F32, stream=s))
    for bad in (dict(x=None), dict(w=None), dict(y=None)):
        c.refuses(**bad)
    c.takes(bias=None, res=None, pre=None)


def test_dense_backward_launches(lib, ctx):
    c = backward(lib, ctx)
    c.takes(["dense_split", "dense_gemm"])
    c.takes(["dense_split", "dense_gemm"], act=0)                       # rows that are no multiple of 8
    c.takes(["dense_gemm", "dense_split"], act=0, rows=32)              # the sums of dz, last
    c.takes(["dense_gemm"], act=0, rows=32, db=None)
    c.takes(["dense_split", "dense_gemm"], act=0, rows=32, db=None, dy=9 * A + 2)
    c.takes(["dense_split", "dense_split", "dense_gemm"], xd=F32)
    c.takes(["dense_split", "dense_gemm"], xd=F32, dw=None)
    c.takes(["dense_split"], dx=None, dw=None)
    for s, want in ((None, STREAM), (OTHER, OTHER)):
        assert all(m[1] == want for m in c.takes(xd=F32, stream=s))
        dw, db = (ctypes.create_string_buffer(n) for n in (33 * 64 * 4 + 16, 33 * 4 + 16))  # (sets take effect)
        at = {n: (ctypes.addressof(v) + 15) // 16 * 16 for n, v in (("dw", dw), ("db", db))}
        assert all(m == ("set", want) for m in c.takes(["set", "set"], tokens=0, stream=s, **at))
    for bad in (dict(dy=None), dict(pre=None), dict(x=None), dict(w=None), dict(dx=None, dw=None, db=None)):
        c.refuses(**bad)
    c.takes(act=0, pre=None)
    c.takes(x=None, dw=None)
    c.takes(w=None, dx=None)


@pytest.mark.parametrize("xd,wd,yd,act", [(F32, BF16, F32, 0), (F32, BF16, BF16, 1), (BF16, BF16, BF16, 0),
                                          (F16, F16, F16, 2)])
def test_dense_workspaces(lib, ctx, xd, wd, yd, act):
    f, b = ctypes.c_size_t(7), ctypes.c_size_t(7)

    def ask(tokens, rows=33, cols=64):
        assert lib.moe_dense_workspace(ctx, xd, wd, yd, act, tokens, rows, cols, ctypes.byref(f), ctypes.byref(b)) == 0
        return f.value, b.value

    for tokens in (1, 4, 5, 9, 1000):
        need_f, need_b = ask(tokens)
        assert need_f == (0 if xd != F32 or tokens <= 4 else (tokens * 64 * 6 + 255) // 256 * 256)
        # dz with rows of 8, its column sums, x in parts
        assert need_b >= tokens * 40 * 2 + 33 * 4 + (tokens * 64 * 6 if xd == F32 else 0)
        for c, need in ((forward(lib, ctx), need_f), (backward(lib, ctx), need_b)):
            at = dict(xd=xd, wd=wd, yd=yd, act=act, tokens=tokens)
            c.takes(ws_bytes=need, **at)
            if need:
                c.refuses(ws_bytes=need - 1, **at)
                c.refuses(ws=None, **at)
                c.refuses(ws=99 * A + 8, **at)
    # a workspace of more tokens serves fewer
    before = (0, 0)
    for tokens in range(1, 5000):
        now = ask(tokens)
        assert all(s <= l for s, l in zip(before, now)), tokens
        before = now
    assert lib.moe_dense_workspace(ctx, xd, wd, yd, act, 5, 33, 64, None, None) == 0
    assert lib.moe_dense_workspace(ctx, xd, wd, yd, act, 5, 33, 60, ctypes.byref(f), ctypes.byref(b)) == -1


def test_dense_addresses(lib, ctx):
    f, b = forward(lib, ctx), backward(lib, ctx)
    for name in ("x", "w"):
        for off in (2, 4, 8):
            f.refuses(**{name: 9 * A + off})
            b.refuses(**{name: 9 * A + off})
    for call, names in ((f, ("res", "y", "pre")), (b, ("dy", "pre", "dx"))):
        for name in names:
            call.refuses(**{name: 9 * A + 1})
            call.takes(**{name: 9 * A + 2})
            call.refuses(yd=F32, xd=F32, **{name: 9 * A + 2})
    for call, name in ((f, "bias"), (b, "db"), (b, "dw")):
        call.refuses(**{name: 9 * A + 2})
        call.takes(**{name: 9 * A + 4})
    b.takes(dw=9 * A + 2, dwd=BF16)
    # what a call does not read is not looked at
    b.takes(x=9 * A + 1, dw=None)
    b.takes(w=9 * A + 1, dx=None)
    b.takes(pre=9 * A + 1, act=0)


def test_dense_buffers_that_meet(lib, ctx):
    n = 9 * 33
    sizes = dict(x=9 * 64 * 2, w=33 * 64 * 2, bias=33 * 4, res=n * 2, y=n * 2, pre=n * 2)
    overlaps(forward(lib, ctx), ("y", "pre"), sizes, {("y", "res")}, ws=None, ws_bytes=0)
    need = lambda i, *a: _need(lib, ctx, i, *a)  # noqa: E731
    fw = dict(xd=F32, yd=F32)
    sizes = dict(x=9 * 64 * 4, w=33 * 64 * 2, bias=33 * 4, res=n * 4, y=n * 4, pre=n * 4, ws=need(0, F32, BF16, F32))
    overlaps(forward(lib, ctx, **fw), ("y", "pre", "ws"), sizes, {("y", "res")})
    sizes = dict(x=9 * 64 * 2, w=33 * 64 * 2, dy=n * 2, pre=n * 2, dx=9 * 64 * 2, dw=33 * 64 * 4, db=33 * 4,
                 ws=need(1, BF16, BF16, BF16))
    overlaps(backward(lib, ctx), ("dx", "dw", "db", "ws"), sizes)


def _need(lib, ctx, which, xd, wd, yd):
    got = (ctypes.c_size_t(), ctypes.c_size_t())
    assert lib.moe_dense_workspace(ctx, xd, wd, yd, 1, 9, 33, 64, *(ctypes.byref(g) for g in got)) == 0
    return got[which].value


def test_without_tokens_the_gradients_outputs_may_not_meet(lib, ctx):
    backward(lib, ctx).refuses(tokens=0, dw=A, db=A)


def test_failures_are_reported_once(lib, ctx):
    for call, launch, change in ((logprobs(lib, ctx), b"token_logprobs", {}), (grad(lib, ctx), b"token_grad", {}),
                                 (forward(lib, ctx), b"dense_few", dict(tokens=2)),
                                 (forward(lib, ctx), b"dense_gemm", {}),
                                 (forward(lib, ctx), b"dense_split", dict(xd=F32)),
                                 (backward(lib, ctx), b"dense_split", {}), (backward(lib, ctx), b"dense_gemm", {})):
        lib.host_fail_launch(launch)
        assert call(**change) == -3
        assert launch[:5] in lib.moe_last_error(ctx).replace(b"token_logprobs_grad", b"token_grad")
        assert lib.host_last_error() == 0
        lib.host_fail_launch(b"")
        call.takes(**change)
