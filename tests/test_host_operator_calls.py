"""The C entry points of the operators around the experts, built for the host
over a stand-in for the CUDA runtime (`tests/host/api_host.cpp`): which stream
the uploads and kernels of a call go to, and what is refused before any launch.
These run wherever the CPU suite runs; the GPU tests hold the same calls to
their results."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import quantized_expert_cache_gb300 as qec
from test_host_format_path import CSRC, ROOT, _cuda_include

SRC = os.path.join(ROOT, "tests", "host", "api_host.cpp")
OUT = os.path.join(ROOT, "tests", "host", "_build", "libapi_host.so")
STREAM = 0x1000  # a stream of the caller's that the legacy stream does not order


class Host:
    """The library's entry points over the stand-in, and its log."""

    def __init__(self, path):
        self.lib = ctypes.CDLL(path)
        for name in ("moe_layer_init", "moe_destroy", "moe_last_error", "moe_rms_norm", "moe_linear_register",
                     "moe_linear_forward", "moe_router_loss", "register_shared_expert", "moe_set_router",
                     "register_expert_tensor", "moe_set_preheat", "moe_pool_borrow", "moe_pool_return"):
            f = getattr(self.lib, name)
            f.restype, f.argtypes = qec.SIGNATURES[name]
        self.lib.host_log.restype = ctypes.c_char_p
        self.lib.host_fail_launch.argtypes = [ctypes.c_char_p]

    def context(self, max_tokens=64, experts=8, k=2, stream=STREAM, slots=0, shared=0):
        cfg = qec.moe_cfg(64, 32, experts, k, 1, slots, max_tokens, 64, 0, 1, 10000, 0, qec.FMT_Q4_0, shared)
        out = ctypes.c_void_p()
        assert self.lib.moe_layer_init(ctypes.byref(cfg), stream, ctypes.byref(out)) == 0
        self.lib.host_clear()
        return out.value

    def register(self, ctx, w, fmt, rows, cols):
        lid = ctypes.c_int(-1)
        return self.lib.moe_linear_register(ctx, w.ctypes.data, fmt, rows, cols, ctypes.byref(lid)), lid.value

    def log(self):
        """(what, stream, first address, second address, size) of every call since the last clear."""
        rows = [line.split() for line in self.lib.host_log().decode().splitlines()]
        return [(r[0], int(r[1], 16), int(r[2], 16), int(r[3], 16), int(r[4])) for r in rows]


@pytest.fixture(scope="module")
def host():
    inc = _cuda_include()
    if inc is None or shutil.which("g++") is None:
        pytest.skip("needs g++ and the CUDA headers")
    deps = [SRC, os.path.join(ROOT, "include", "moe_cache.h")]
    deps += [os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith((".h", ".cuh")) or h == "moe_cache.cu"]
    if not os.path.exists(OUT) or any(os.path.getmtime(d) > os.path.getmtime(OUT) for d in deps):
        os.makedirs(os.path.dirname(OUT), exist_ok=True)
        tmp = OUT + f".{os.getpid()}.tmp"
        subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-fvisibility-inlines-hidden",
                        "-Wl,-Bsymbolic", "-Wno-unknown-pragmas", "-Wno-class-memaccess", "-Wno-subobject-linkage",
                        "-I" + inc, "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, SRC, "-o", tmp, "-lpthread"],
                       check=True)
        os.replace(tmp, OUT)
    return Host(OUT)


@pytest.mark.parametrize("max_tokens", [1, 64])
@pytest.mark.parametrize("fmt,block", [(qec.FMT_Q4_0, 18), (qec.FMT_Q4_K, 144)])
def test_registration_uploads_on_the_stream_that_reads(host, fmt, block, max_tokens):
    # A copy of pageable memory on the legacy stream may return before its last bytes have landed, and
    # a non-blocking stream is not ordered after it: the blocks go up on the stream of the kernel that
    # repacks them, and nothing of the call is on another stream.
    ctx = host.context(max_tokens)
    w = np.zeros((24, 512 // (32 if block == 18 else 256), block), np.uint8)
    rc, _ = host.register(ctx, w, fmt, 24, 512)
    assert rc == 0
    log = host.log()
    repack = next(i for i, c in enumerate(log) if c[0] == "linear_repack")
    upload = next(i for i, c in enumerate(log) if c[0] == "copy" and c[3] == w.ctypes.data)
    assert upload < repack and log[upload][2] == log[repack][2] and log[upload][4] == w.nbytes
    assert all(c[1] == STREAM for c in log), log
    # and the call returns when the caller's memory has been read
    assert any(c[0] == "sync" for c in log[upload:])
    host.lib.moe_destroy(ctx)


def test_later_uploads_and_sets_are_on_the_stream_that_reads(host):
    # the same for a shared expert, a router for lookahead, and the use counts that a returned pool clears
    lib, ctx = host.lib, host.context(slots=4, shared=1)
    gate, down = np.zeros((32, 2, 18), np.uint8), np.zeros((64, 1, 18), np.uint8)
    for kind in range(3):
        w = down if kind == 2 else gate
        assert lib.register_shared_expert(ctx, 0, kind, w.ctypes.data, w.shape[0], w.shape[1] * 32) == 0
    router = np.zeros((8, 64), np.float32)
    for _ in range(2):
        assert lib.moe_set_router(ctx, 0, router.ctypes.data, None) == 0
    log = host.log()
    moved = [c for c in log if c[0] in ("copy", "set")]
    assert len(moved) == 2 * 3 + 3 + 2 * 2 and all(c[1] == STREAM for c in moved), moved
    assert log[-1][:2] == ("sync", STREAM)
    for kind in range(3):
        w = np.concatenate([down if kind == 2 else gate] * 8)
        assert lib.register_expert_tensor(ctx, 0, kind, w.ctypes.data, w.shape[0] // 8, w.shape[1] * 32, 4, None, 4,
                                          None) == 0
    assert lib.moe_set_preheat(ctx, 1) == 0
    ws, size = ctypes.c_void_p(), ctypes.c_size_t()
    assert lib.moe_pool_borrow(ctx, 3, ctypes.byref(ws), ctypes.byref(size)) == 0
    host.lib.host_clear()
    assert lib.moe_pool_return(ctx) == 0
    sets = [c for c in host.log() if c[0] == "set"]
    assert sets and all(c[1] == STREAM for c in sets), sets
    lib.moe_destroy(ctx)


# ---- refusals before any launch: addresses stand for device buffers, which nothing here reads
A = 1 << 32  # far from one another unless a test moves them


def buffers(names, **change):
    at = {n: (i + 1) * A for i, n in enumerate(names)}
    return dict(at, **change)


def norm(host, ctx, dtype=0, tokens=3, width=64, **change):
    b = buffers(("x", "res", "weight", "sum", "y", "q", "d"), **change)
    return host.lib.moe_rms_norm(ctx, b["x"], b["res"], dtype, b["weight"], tokens, width, 1e-6, b["sum"], b["y"],
                                 b["q"], b["d"], None)


def linear(host, ctx, lid, tokens=3, **change):
    b = buffers(("x", "q", "d", "y"), **change)
    return host.lib.moe_linear_forward(ctx, lid, b["x"], b["q"], b["d"], tokens, b["y"], None)


def router(host, ctx, tokens=3, **change):
    b = buffers(("logits", "idx", "mask", "gw", "loss", "counts", "dlogits"), **change)
    return host.lib.moe_router_loss(ctx, b["logits"], b["idx"], b["mask"], b["gw"], tokens, 8, 2, 0.1, 0.1, b["loss"],
                                    b["counts"], b["dlogits"], None)


class Call:
    """One operator of a context: whether a call is taken, and that a refused one launches nothing."""

    def __init__(self, host, call, *args):
        self.host, self.call, self.args = host, call, args

    def takes(self, **change):
        self.host.lib.host_clear()
        assert self.call(self.host, *self.args, **change) == 0, change
        assert len(self.host.log()) == 1

    def refuses(self, **change):
        self.host.lib.host_clear()
        assert self.call(self.host, *self.args, **change) == -1, change
        assert not self.host.log()


@pytest.fixture()
def calls(host):
    ctx = host.context()
    rc, lid = host.register(ctx, np.zeros((24, 2, 18), np.uint8), qec.FMT_Q4_0, 24, 64)
    assert rc == 0
    yield Call(host, norm, ctx), Call(host, linear, ctx, lid), Call(host, router, ctx)
    host.lib.moe_destroy(ctx)


def test_addresses_off_their_elements_are_refused(calls):
    norms, linears, routers = calls
    norms.takes()
    for name, size in dict(x=4, res=4, sum=4, weight=4, y=4, d=2).items():
        for off in range(1, size):
            norms.refuses(**{name: 16 * A + off})
        norms.takes(**{name: 16 * A + size})
    for dtype in (1, 2):
        for name in ("x", "res", "sum"):
            norms.refuses(dtype=dtype, **{name: 16 * A + 1})
            norms.takes(dtype=dtype, **{name: 16 * A + 2})
    norms.takes(q=16 * A + 1)
    codes = dict(x=None)
    values = dict(q=None, d=None)
    linears.takes(**codes)
    linears.takes(**values)
    linears.refuses(x=16 * A + 4, q=None, d=None)
    linears.refuses(x=None, q=16 * A + 4)
    linears.refuses(x=None, d=16 * A + 1)
    linears.refuses(y=16 * A + 2, **values)
    linears.takes(y=16 * A + 4, **values)
    routers.takes()
    for name in ("logits", "idx", "gw", "loss", "counts", "dlogits"):
        for off in (1, 2, 3):
            routers.refuses(**{name: 16 * A + off})
        routers.takes(**{name: 16 * A + 4})
    routers.takes(mask=16 * A + 1)


def sizes(call, dtype=0, n=3 * 64):
    el = 2 if dtype else 4
    return dict(norm=dict(x=n * el, res=n * el, weight=64 * 4, sum=n * el, y=n * 4, q=n, d=n // 32 * 2),
                linear=dict(x=n * 4, q=n, d=n // 32 * 2, y=3 * 24 * 4),
                router=dict(logits=3 * 8 * 4, idx=3 * 2 * 4, mask=3, gw=3 * 2 * 4, loss=8, counts=8 * 4,
                            dlogits=3 * 8 * 4))[call]


def check_overlaps(call, names, outs, size, same=(), **fixed):
    """Every output against every other buffer of the call: side by side is taken; the first byte on the
    last, the last on the first, and the same address (but for the pairs of `same`) are refused."""
    base = 64 * A
    gap = lambda n: (n + 15) // 16 * 16  # noqa: E731  (aligned for every type)
    for o in outs:
        for i in names:
            if i == o:
                continue
            call.takes(**fixed, **{i: base, o: base + gap(size[i])})
            call.takes(**fixed, **{i: base, o: base - gap(size[o])})
            last = (size[i] - 1) // 16 * 16  # the last aligned address inside i
            for at in (last, -((size[o] - 1) // 16 * 16)):
                if at:
                    call.refuses(**fixed, **{i: base, o: base + at})
            (call.takes if (o, i) in same else call.refuses)(**fixed, **{i: base, o: base})


def test_buffers_that_meet_are_refused(calls):
    norms, linears, routers = calls
    outs = ("sum", "y", "q", "d")
    same = {("sum", "x"), ("sum", "res")}
    names = ("x", "res", "weight") + outs
    check_overlaps(norms, names, outs, sizes("norm"), same | {("y", "x"), ("y", "res")})
    for dtype in (1, 2):
        check_overlaps(norms, names, outs, sizes("norm", dtype), same, dtype=dtype)
    norms.takes(x=A, res=A)                      # inputs may be one buffer
    norms.takes(x=A, res=A, sum=A)
    norms.takes(x=A, res=2 * A, sum=2 * A, y=A)
    norms.refuses(x=A, sum=A, y=A)               # two outputs on it may not
    norms.refuses(x=A, res=A + 16, sum=A)        # and not where the other input is read elsewhere
    check_overlaps(linears, ("x", "y"), ("y",), sizes("linear"), q=None, d=None)
    check_overlaps(linears, ("q", "y"), ("y",), sizes("linear"), x=None)
    check_overlaps(linears, ("d", "y"), ("y",), sizes("linear"), x=None)
    check_overlaps(routers, ("logits", "idx", "mask", "gw", "loss", "counts", "dlogits"),
                   ("loss", "counts", "dlogits"), sizes("router"))


def test_calls_without_tokens_meet_nothing(host, calls):
    norms, linears, routers = calls
    host.lib.host_clear()
    assert norm(host, norms.args[0], tokens=0, x=A, y=A, sum=A) == 0
    assert linear(host, *linears.args, tokens=0, x=A, y=A) == 0
    assert not host.log()
    routers.takes(tokens=0, logits=A, dlogits=A + 4)
    routers.refuses(tokens=0, loss=A, counts=A)


def test_a_failure_is_reported_once(host, calls):
    # the runtime keeps a call's error as its last one; left there, the next launch, the library's or the
    # caller's own, would answer with it
    ctx = calls[0].args[0]
    assert host.lib.host_last_error() == 0
    rc, _ = host.register(ctx, np.zeros((24, 2, 18), np.uint8), qec.FMT_Q4_0, 1 << 26, 65536)  # no memory for it
    assert rc == -2 and host.lib.host_last_error() == 0
    cfg = qec.moe_cfg(64, 32, 8, 2, 1, 0, 1 << 30, 64, 0, 1, 10000, 0, qec.FMT_Q4_0, 0)
    out = ctypes.c_void_p()
    assert host.lib.moe_layer_init(ctypes.byref(cfg), STREAM, ctypes.byref(out)) == -2
    assert host.lib.host_last_error() == 0
    codes = dict(x=None)
    for call, launch, change in ((calls[0], b"rms_norm", {}), (calls[1], b"linear", codes),
                                 (calls[1], b"linear_gemm", dict(codes, tokens=40)), (calls[2], b"router_loss", {})):
        host.lib.host_fail_launch(launch)
        assert call.call(host, *call.args, **change) == -3
        assert host.lib.host_last_error() == 0, launch
        host.lib.host_fail_launch(b"")
    for launch in (b"linear_repack", b"linear_max"):
        host.lib.host_fail_launch(launch)
        rc, _ = host.register(ctx, np.zeros((24, 2, 18), np.uint8), qec.FMT_Q4_0, 24, 64)
        assert rc == -3 and host.lib.host_last_error() == 0, launch
        host.lib.host_fail_launch(b"")


def test_router_counts_start_from_zero_after_a_failed_launch(host, calls):
    # the picks are counted by a launch before the one that uses them and sets them back
    routers = calls[2]
    host.lib.host_fail_launch(b"router_loss")
    host.lib.host_clear()
    assert routers.call(host, *routers.args, tokens=5000) == -3
    host.lib.host_fail_launch(b"")
    log = host.log()
    counts = log[0][3]
    assert [c[0] for c in log] == ["router_loss", "set"]
    what, stream, start, _, size = log[1]
    assert stream == STREAM and start <= counts and start + size >= counts + 4 * (4096 + 1)
    routers.takes(tokens=5000)
