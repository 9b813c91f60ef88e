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
                     "moe_linear_forward", "moe_router_loss"):
            f = getattr(self.lib, name)
            f.restype, f.argtypes = qec.SIGNATURES[name]
        self.lib.host_log.restype = ctypes.c_char_p
        self.lib.host_fail_launch.argtypes = [ctypes.c_char_p]

    def context(self, max_tokens=64, experts=8, k=2, stream=STREAM):
        cfg = qec.moe_cfg(64, 32, experts, k, 1, 0, max_tokens, 64, 0, 1, 10000, 0, qec.FMT_Q4_0, 0)
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
