"""Refusals of the token log probabilities and the 16-bit dense layers that guard their
results, on the host over a stand-in for the CUDA runtime."""
import ctypes
import math

from test_host_token_dense import BF16, F32, backward, ctx, grad, lib, logprobs  # noqa: F401


def test_without_tokens_the_gradients_outputs_may_not_meet_the_weights(lib, ctx):  # noqa: F811
    # (sums over no tokens are written as zeros, and sets take effect here: over weights, those would go)
    c = backward(lib, ctx, tokens=0)
    room = ctypes.create_string_buffer(1 << 16)
    w = (ctypes.addressof(room) + (1 << 14) + 255) // 256 * 256
    n = 33 * 64 * 2
    for out, size, dwd in (("dw", 33 * 64 * 4, F32), ("dw", n, BF16), ("db", 33 * 4, F32)):
        other = dict(dw=None) if out == "db" else dict(db=None)
        for at in (0, n - 16, -((size - 1) // 16 * 16)):
            c.refuses(w=w, dwd=dwd, **{out: w + at}, **other)
        for at in (n, -((size + 15) // 16 * 16)):
            c.takes(["set"], w=w, dwd=dwd, **{out: w + at}, **other)
    # (weights that a call does not read are not looked at)
    c.takes(["set"], w=w, dx=None, dw=w, db=None)


def test_scales_whose_binary_logarithm_passes_fp32(lib, ctx):  # noqa: F811
    # scale / ln 2 has to be finite: the row's largest logit is 0 times it
    for make in (logprobs, grad):
        c = make(lib, ctx)
        c.takes(scale=2.0 ** 127)
        c.takes(scale=2.0 ** -149)
        for scale in (math.nextafter(2.0 ** 127, math.inf) * (1 + 2.0 ** -23), 2.4e38, 3.4028234e38):
            c.refuses(scale=scale)
