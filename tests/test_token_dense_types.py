"""The binding of the token log probabilities and the dense layers refuses a tensor of
another type than the C call reads, one that is not contiguous or not on a GPU, and
passes the types that it found.  Stand-ins take the place of CUDA tensors and of the
library, so this runs on the CPU."""
import pytest

import quantized_expert_cache_gb300 as qec
from test_operator_types import SIZES, Tensor as T


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


class Space(T):
    nbytes = 4096


F32, I32 = T("float32"), T("int32")
TOKEN = dict(ctx=1, logits=F32, targets=I32, n_tokens=1, vocab=8)
ARGS = {
    "moe_token_logprobs": dict(TOKEN, logp=F32, entropy=F32, n_top=1, top_idx=I32, top_logp=F32, stats=F32),
    "moe_token_logprobs_grad": dict(TOKEN, stats=F32, entropy=F32, g_logp=F32, g_entropy=F32, dlogits=F32),
    "moe_dense_forward": dict(ctx=1, x=F32, w=T("bfloat16"), n_tokens=1, rows=8, cols=8, y=F32, bias=F32, res=F32,
                              pre=F32, ws=Space("uint8")),
    "moe_dense_backward": dict(ctx=1, x=F32, w=T("bfloat16"), dy=F32, n_tokens=1, rows=8, cols=8, dx=F32, dw=F32,
                               db=F32, pre=F32, ws=Space("uint8")),
}
# arguments that set a type of their own, and those that go with one of them
FREE = {"moe_token_logprobs": ("logits",), "moe_token_logprobs_grad": (), "moe_dense_forward": ("x", "w"),
        "moe_dense_backward": ("w", "dw")}
SAME = {"moe_token_logprobs_grad": [("logits", "dlogits")], "moe_dense_forward": [("y", "res", "pre")],
        "moe_dense_backward": [("x", "dx"), ("dy", "pre")]}


@pytest.fixture()
def lib(monkeypatch):
    made = Library()
    monkeypatch.setattr(qec, "_lib", made)
    return made


@pytest.mark.parametrize("name", ARGS)
def test_types(lib, name):
    fn, args = getattr(qec, name), ARGS[name]
    fn(**args)
    assert len(lib.calls) == 1
    grouped = {n for g in SAME.get(name, ()) for n in g}
    for arg, tensor in args.items():
        if not isinstance(tensor, T) or arg == "ws":
            continue
        for other in SIZES:
            calls = len(lib.calls)
            allowed = (("float32", "float16", "bfloat16") if arg in FREE[name] else
                       ("int32", "uint32") if tensor is I32 else ("float32",))
            if other in allowed:
                fn(**dict(args, **{arg: T(other)}))
                assert len(lib.calls) == calls + 1
            else:
                with pytest.raises(ValueError):
                    fn(**dict(args, **{arg: T(other)}))
                assert len(lib.calls) == calls
        for bad in (T(tensor.dtype.name, cuda=False), T(tensor.dtype.name, contiguous=False)):
            with pytest.raises(ValueError):
                fn(**dict(args, **{arg: bad}))
    for group in SAME.get(name, ()):
        for other in ("float16", "bfloat16"):
            fn(**dict(args, **{n: T(other) for n in group}))
    assert grouped <= set(args)


def test_codes_of_the_types(lib):
    args = ARGS["moe_dense_forward"]
    for name, code in (("float32", qec.F32), ("float16", qec.F16), ("bfloat16", qec.BF16)):
        qec.moe_dense_forward(**dict(args, x=T(name), w=T(name), y=T(name), res=None, pre=None))
        sent = lib.calls[-1][1]
        assert (sent[2], sent[4], sent[12]) == (code, code, code) and sent[14:16] == (4096, 4096)
        qec.moe_dense_forward(**dict(args, x=64, w=128, y=256, res=None, pre=None, ws=None, x_dtype=code,
                                     w_dtype=code, y_dtype=code))
        sent = lib.calls[-1][1]
        assert (sent[1], sent[2], sent[3], sent[4], sent[12]) == (64, code, 128, code, code) and sent[14:16] == (None, 0)
        with pytest.raises(ValueError):
            qec.moe_dense_forward(**dict(args, x=T("float32" if code else "float16"), x_dtype=code))
    qec.moe_dense_backward(**dict(ARGS["moe_dense_backward"], x=None, dx=None, dw=None, db=None, x_dtype=qec.BF16))
    sent = lib.calls[-1][1]
    assert sent[1:3] == (None, qec.BF16) and sent[13] is None


def test_workspace_takes_tensors_types_and_codes(lib):
    for x, w, y in ((F32, T("bfloat16"), T("float16")), (F32.dtype, T("bfloat16").dtype, T("float16").dtype),
                    (qec.F32, qec.BF16, qec.F16)):
        assert qec.moe_dense_workspace(1, x, w, y, 0, 2, 8, 16) == (0, 0)
        assert lib.calls[-1][1][1:8] == (qec.F32, qec.BF16, qec.F16, 0, 2, 8, 16)
    for bad in (T("float64"), T("float64").dtype):
        with pytest.raises(ValueError):
            qec.moe_dense_workspace(1, bad, qec.BF16, qec.F32, 0, 2, 8, 16)


def test_an_error_raises(monkeypatch):
    class Refusing:
        def __getattr__(self, name):
            return (lambda ctx: b"no") if name == "moe_last_error" else lambda *a: -1

    monkeypatch.setattr(qec, "_lib", Refusing())
    for name, args in ARGS.items():
        with pytest.raises(qec.MoeError, match="no"):
            getattr(qec, name)(**args)
