"""The binding of the operators around the routed experts refuses a tensor whose
elements are not of the type the C call reads: one of another size would be read
or written past its end.  Stand-ins take the place of CUDA tensors and of the
library, so this runs on the CPU."""
import pytest

import quantized_expert_cache_gb300 as qec

SIZES = dict(float64=8, int64=8, float32=4, int32=4, uint32=4, float16=2, bfloat16=2, int16=2, uint16=2, int8=1,
             uint8=1, bool=1)


class Type:
    """As torch names its types: one object each, str "torch.<name>"."""
    made = {}

    def __new__(cls, name):
        if name not in cls.made:
            cls.made[name] = super().__new__(cls)
            cls.made[name].name = name
        return cls.made[name]

    def __str__(self):
        return "torch." + self.name


class Tensor:
    def __init__(self, name, cuda=True, contiguous=True):
        self.dtype, self.is_cuda, self.contiguous = Type(name), cuda, contiguous

    def is_contiguous(self):
        return self.contiguous

    def element_size(self):
        return SIZES[self.dtype.name]

    def data_ptr(self):
        return 4096


class Library:
    calls = 0

    def __getattr__(self, name):
        def call(*args):
            Library.calls += 1
            return 0
        return call


T = Tensor
F32, F16 = T("float32"), T("float16")
ARGS = {
    "moe_rms_norm": dict(ctx=1, x=F32, res=F32, weight=F32, n_tokens=1, width=32, eps=1e-6, sum=F32, y=F32,
                         q=T("int8"), d=F16),
    "moe_linear_forward": dict(ctx=1, linear_id=0, x=F32, n_tokens=1, y=F32, q=T("int8"), d=F16),
    "moe_router_loss": dict(ctx=1, logits=F32, idx=T("int32"), mask=T("uint8"), gw=F32, n_tokens=1, n_experts=8, k=2,
                            balance_coef=0.1, z_coef=0.1, loss=F32, counts=T("int32"), dlogits=F32),
}
TAKES = dict(float32=("float32",), float16=("float16", "int16", "uint16"), int8=("int8", "uint8"),
             int32=("int32", "uint32"), uint8=("uint8", "int8", "bool"))
ROWS = ("x", "res", "sum")  # of the norm: any of the three types, all of one


@pytest.fixture(autouse=True)
def library(monkeypatch):
    monkeypatch.setattr(qec, "load", lambda: Library())


def takes(call, **change):
    before = Library.calls
    getattr(qec, call)(**dict(ARGS[call], **change))
    assert Library.calls == before + 1


def refuses(call, **change):
    before = Library.calls
    with pytest.raises(ValueError):
        getattr(qec, call)(**dict(ARGS[call], **change))
    assert Library.calls == before, "the library was called"


@pytest.mark.parametrize("call", sorted(ARGS))
def test_other_element_types_are_refused(call):
    for arg, right in ARGS[call].items():
        if not isinstance(right, Tensor):
            continue
        rows = call == "moe_rms_norm" and arg in ROWS
        for name in SIZES:
            if rows and name != "float32" or not rows and name not in TAKES[right.dtype.name]:
                refuses(call, **{arg: T(name)})
            else:
                takes(call, **{arg: T(name)})


@pytest.mark.parametrize("name", ["float16", "bfloat16"])
def test_norm_rows_of_16_bits(name):
    t = T(name)
    takes("moe_rms_norm", x=t, res=t, sum=t)
    takes("moe_rms_norm", x=t, res=None, sum=None)
    refuses("moe_rms_norm", x=t, res=t, sum=t, weight=t)  # a model file's weights
    refuses("moe_rms_norm", x=t, res=t, sum=t, y=t)


def test_norm_with_its_type_given():
    takes("moe_rms_norm", x=T("int16"), res=T("int16"), sum=T("int16"), dtype=qec.BF16)  # the bits of one
    takes("moe_rms_norm", x=4096, res=F32, sum=None, dtype=qec.F32)
    refuses("moe_rms_norm", x=F16, res=F16, sum=F16, dtype=qec.F32)
    refuses("moe_rms_norm", dtype=qec.BF16)
    refuses("moe_rms_norm", x=4096, dtype=qec.F16)


@pytest.mark.parametrize("call", sorted(ARGS))
def test_addresses_none_and_layout(call):
    for arg, right in ARGS[call].items():
        if isinstance(right, Tensor):
            takes(call, **{arg: None})
            takes(call, **{arg: 4096})
            refuses(call, **{arg: T(right.dtype.name, cuda=False)})
            refuses(call, **{arg: T(right.dtype.name, contiguous=False)})
