"""A bounded wait may expire for some lanes of a warp and not for others, and an
instruction that takes the converged warp (elect.sync, a tcgen05 load or store, a
shuffle of all lanes) must not be met by the rest alone.  So in the kernel of the
4-bit linear layer's batches every wait or test of a barrier is one thread's, or
ends in a vote or a broadcast of the whole warp.  Such a parting of lanes cannot be
brought about from outside: this reads the source."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_expert_cache_gb300", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_a_warp_leaves_a_wait_as_one():
    src = _code("kernels_linear_gemm.cu")
    tma = src[src.index("if (warp == kWTma) {"):src.index("tma_done:;")]
    one_thread = tma[tma.index("if (lane == 0) {"):]  # the copies' thread
    rest = src.replace(one_thread, "")
    calls = re.findall(r"[^;{}]*\bmbar_(?:wait|wait_spin|wait_warp|test|try)\s*\(", rest)
    assert len(calls) >= 6
    for call in calls:
        assert "mbar_wait_warp(" in call or "__all_sync(0xffffffffu, mbar_test(" in call \
            or re.search(r"if \(lane == 0\) ok = mbar_wait\($", call), call
    # lane 0's outcome goes to all lanes before the next branch
    for after in re.split(r"if \(lane == 0\) ok = mbar_wait\(", rest)[1:]:
        assert re.match(r"[^;]*;\s*ok = __shfl_sync\(0xffffffffu, ok \? 1 : 0, 0\) != 0;", after), after[:200]


def test_the_warp_wait_votes():
    src = _code("tcgen05.cuh")
    body = src[src.index("bool mbar_wait_warp("):]
    assert "return __all_sync(0xffffffffu, mbar_wait_spin(" in body[:body.index("}")]
