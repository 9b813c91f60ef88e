"""The kernels of moe_rms_norm that are compiled are the ones a call can reach: the
launch rule restated, over widths, token counts and alignments, against the kernels
that the built library names."""
import re
import shutil
import subprocess

import pytest

import quantized_expert_cache_gb300 as qec


def kernel(size, width, tokens, aligned):
    """(elements a pack, packs a thread, a warp a row) of the rule, or None: the kernel of very wide rows."""
    many = tokens > 256
    if size == 2 and width % 8 == 0 and many and aligned:
        vec = 8
    else:
        vec = 4 if width % 4 == 0 and aligned else 1
    n = width // vec
    for items in (1, 2, 4):
        if n <= 32 * items:
            return vec, items, True
    if many and n <= 256:
        return vec, 8, True
    if not many and n <= 1024:
        return vec, 1, False
    if n <= 512:
        return (1, 16, True) if vec == 1 else (vec, 2, False)
    for items, most in ((4, 2048), (8, 8192)):
        if n <= most:
            return vec, items, False
    return None


def test_every_compiled_norm_kernel_can_be_reached():
    nm = shutil.which("nm")
    if nm is None:
        pytest.skip("needs nm")
    qec.load()
    names = subprocess.run([nm, "-C", qec.lib_path()], capture_output=True, text=True, check=True).stdout
    built = {(t, int(v), int(i), w == "true")
             for t, v, i, w in re.findall(r"rms_norm_kernel<(\w+), (\d+), (\d+), (true|false)>", names)}
    widths = sorted({max(1, (1 << s) + o) for s in range(18) for o in (-32, -1, 0, 1, 4, 8, 32)})
    reached = {(t,) + k for t, size in (("float", 4), ("__half", 2), ("__nv_bfloat16", 2)) for w in widths
               for tokens in (1, 256, 257, 5000) for aligned in (True, False)
               for k in [kernel(size, w, tokens, aligned)] if k}
    assert built == reached, (sorted(built - reached), sorted(reached - built))
