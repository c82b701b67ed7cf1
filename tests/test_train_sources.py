"""What the training operators' device sources must not hold, whatever a run shows (no GPU)."""
import os
import re

from nvfp4_quantized_b200 import build as qbuild


def device_sources():
    """The files of csrc that the training library is compiled from, comments taken out."""
    found, todo = {}, ["qt2_train.cu"]
    while todo:
        name = todo.pop()
        path = os.path.join(qbuild.CSRC, name)
        if name in found or not os.path.exists(path):
            continue
        text = re.sub(r"/\*.*?\*/|//[^\n]*", "", open(path).read(), flags=re.S)
        found[name] = text
        todo += re.findall(r'#include "([^"]+)"', text)
    assert {"norm_kernels.cuh", "xent_kernels.cuh", "grad_kernels.cuh"} <= set(found)
    return found


def test_no_read_only_loads():
    """Every kernel starts while the one before it in the stream may still write what it is going to
    read.  Loads that promise memory which nobody writes during the kernel's life are bound neither
    by the wait for that kernel nor by the compiler's order around it."""
    for name, text in device_sources().items():
        for pattern in (r"__ldg\w*\s*\(", r"\bld\.global\.\w*\.?nc\b", r"\.nc\.", r"__restrict(__)?\b", r"\btex\w+Dfetch"):
            assert not re.search(pattern, text), (name, pattern)
