"""What the sources of the layer's products must not hold, checked by reading them: no GPU shows
these faults on demand."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "relative_bias_hybrid_gb300", "csrc")


@pytest.mark.parametrize("name", ["linear.cu", "linear_few.cu", "route.cu"])
def test_no_non_coherent_loads(name):
    """Kernels that may be resident while the kernel before them still writes their inputs read
    them coherently, behind the wait for that kernel: ld.global.nc (__ldg, const __restrict__
    pointers) is for memory that nobody writes meanwhile."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    assert re.findall(r"__ldg|ld\.global\.nc|__restrict__", text) == []


@pytest.mark.parametrize("name,arrays", [
    ("output_conv.cu", ["y"]),                       # of inkattn_linear or inkattn_expert_combine
    ("prologue.cu", [r"reinterpret_cast<const uint4 \*>\(\s*qb", r"reinterpret_cast<const uint4 \*>\(p\.[kv] ",
                     r"reinterpret_cast<const uint4 \*>\(src"]),   # q, k and v, of inkattn_linear
    ("prefill_tc.cu", [r"src \+ j\);\s*\}\s*float n2",             # r, of inkattn_qkvr_prologue
                       r"p\.block_table"]),                          # (the expansion of an E4M3 cache writes one)
    ("prefill_2q.cu", [r"p\.block_table"]),
    ("decode_tc.cu", [r"reinterpret_cast<const uint32_t \*>\(rh"]),
    ("dequant.cu", [r"\(stream == 0 \? p\.k_scale", r"reinterpret_cast<const uint4 \*>\(codes"])])   # of the prologue
def test_outputs_of_early_kernels_are_read_coherently(name, arrays):
    """The same for what the other kernels read of a kernel that lets its successor start early."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    for a in arrays:
        assert not re.search(r"__ldg\(" + a, text), a
