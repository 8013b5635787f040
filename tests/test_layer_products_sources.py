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
    pointers) is for memory that nobody writes meanwhile, and the header's __ldcs is no volatile
    load, so nothing keeps it behind the wait."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    assert re.findall(r"__ldg|__ldcs|ld\.global\.nc|__restrict__", text) == []
