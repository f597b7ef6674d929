"""What programmatic dependent launches ask of the kernel sources, checked on the sources: such a kernel may be
resident while the kernel ahead of it still runs, and lets the kernel behind it become resident in turn."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixed_precision_residual_gb300", "csrc")
SOURCES = {os.path.basename(f): open(f).read() for pattern in ("*.cu", "*.cuh", "*.h")
           for f in sorted(glob.glob(os.path.join(CSRC, pattern)))}


def code(text):
    """The source without its comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("name", sorted(SOURCES))
def test_no_read_only_loads(name):
    """ld.global.nc and __ldg are for memory that nobody writes while the kernel lives, and a const __restrict__
    pointer lets the compiler choose them: what the kernel ahead writes is not that."""
    found = re.findall(r"ld\.global\.nc|__ldg|ld\.global\.[a-z:.]*nc|__restrict__", code(SOURCES[name]))
    assert not found, f"{name}: {found}"
