"""What the sources of the microscaled kernels must keep to, whatever a run on one GPU shows."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "mixture_experts_layer_logits_b200", "csrc", "mx_*")))


def code(path):
    """The source without its comments."""
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_read_only_loads(path):
    """These kernels begin while the launch before them may still write what they read
    (programmatic dependent launch), and ld.global.nc wants its data unchanged for the kernel's
    whole life: no __ldg, and no const __restrict__ pointer, for which the compiler may choose it."""
    text = code(path)
    assert "__ldg(" not in text and "ld.global.nc" not in text
    assert not re.search(r"const\s+\w+\s*\*\s*(const\s+)?__restrict__", text)
