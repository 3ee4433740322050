"""What the sources of the microscaled kernels must keep to, whatever a run on one GPU shows."""
import glob
import os
import re
import subprocess
import sys

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


def test_feature_counts_that_cannot_be_rounded_up_are_refused():
    """A pair of CTAs takes 256 features; a count within 255 of 2^31 would overflow when rounded up to that, and the
    product would do nothing and report success."""
    import mixture_experts_layer_logits_b200 as moe
    from mixture_experts_layer_logits_b200 import build

    build.build()
    top = 2 ** 31 - 256
    assert moe.moe_grouped_mm_workspace_size(1, 1, top, 128) > 0
    assert moe.moe_grouped_mm_workspace_size(1, 1, 2 ** 31 - 8, 128) == 0
    assert moe.moe_grouped_mm_workspace_size(1, 3, (2 ** 31 - 8) // 24 * 8, 128) == 0
    assert moe.moe_mx4_workspace_size(1, 1, 1, top, 128) > 0
    assert moe.moe_mx4_workspace_size(1, 1, 1, 2 ** 31 - 128, 128) == 0


@pytest.fixture(scope="module")
def status_string():
    import mixture_experts_layer_logits_b200 as moe
    from mixture_experts_layer_logits_b200 import build

    build.build()
    return lambda status: moe.load_library().moe_status_string(status).decode()


def test_the_alignment_error_names_both_rules(status_string):
    """E2M1 weights that are 16-byte aligned only are refused with this status too."""
    import mixture_experts_layer_logits_b200 as moe

    text = status_string(moe.MOE_ERR_MISALIGNED)
    assert "16" in text and "E2M1" in text and "32" in text
    assert text in str(moe.MoeError(moe.MOE_ERR_MISALIGNED, "moe_grouped_mm_mx4"))


def test_the_argument_error_is_not_only_of_null_pointers(status_string):
    """A negative eps or an unknown format gets it as well."""
    import mixture_experts_layer_logits_b200 as moe

    assert "value" in status_string(moe.MOE_ERR_INVALID_ARG)


PUBLIC_ONLY = """
import sys, torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
torch.cuda.current_device = lambda: 0
torch.cuda.current_stream = lambda index: type("S", (), {"cuda_stream": 1234 + index})
import mixture_experts_layer_logits_b200 as moe
seen = []
moe._call(lambda *a: seen.append(a) or moe.MOE_OK, "f", torch.device("cuda", 0), 7)
assert seen == [(7, 1234)], seen
print("called")
"""


def test_calls_without_torchs_private_entries():
    r = subprocess.run([sys.executable, "-c", PUBLIC_ONLY], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "called" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
