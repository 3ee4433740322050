"""Index checks of the debug build in the microscaled kernels: a permuted row outside [0, T*k) is
reported by moe_device_status and its access redirected, in the streaming and in the pair form.
The debug library is chosen at import, so each case runs in a child process.
"""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import sys, torch
sys.path.insert(0, {root!r})
import mixture_experts_layer_logits_b200 as moe
from mixture_experts_layer_logits_b200 import workloads as wl
assert moe.library_path == moe.debug_library_path
T, E, k, H, I = {T}, 4, 2, 256, 256
w = wl.custom("dbg", T, E, k, H, I)
d = wl.make_inputs(w, seed=1, device="cuda")
x, sx = moe.moe_quantize_mx(d["x"], "e4m3")
w13, s13 = moe.moe_quantize_mx(d["w13"])
w2, s2 = moe.moe_quantize_mx(d["w2"])
ids, _ = moe.moe_route(d["logits"], k)
off, rows = moe.moe_permute(ids, E)
ws = moe.workspace_mx4(T, E, k, H, I)
good = moe.moe_grouped_ffn_mx4(x, sx, w13, s13, w2, s2, off, rows, k, ws=ws)
assert moe.moe_device_status(ws) == moe.MOE_OK
rows[1] = {bad}
moe.moe_grouped_ffn_mx4(x, sx, w13, s13, w2, s2, off, rows, k, ws=ws)
assert moe.moe_device_status(ws) == moe.MOE_ERR_DEVICE_BOUNDS
assert moe.moe_device_status(ws) == moe.MOE_OK
print("checked")
"""


@pytest.mark.parametrize("T", [9, 300])
@pytest.mark.parametrize("bad", [-1, 10**9])
def test_permuted_row_out_of_range_is_reported(T, bad):
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for -m gpu tests")
    from mixture_experts_layer_logits_b200 import build

    build.build()
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, T=T, bad=bad)],
                       env=dict(os.environ, MOE_LIBRARY="debug"), cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "checked" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]
