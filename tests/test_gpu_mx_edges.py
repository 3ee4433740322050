"""The microscaled operators at the edges of what they accept: launches that follow each other at once,
values at the ends of the range, captured calls (64-bit forms and bounds of mx_ref.py)."""
import os
import sys

import pytest
import torch

import mixture_experts_layer_logits_b200 as moe

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import mx_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for -m gpu tests")
    from mixture_experts_layer_logits_b200 import build

    build.build()
    moe.load_library()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(*shape, g):
    return torch.randn(*shape, generator=g, device="cuda")


def offsets_of(counts):
    return torch.tensor([0] + list(counts), dtype=I32, device="cuda").cumsum(0).to(I32)


def mm_operands(counts, N, K, seed):
    g = gen(seed)
    R, E = sum(counts), len(counts)
    return (*moe.moe_quantize_mx(randn(max(R, 1), K, g=g).to(BF16), "e4m3"),
            *moe.moe_quantize_mx(randn(E, N, K, g=g).to(BF16)), offsets_of(counts))


# ------------------------------------------------------------------ launches that follow each other


def test_launches_that_follow_each_other_at_once():
    """A launch's shared memory goes to the next one's CTAs, whose barriers lie elsewhere in it: an arrival
    that outlives its launch would be counted there.  Kernels of every tile width in turn, among
    them some with no tile, one, or fewer than there are pairs of CTAs."""
    shapes = [([1], 8, 128), ([0, 0], 128, 128), ([30, 2], 136, 256), ([64], 512, 640), ([100, 0, 90], 264, 384),
              ([500], 256, 128), ([3] * 40, 1160, 128)]
    calls = []
    for i, (counts, N, K) in enumerate(shapes):
        ops = mm_operands(counts, N, K, 100 + i)
        ws = torch.empty(moe.moe_grouped_mm_workspace_size(ops[0].shape[0], len(counts), N, K), dtype=U8,
                         device="cuda")
        y = torch.zeros(ops[0].shape[0], N, dtype=BF16, device="cuda")
        want, tol = ref.grouped_mm(ref.decode(ops[0], ops[1], "e4m3"), ops[2], ops[3], ops[4])
        moe.moe_grouped_mm_mx4(*ops, ws=ws, y=y)
        assert moe.moe_device_status(ws) == moe.MOE_OK
        n = sum(counts)
        ref.assert_within(y[:n], want[:n], tol[:n], f"y {i}")
        calls.append((ops, ws, y, y.clone()))
    order = torch.randint(0, len(calls), (600,), generator=torch.Generator().manual_seed(7)).tolist()
    for i in order:
        ops, ws, y, _ = calls[i]
        moe.moe_grouped_mm_mx4(*ops, ws=ws, y=y)
    for _, ws, y, first in calls:
        assert moe.moe_device_status(ws) == moe.MOE_OK
        assert torch.equal(y, first)
