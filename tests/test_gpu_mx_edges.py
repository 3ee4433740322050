"""The microscaled operators at the edges of what they accept: launches that follow each other at once,
values at the ends of the range, captured calls (64-bit forms and bounds of mx_ref.py)."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import mixture_experts_layer_logits_b200 as moe
from mixture_experts_layer_logits_b200 import workloads as wl

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


# ------------------------------------------------------------------ norm: the whole range of bf16


def check_norm(x, w, eps, residual=None):
    h, out, codes, scales = moe.moe_add_rmsnorm(x, w, eps, residual=residual, quantize=True)
    want_h, n, err = ref.rmsnorm(x, residual, w, eps)
    if residual is not None:
        assert torch.equal(h, want_h)
    # Below its normal numbers fp32 rounds by up to 2^-150: h brought to a root mean square of 2^-13
    # (an error that the weight and then r <= 2^14 multiply), its product with the weight (r), and n itself:
    # 2^-136 (|w| + 1) + 2^-150.  bf16 rounds by up to 2^-134 there.
    err = err + 2.0 ** -135 * (1 + w.to(ref.F64).abs())
    ref.assert_within(out, n, err + ref.BF16_HALF_STEP * (n.abs() + err) + 2.0 ** -134, "out")
    ref.assert_within(ref.decode(codes, scales, "e4m3"), ref.mx(n), ref.mx_shift(n, err), "codes")
    assert torch.equal(moe.moe_add_rmsnorm(x, w, eps, residual=residual)[1], out)   # without the blocks
    return out


@pytest.mark.parametrize("H", [32, 256, 4128, 65536])
@pytest.mark.parametrize("eps", [1e-6, 0.0, 1e-38])
def test_norm_of_rows_of_any_size(H, eps):
    """Rows scaled by 2^-120 .. 2^124, on both sides of where a sum of H squares overflows (2^64 / sqrt(H)) and
    underflows fp32."""
    e = torch.tensor([-120, -100, -80, -76, -66, -62, -50, -45, -20, 0, 40, 52, 55, 56, 57, 59, 60, 61, 63, 64, 65,
                      80, 100, 120, 124], device="cuda")
    x = randn(len(e), H, g=gen(70)).clamp(-4, 4).to(BF16)
    x = torch.ldexp(x.to(ref.F64), e[:, None]).to(BF16)
    w = (1 + 0.3 * randn(H, g=gen(71))).to(BF16)
    check_norm(x, w, eps)


@pytest.mark.parametrize("H", [32, 4128])
def test_norm_without_eps_does_not_depend_on_a_power_of_two(H):
    """One row times 2^-100 .. 2^120: every step scales exactly, so the norms are the same bits."""
    e = torch.arange(-100, 121, device="cuda")
    row = randn(1, H, g=gen(75)).clamp(-4, 4).to(BF16)
    x = torch.ldexp(row.to(ref.F64).expand(len(e), H), e[:, None]).to(BF16)
    w = (1 + 0.3 * randn(H, g=gen(76))).to(BF16)
    out = check_norm(x, w, 0.0)
    assert torch.equal(out, out[100:101].expand_as(out))


@pytest.mark.parametrize("T", [1, 5, 1100])
def test_norm_of_few_huge_or_tiny_elements(T):
    """One element that decides the row, beside ordinary ones, with the largest and smallest of bf16."""
    H = 4128
    top = torch.finfo(BF16).max
    for value in (top, -top, 2.0 ** 66, 2.0 ** 57):
        x = randn(T, H, g=gen(72)).to(BF16)
        x[T // 2, 77] = value
        check_norm(x, torch.ones(H, dtype=BF16, device="cuda"), 1e-6)
    x = torch.zeros(T, H, dtype=BF16, device="cuda")
    x[:, 5] = 2.0 ** -133
    check_norm(x, torch.ones(H, dtype=BF16, device="cuda"), 0.0)
    x[:] = top
    check_norm(x, torch.ones(H, dtype=BF16, device="cuda"), 1e-6, residual=torch.zeros_like(x))


@pytest.mark.parametrize("size", [-50, -10, 0, 40, 70, 110])
@pytest.mark.parametrize("T,H", [(3, 512), (1100, 4096), (2, 20480), (1, 65536)])
def test_norm_with_weights_of_any_size(T, H, size):
    """The product of a row and its weights may pass fp32's range where the norm does not."""
    x = torch.ldexp(randn(T, H, g=gen(73)).to(BF16), torch.tensor(size, device="cuda"))
    we = torch.tensor([-120, -90, -60, 0, 60, 90, 110, 124], device="cuda").repeat_interleave(64).repeat(H // 512)
    w = torch.ldexp(1 + 0.3 * randn(H, g=gen(74)).clamp(-2, 2), we).to(BF16)
    check_norm(x, w, 1e-30, residual=torch.zeros_like(x) if H == 4096 else None)


def test_norm_of_zero_rows_without_eps_is_nan():
    x = torch.zeros(2, 64, dtype=BF16, device="cuda")
    x[1] = 1
    _, out, _, scales = moe.moe_add_rmsnorm(x, x[1].clone(), 0.0, quantize=True)
    assert bool(torch.isnan(out[0]).all()) and bool((scales[0] == 255).all()) and bool((out[1] == 1).all())


# ------------------------------------------------------------------ products: the whole range of scales


def draw_codes(R, N, K, seed):
    g = gen(seed)
    a = torch.randint(0, 0x7F, (R, K), generator=g, device="cuda", dtype=U8)   # not negative
    w = torch.randint(0, 256, (1, N, K // 2), generator=g, device="cuda", dtype=U8)
    return a, w


def under_scales(a, w, sa, sw):
    A = torch.full((a.shape[0], a.shape[1] // 32), sa, dtype=U8, device="cuda")
    W = torch.full((1, w.shape[1], w.shape[2] // 16), sw, dtype=U8, device="cuda")
    y = moe.moe_grouped_mm_mx4(a, A, w, W, offsets_of([a.shape[0]]))
    want, tol = ref.grouped_mm(ref.decode(a, A, "e4m3"), w, W, offsets_of([a.shape[0]]))
    return y, want, tol


@pytest.mark.parametrize("R", [20, 300])
@pytest.mark.parametrize("sa,sw", [(254, 254), (200, 240), (240, 140), (140, 240), (250, 127), (127, 250), (186, 186)])
def test_products_past_the_largest_number_are_infinite(R, sa, sw):
    """Rows of one sign, so that no partial sum is larger than the whole: past fp32's or bf16's range the
    result is the infinity of its sign, and below it is the ordinary one."""
    a, w = draw_codes(R, 136, 384, 80)
    w &= 0x77
    w[0, 1::2] |= 0x88                                   # odd features: all weights negative
    y, want, tol = under_scales(a, w, sa, sw)
    # bf16 rounds to infinity from 2^128 (1 - 2^-9) on; a sum that may lie on either side of that is not looked at
    edge = 2.0 ** 128 * (1 - 2.0 ** -9)
    over, under = want.abs() - tol >= edge, want.abs() + tol < edge
    assert bool(over.any())
    assert torch.equal(y[over].to(ref.F64), torch.sign(want[over]) * float("inf"))
    ref.assert_within(y[under], want[under], tol[under], "y")


@pytest.mark.parametrize("R", [20, 300])
@pytest.mark.parametrize("sa,sw", [(1, 126), (100, 27), (60, 60), (0, 120), (120, 0), (40, 75), (10, 100), (40, 60),
                                   (0, 0)])
def test_products_below_the_smallest_normal_number(R, sa, sw):
    """Weights and products of either sign under scales that bring the sums below bf16's and fp32's normal numbers.  There
    each of K fp32 sums may round by 2^-149, and bf16 by half a step, 2^-134."""
    K = 384
    a, w = draw_codes(R, 136, K, 81)
    y, want, tol = under_scales(a, w, sa, sw)
    ref.assert_within(y, want, tol + K * 2.0 ** -149 + 2.0 ** -134, "y")


# ------------------------------------------------------------------ the index checks of the debug build

DEBUG_CHILD = """
import sys, torch
sys.path.insert(0, {root!r})
import mixture_experts_layer_logits_b200 as moe
from mixture_experts_layer_logits_b200 import workloads as wl
assert moe.library_path == moe.debug_library_path
T, E, k, H, I = {T}, 4, 2, 256, 256
d = wl.make_inputs(wl.custom("dbg", T, E, k, H, I), seed=1, device="cuda")
x, sx = moe.moe_quantize_mx(d["x"], "e4m3")
experts = (*moe.moe_quantize_mx(d["w13"]), *moe.moe_quantize_mx(d["w2"]))
off, rows = moe.moe_permute(moe.moe_route(d["logits"], k)[0], E)
ws = moe.workspace_mx4(T, E, k, H, I)
good = moe.moe_grouped_ffn_mx4(x, sx, *experts, off, rows, k, ws=ws)
assert moe.moe_device_status(ws) == moe.MOE_OK
at = {at} % rows.numel()
lost = int(rows[at])
rows[at] = {bad}
y = torch.full_like(good, 7.0)
moe.moe_grouped_ffn_mx4(x, sx, *experts, off, rows, k, ws=ws, y=y)
assert moe.moe_device_status(ws) == moe.MOE_ERR_DEVICE_BOUNDS
assert moe.moe_device_status(ws) == moe.MOE_OK
# the bad position reads and writes row 0 instead; every other row is as it was, the lost one not written
keep = torch.ones(T * k, dtype=torch.bool, device="cuda")
keep[0] = keep[lost] = False
assert torch.equal(y[keep], good[keep])
assert lost == 0 or bool((y[lost] == 7.0).all())
print("checked")
"""


@pytest.mark.parametrize("T,at,bad", [(1, 0, -1), (9, 1, 10 ** 9), (300, 1, -1), (300, -1, 600)])
def test_debug_build_leaves_other_rows_alone(T, at, bad):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", DEBUG_CHILD.format(root=root, T=T, at=at, bad=bad)],
                       env=dict(os.environ, MOE_LIBRARY="debug"), cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "checked" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]


# ------------------------------------------------------------------ SwiGLU far from zero


def test_swiglu_of_large_negative_gates():
    """Gates and ups that the products give exactly, 32 features of each, so that act's error is that of the
    activation alone: down to where e^g = 2^-251, with ups that bring the product back."""
    gates = [6.0, -0.25, -16.0, -48.0, -63.0, -64.0, -65.0, -80.0, -87.0, -87.5, -88.0, -90.0, -96.0, -104.0, -152.0,
             -174.0]
    ups = [1.5, -2.0 ** 30, 3 * 2.0 ** 60, 2.0 ** 100]
    H, blocks = 256, [(g, u) for g in gates for u in ups]
    I = 32 * len(blocks)
    w13 = torch.zeros(1, 2 * I, H, dtype=ref.F64)
    for b, (g, u) in enumerate(blocks):
        rest, at = abs(g), 0
        while rest:  # a power of two, or 1.5 of one, in a block of columns of its own
            p = 2.0 ** (int(rest).bit_length() - 1 if rest >= 1 else -2)
            p = 1.5 * p if 1.5 * p <= rest else p
            w13[0, 32 * b:32 * b + 32, 32 * at] = p if g > 0 else -p
            rest, at = rest - p, at + 1
        w13[0, I + 32 * b:I + 32 * b + 32, 5] = u
    w2 = torch.zeros(1, H, I, dtype=ref.F64)
    w2[0, torch.arange(H), 8 * torch.arange(H)] = 1   # four features of each block
    (q13, s13), (q2, s2) = ref.quantize(w13.cuda(), "e2m1"), ref.quantize(w2.cuda(), "e2m1")
    assert torch.equal(ref.decode(q13, s13, "e2m1"), w13.cuda())
    T = 3
    x = torch.tensor([1.0, 0.5, 1.0], dtype=ref.F64, device="cuda")[:, None].expand(T, H)
    qx, sx = ref.quantize(x, "e4m3")
    off, rows = offsets_of([T]), torch.arange(T, dtype=I32, device="cuda")
    y = moe.moe_grouped_ffn_mx4(qx, sx, q13, s13, q2, s2, off, rows, 1)
    h = x @ w13.cuda()[0].T
    act, err = ref.swiglu(h, torch.zeros_like(h))
    err = err + 2.0 ** -149   # a product below fp32's normal numbers
    want, tol = ref.grouped_mm(ref.mx(act), q2, s2, off, ref.mx_shift(act, err))
    ref.assert_within(y, want, tol + 2.0 ** -134, "y")   # half a step of bf16 below its normal numbers


# ------------------------------------------------------------------ captured calls on new inputs


def replayed(call, refill, rounds=4):
    """Captures call() and replays it on new contents of its inputs, twice in a row each time; yields its outputs
    beside those of an uncaptured call."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    for i in range(rounds):
        refill(i)
        graph.replay()
        graph.replay()
        yield [t.clone() for t in outs], call()


def distinct_ids(T, E, k, seed):
    return torch.topk(randn(T, E, g=gen(seed)), k, dim=1).indices.to(I32)


def sorted_by_expert(ids, E):
    flat = ids.flatten().long()
    counts = torch.bincount(flat, minlength=E)
    return offsets_of(counts.tolist()), torch.argsort(flat, stable=True).to(I32)


@pytest.mark.parametrize("T,E,k", [(60, 64, 8), (700, 64, 8), (9000, 300, 4)])
@pytest.mark.parametrize("noalloc", [False, True])
def test_captured_permutation_on_new_ids(T, E, k, noalloc):
    ids = distinct_ids(T, E, k, 1)
    ws = moe.workspace(T, E, k)

    def call():
        if not noalloc:
            return moe.moe_permute(ids, E, ws=ws)
        off = torch.empty(E + 1, dtype=I32, device="cuda")
        rows = torch.empty(T * k, dtype=I32, device="cuda")
        lib = moe.load_library()
        lib.moe_permute_noalloc.argtypes = [ctypes.c_void_p, moe.Shape] + [ctypes.c_void_p] * 3
        assert lib.moe_permute_noalloc(ids.data_ptr(), moe.Shape(T, E, k, 0, 0), off.data_ptr(), rows.data_ptr(),
                                       torch.cuda.current_stream().cuda_stream) == moe.MOE_OK
        return off, rows

    # skewed and even in turn, so that counts of the replay before would be far off
    def refill(i):
        ids.copy_(distinct_ids(T, E, k, 10 + i) if i % 2 else torch.arange(k, dtype=I32, device="cuda").expand(T, k))

    for got, again in replayed(call, refill):
        for a, b, want in zip(got, again, sorted_by_expert(ids, E)):
            assert torch.equal(a, want) and torch.equal(b, want)
    assert moe.moe_device_status(ws) == moe.MOE_OK


@pytest.mark.parametrize("kind,T", [("bf16", 8), ("bf16", 64), ("bf16", 700), ("w8", 1), ("w8", 8), ("w8", 64),
                                    ("mx4", 8), ("mx4", 700), ("steps", 700)])
def test_captured_layer_on_new_inputs(kind, T):
    """Inputs whose size changes by powers of two from replay to replay, so that a row scaled by what the
    replay before had published would be far off or saturate."""
    E, k, H, I = 16, 8, 256, 256
    w = wl.custom("cap", T, E, k, H, I)
    w13, w2 = wl.make_weights(w, seed=3, device="cuda")
    x, logits = randn(T, H, g=gen(4)).to(BF16), randn(T, E, g=gen(5))
    ws = moe.workspace(T, E, k, H, I)
    if kind == "w8":
        g = gen(6)
        c13 = torch.randint(0, 120, tuple(w13.shape), generator=g, device="cuda", dtype=U8)
        c2 = torch.randint(0, 120, tuple(w2.shape), generator=g, device="cuda", dtype=U8)
        s13 = torch.rand(E, 2 * I, generator=g, device="cuda") * 2.0 ** -12
        s2 = torch.rand(E, H, generator=g, device="cuda") * 2.0 ** -12
    if kind in ("mx4", "steps"):
        experts = (*moe.moe_quantize_mx(w13), *moe.moe_quantize_mx(w2))
        ws = moe.workspace_mx4(T, E, k, H, I)

    def call():
        if kind == "bf16":
            return [moe.moe_forward(x, logits, w13, w2, k, ws=ws)]
        if kind == "w8":
            return [moe.moe_forward_w8(x, logits, c13, s13, c2, s2, k, ws=ws)]
        q, s = moe.moe_quantize_mx(x, "e4m3")
        if kind == "mx4":
            return [moe.moe_forward_mx4(q, s, logits, *experts, k, ws=ws)]
        ids, p = moe.moe_route(logits, k)
        off, rows = moe.moe_permute(ids, E)
        y = moe.moe_grouped_ffn_mx4(q, s, *experts, off, rows, k, ws=ws)
        return [moe.moe_combine(y, p), off, rows]

    def refill(i):
        x.copy_(randn(T, H, g=gen(20 + i)) * 2.0 ** (6 * (i % 2) - 3))
        logits.copy_(randn(T, E, g=gen(40 + i)) * (1 + 9 * (i % 2)))

    last = None
    for got, again in replayed(call, refill):
        for a, b in zip(got, again):
            assert torch.equal(a, b)
        assert moe.moe_device_status(ws) == moe.MOE_OK
        assert last is None or not torch.equal(got[0], last)
        last = got[0]
