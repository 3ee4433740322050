"""The microscaled operators on a GPU against their 64-bit forms (mx_ref.py, whose tolerances are
derived there), at the sizes and values where they can go wrong."""
import os
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


# ------------------------------------------------------------------ quantisation


def check_quantised(src, fmt):
    codes, scales = moe.moe_quantize_mx(src, fmt)
    want_codes, want_scales = ref.quantize(src.to(ref.F64), fmt)
    assert torch.equal(scales, want_scales)
    assert torch.equal(codes, want_codes)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(1, 32), (3, 32), (1, 96), (7, 4128), (257, 320), (5, 3, 64), (64,)])
def test_quantize_is_exact(shape, dtype, fmt):
    g = gen(1)
    src = randn(*shape, g=g) * torch.exp(3 * randn(*shape[:-1], 1, g=g))
    check_quantised(src.to(dtype), fmt)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_many_blocks_ragged_end(dtype, fmt):
    check_quantised(randn(5003, 1056, g=gen(1)).to(dtype), fmt)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_quantize_every_bf16_value(fmt):
    """Every finite bf16 value beside a largest magnitude of each binade: all ties, saturation,
    subnormal elements and scales, both zeros."""
    v = torch.arange(65536, dtype=I32, device="cuda").to(torch.int16).view(BF16)
    v = v[torch.isfinite(v)]
    v = torch.cat([v, v.new_zeros(-v.numel() % 31)]).view(-1, 31)
    for top in (0.0, 2.0 ** -133, 2.0 ** -126, 2.0 ** -120, 1.0, 1.9921875, 6.0, 448.0, 2.0 ** 127):
        check_quantised(torch.cat([v, v.new_full((v.shape[0], 1), top)], 1).contiguous(), fmt)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_quantize_fp32_ties_and_extremes(fmt):
    lv = ref.levels(fmt, "cuda")
    mids = (lv[1:] + lv[:-1]) / 2
    near = torch.cat([mids, mids * (1 + 2.0 ** -23), mids * (1 - 2.0 ** -23)]).float()
    near = torch.cat([near, -near])
    near = torch.cat([near, near.new_zeros(-near.numel() % 31)]).view(-1, 31)
    for s in (2.0 ** -130, 2.0 ** -60, 1.0, 2.0 ** 60, 2.0 ** 118):
        row = torch.cat([near, near.new_full((near.shape[0], 1), float(lv[-1]))], 1) * s
        check_quantised(row.contiguous(), fmt)
    tiny = torch.full((1, 32), 2.0 ** -149, device="cuda")
    check_quantised(tiny, fmt)
    check_quantised(torch.full((1, 32), torch.finfo(F32).max, device="cuda"), fmt)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_quantize_marks_blocks_that_are_not_finite(fmt, bad):
    src = randn(4, 128, g=gen(2)).to(BF16)
    clean_codes, clean_scales = moe.moe_quantize_mx(src, fmt)
    src[2, 70] = bad
    codes, scales = moe.moe_quantize_mx(src, fmt)
    hit = torch.zeros(4, 4, dtype=torch.bool, device="cuda")
    hit[2, 2] = True
    assert bool((scales[hit] == 255).all()) and torch.equal(scales[~hit], clean_scales[~hit])
    per = codes.view(4, 4, -1)
    assert bool((per[hit] == (0 if fmt == "e2m1" else 0x7F)).all())
    assert torch.equal(per[~hit], clean_codes.view(4, 4, -1)[~hit])


# ------------------------------------------------------------------ norm


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H", [(1, 32), (1, 2048), (3, 96), (5, 160), (64, 7168), (37, 1056),
                                 (2, 8192), (3, 8224), (2, 16384), (2, 32800), (1, 65536),
                                 (4099, 128)])
def test_norm(T, H, residual):
    g = gen(3)
    x = randn(T, H, g=g).to(BF16)
    res = (4 * randn(T, H, g=g)).to(BF16) if residual else None
    w = (1 + 0.3 * randn(H, g=g)).to(BF16)
    h, out, codes, scales = moe.moe_add_rmsnorm(x, w, 1e-6, residual=res, quantize=True)
    want_h, n, err = ref.rmsnorm(x, res, w, 1e-6)
    if residual:
        assert torch.equal(h, want_h)
    else:
        assert h is None
    ref.assert_within(out, n, err + ref.BF16_HALF_STEP * (n.abs() + err), "out")
    ref.assert_within(ref.decode(codes, scales, "e4m3"), ref.mx(n), ref.mx_shift(n, err), "codes")
    # without the blocks, and with outputs that the caller owns; the residual in place
    out2 = torch.empty_like(out)
    h2, got2, none, none2 = moe.moe_add_rmsnorm(x, w, 1e-6, residual=res, out=out2, sum_out=res)
    assert got2 is out2 and none is None and none2 is None and torch.equal(out2, out)
    if residual:
        assert h2 is res and torch.equal(res, h)


@pytest.mark.parametrize("T,H", [(1035, 4128), (1100, 2080), (1100, 6176), (1100, 8224), (1100, 16416)])
def test_norm_many_rows(T, H):
    test_norm(T, H, True)


def test_norm_extremes():
    """A zero row is zero (eps > 0), a huge row does not overflow before 2^64, tiny rows are scaled by
    eps, and a row with a NaN or an infinity does not touch its neighbours."""
    H = 256
    x = randn(6, H, g=gen(4)).to(BF16)
    x[0] = 0
    x[1] *= 2.0 ** 40
    x[2] *= 2.0 ** -60
    x[4, 17] = float("nan")
    x[5, 3] = float("inf")
    w = torch.ones(H, dtype=BF16, device="cuda")
    _, out, codes, scales = moe.moe_add_rmsnorm(x, w, 1e-6, quantize=True)
    _, n, err = ref.rmsnorm(x[:4], None, w, 1e-6)
    ref.assert_within(out[:4], n, err + ref.BF16_HALF_STEP * (n.abs() + err) + 2.0 ** -133, "out")
    ref.assert_within(ref.decode(codes[:4], scales[:4], "e4m3"), ref.mx(n), ref.mx_shift(n, err),
                      "codes")
    assert bool((out[0] == 0).all()) and bool(torch.isnan(out[4]).all())
    assert bool((scales[4] == 255).all())
    # infinity: 1 / sqrt(inf) = 0, so finite elements are 0 and the infinite one is NaN
    assert bool(torch.isnan(out[5, 3])) and int(torch.isnan(out[5]).sum()) == 1


# ------------------------------------------------------------------ grouped products


def offsets_of(counts):
    c = torch.tensor([0] + list(counts), dtype=I32, device="cuda")
    return c.cumsum(0).to(I32)


def draw_mm(R, E, N, K, seed=0):
    g = gen(seed)
    a, sa = ref.quantize(randn(R, K, g=g).to(ref.F64), "e4m3")
    w = torch.empty(E, N, K // 2, dtype=U8, device="cuda")
    sw = torch.empty(E, N, K // 32, dtype=U8, device="cuda")
    for e in range(E):
        w[e], sw[e] = ref.quantize(randn(N, K, g=g).to(ref.F64) * torch.exp(randn(N, 1, g=g)), "e2m1")
    return a, sa, w, sw


MM = [
    # counts per expert, N, K
    ([1], 8, 128), ([1], 128, 128), ([16], 136, 256), ([17], 264, 384), ([0, 3, 0, 0, 1, 0], 128, 256),
    ([5, 0, 31, 32, 33, 1], 376, 640), ([129, 64, 0, 255], 256, 128), ([300, 1, 0, 513], 520, 512),
    ([700, 33, 225, 0, 449], 384, 1152), ([2] * 200, 64, 128), ([40] * 9, 1160, 2176),
    ([0, 0, 4], 2048, 7168),
    # experts with many rows (pairs of CTAs), each pitch of the scale rows, one and many K tiles
    ([208], 256, 128), ([209, 300], 136, 768), ([416, 0, 1, 1000], 640, 512), ([150] * 7, 128, 2048),
    ([257, 129], 2056, 896), ([2000], 384, 256),
    # more than 32 tiles for each pair of CTAs, and more than 64
    ([3, 0, 20] * 100, 4096, 128), ([1] * 320, 4104, 256),
]


@pytest.mark.parametrize("counts,N,K", MM, ids=[f"E{len(c)}R{sum(c)}N{n}K{k}" for c, n, k in MM])
def test_grouped_mm(counts, N, K):
    R = sum(counts)
    a, sa, w, sw = draw_mm(R, len(counts), N, K)
    off = offsets_of(counts)
    ws = torch.empty(moe.moe_grouped_mm_workspace_size(R, len(counts), N, K), dtype=U8, device="cuda")
    y = moe.moe_grouped_mm_mx4(a, sa, w, sw, off, ws=ws)
    assert moe.moe_device_status(ws) == moe.MOE_OK
    want, tol = ref.grouped_mm(ref.decode(a, sa, "e4m3"), w, sw, off)
    ref.assert_within(y, want, tol, "y")
    # the same bits again
    assert torch.equal(moe.moe_grouped_mm_mx4(a, sa, w, sw, off), y)


@pytest.mark.parametrize("counts", [[77, 0, 126], [300, 0, 513]])
def test_grouped_mm_small_integers_are_exact(counts):
    """Small whole numbers under scales of one: every product and sum is exact, so a wrong element,
    scale or place cannot hide inside a tolerance."""
    g = gen(9)
    R, E, N, K = sum(counts), 3, 264, 384
    a = torch.randint(-4, 5, (R, K), generator=g, device="cuda")
    w = torch.randint(-4, 5, (E, N, K), generator=g, device="cuda")
    sa = torch.randint(125, 130, (R, K // 32), generator=g, device="cuda").to(U8)
    sw = torch.randint(125, 130, (E, N, K // 32), generator=g, device="cuda").to(U8)
    _, pa = ref.round_to(a.to(ref.F64), "e4m3")
    ca = (pa | ((a < 0).long() << 7)).to(U8)
    _, pw = ref.round_to(w.to(ref.F64), "e2m1")
    cw = (pw | ((w < 0).long() << 3)).to(U8)
    cw = cw[..., 0::2] | (cw[..., 1::2] << 4)
    off = offsets_of(counts)
    y = moe.moe_grouped_mm_mx4(ca, sa, cw.contiguous(), sw, off)
    want, _ = ref.grouped_mm(ref.decode(ca, sa, "e4m3"), cw, sw, off)
    assert torch.equal(y, want.to(F32).to(BF16))   # the sums fit fp32 exactly


@pytest.mark.parametrize("R", [300, 900])
def test_grouped_mm_leaves_rows_behind_the_last_group(R):
    a, sa, w, sw = draw_mm(R, 4, 256, 256)
    off = offsets_of([40, 0, 100, 3])
    y = torch.full((R, 256), 7.0, dtype=BF16, device="cuda")
    moe.moe_grouped_mm_mx4(a, sa, w, sw, off, y=y)
    want, tol = ref.grouped_mm(ref.decode(a, sa, "e4m3"), w, sw, off)
    ref.assert_within(y[:143], want[:143], tol[:143], "y")
    assert bool((y[143:] == 7.0).all())
    y.fill_(3.0)
    moe.moe_grouped_mm_mx4(a, sa, w, sw, torch.zeros_like(off), y=y)   # no rows at all
    assert bool((y == 3.0).all())


def test_grouped_mm_nan_blocks_stay_in_their_row_and_column():
    a, sa, w, sw = draw_mm(50, 2, 128, 256)
    off = offsets_of([30, 20])
    clean = moe.moe_grouped_mm_mx4(a, sa, w, sw, off)
    sa[7, 3] = 255
    a[41, 9] = 0x7F
    sw[1, 100, 2] = 255
    y = moe.moe_grouped_mm_mx4(a, sa, w, sw, off)
    bad = torch.zeros(50, 128, dtype=torch.bool, device="cuda")
    bad[7] = bad[41] = True
    bad[30:, 100] = True
    assert bool(torch.isnan(y[bad]).all()) and torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("R", [100, 700])
def test_grouped_mm_offsets_out_of_contract_stay_inside(R):
    """Offsets that descend or pass R are taken as empty or cut groups: nothing is read or written
    outside the operands."""
    a, sa, w, sw = draw_mm(R, 4, 136, 128)
    buf, y = guarded((R, 136), BF16)
    y.fill_(2.0)
    off = torch.tensor([0, 50, 20, R + 500, R - 10], dtype=I32, device="cuda")
    ws = torch.empty(moe.moe_grouped_mm_workspace_size(R, 4, 136, 128), dtype=U8, device="cuda")
    moe.moe_grouped_mm_mx4(a, sa, w, sw, off, ws=ws, y=y)
    moe.moe_grouped_mm_mx4(a, sa, w, sw, -off - 1, ws=ws, y=y)
    assert moe.moe_device_status(ws) == moe.MOE_OK and intact(buf)


def test_grouped_mm_extreme_scales():
    """Scales at both ends: a product of 2^-127 and 2^127 blocks is ordinary, and sums beyond bf16's
    range are infinite."""
    a, sa, w, sw = draw_mm(20, 1, 128, 128)
    off = offsets_of([20])
    sa[:], sw[:] = 0, 254
    y = moe.moe_grouped_mm_mx4(a, sa, w, sw, off)
    want, tol = ref.grouped_mm(ref.decode(a, sa, "e4m3"), w, sw, off)
    ref.assert_within(y, want, tol, "y")


# ------------------------------------------------------------------ past 32-bit offsets


def test_norm_and_quantize_past_2_to_31_elements():
    T, H = 70_001, 32_768
    x = torch.empty(T, H, dtype=BF16, device="cuda")
    for i in range(0, T, 10_000):
        x[i:i + 10_000] = randn(min(10_000, T - i), H, g=gen(60 + i))
    w = (1 + 0.1 * randn(H, g=gen(61))).to(BF16)
    _, out, codes, scales = moe.moe_add_rmsnorm(x, w, quantize=True)
    pick = torch.tensor([0, 1, 65_535, 65_536, T - 1], device="cuda")
    _, n, err = ref.rmsnorm(x[pick], None, w, 1e-6)
    ref.assert_within(out[pick], n, err + ref.BF16_HALF_STEP * (n.abs() + err), "out")
    ref.assert_within(ref.decode(codes[pick], scales[pick], "e4m3"), ref.mx(n), ref.mx_shift(n, err),
                      "codes")
    for fmt in ("e2m1", "e4m3"):
        codes, scales = moe.moe_quantize_mx(x, fmt)
        want = ref.quantize(x[pick].to(ref.F64), fmt)
        assert torch.equal(codes[pick], want[0]) and torch.equal(scales[pick], want[1])


def test_grouped_mm_output_past_2_to_31_elements():
    counts, N, K = [30_000, 3, 39_998], 32_776, 128
    R = sum(counts)
    a, sa = moe.moe_quantize_mx(randn(R, K, g=gen(62)).to(BF16), "e4m3")
    w, sw = moe.moe_quantize_mx(randn(3, N, K, g=gen(63)).to(BF16))
    y = moe.moe_grouped_mm_mx4(a, sa, w, sw, offsets_of(counts))
    for lo, e in ((0, 0), (29_999, 0), (30_000, 1), (30_002, 1), (30_003, 2), (65_530, 2), (R - 1, 2)):
        rows = ref.decode(a[lo:lo + 1], sa[lo:lo + 1], "e4m3")
        want, tol = ref.grouped_mm(rows, w[e:e + 1], sw[e:e + 1], offsets_of([1]))
        ref.assert_within(y[lo:lo + 1], want, tol, f"row {lo}")


def test_grouped_mm_weights_past_2_to_31_bytes():
    E, N, K = 300, 32_768, 512
    w = torch.randint(0, 256, (E, N, K // 2), generator=gen(64), device="cuda", dtype=U8)
    sw = torch.randint(120, 130, (E, N, K // 32), generator=gen(65), device="cuda", dtype=U8)
    a, sa = moe.moe_quantize_mx(randn(6, K, g=gen(66)).to(BF16), "e4m3")
    counts = [0] * E
    counts[1], counts[-2], counts[-1] = 2, 1, 3
    y = moe.moe_grouped_mm_mx4(a, sa, w, sw, offsets_of(counts))
    rows = ref.decode(a, sa, "e4m3")
    for lo, hi, e in ((0, 2, 1), (2, 3, E - 2), (3, 6, E - 1)):
        want, tol = ref.grouped_mm(rows[lo:hi], w[e:e + 1], sw[e:e + 1], offsets_of([hi - lo]))
        ref.assert_within(y[lo:hi], want, tol, f"expert {e}")


# ------------------------------------------------------------------ the FFN and the layer


def draw_ffn(T, E, k, H, I, seed=0, zipf=0.0):
    w = wl.custom("mx", T, E, k, H, I, zipf_s=zipf)
    logits = wl.make_logits(w, seed, "cuda")
    g = gen(seed + 11)
    x, sx = ref.quantize(randn(T, H, g=g).to(ref.F64), "e4m3")
    w13 = torch.empty(E, 2 * I, H // 2, dtype=U8, device="cuda")
    s13 = torch.empty(E, 2 * I, H // 32, dtype=U8, device="cuda")
    w2 = torch.empty(E, H, I // 2, dtype=U8, device="cuda")
    s2 = torch.empty(E, H, I // 32, dtype=U8, device="cuda")
    for e in range(E):
        w13[e], s13[e] = ref.quantize(randn(2 * I, H, g=g).to(ref.F64) / H ** 0.5, "e2m1")
        w2[e], s2[e] = ref.quantize(randn(H, I, g=g).to(ref.F64) / I ** 0.5, "e2m1")
    return logits, (x, sx, w13, s13, w2, s2)


FFN = [
    # T, E, k, H, I
    (1, 1, 1, 128, 128), (1, 8, 2, 256, 384), (3, 128, 8, 256, 128), (16, 8, 2, 256, 512),
    (17, 4, 3, 384, 640), (40, 1024, 16, 128, 128), (64, 32, 8, 896, 256), (100, 8, 2, 384, 640),
    (257, 2, 1, 256, 128), (600, 4, 2, 256, 256), (1100, 16, 4, 256, 256), (8, 128, 8, 2048, 768),
    (400, 300, 3, 128, 2048),  # more than 64 tiles of w13 for each pair of CTAs
]


@pytest.mark.parametrize("T,E,k,H,I", FFN)
def test_grouped_ffn_and_forward(T, E, k, H, I):
    logits, ops = draw_ffn(T, E, k, H, I)
    ids, wts = moe.moe_route(logits, k)
    off, rows = moe.moe_permute(ids, E)
    ws = moe.workspace_mx4(T, E, k, H, I)
    y = moe.moe_grouped_ffn_mx4(*ops, off, rows, k, ws=ws)
    assert moe.moe_device_status(ws) == moe.MOE_OK
    x, sx, *weights = ops
    want, tol = ref.grouped_ffn(ref.decode(x, sx, "e4m3"), *weights, off, rows, k)
    ref.assert_within(y, want, tol, "y")
    # the layer is the same steps
    out = moe.moe_forward_mx4(x, sx, logits, *weights, k, ws=ws)
    assert moe.moe_device_status(ws) == moe.MOE_OK
    assert torch.equal(out, moe.moe_combine(y, wts))
    got = [torch.empty_like(ids), torch.empty_like(wts), torch.empty_like(off), torch.empty_like(rows)]
    again = moe.moe_forward_mx4(x, sx, logits, *weights, k, topk_ids=got[0], topk_weights=got[1],
                                expert_offsets=got[2], permuted_rows=got[3])
    assert torch.equal(again, out)
    for a, b in zip(got, (ids, wts, off, rows)):
        assert torch.equal(a, b)


def test_ffn_with_skewed_routing():
    T, E, k, H, I = 777, 16, 2, 256, 384
    logits, ops = draw_ffn(T, E, k, H, I, seed=3, zipf=1.2)
    ids, _ = moe.moe_route(logits, k)
    off, rows = moe.moe_permute(ids, E)
    y = moe.moe_grouped_ffn_mx4(*ops, off, rows, k)
    x, sx, *weights = ops
    want, tol = ref.grouped_ffn(ref.decode(x, sx, "e4m3"), *weights, off, rows, k)
    ref.assert_within(y, want, tol, "y")


@pytest.mark.parametrize("T", [9, 300])
def test_ffn_token_with_nan_stays_alone(T):
    E, k, H, I = 4, 2, 256, 256
    logits, ops = draw_ffn(T, E, k, H, I, seed=5)
    x, sx, *weights = ops
    clean = moe.moe_forward_mx4(x, sx, logits, *weights, k)
    sx[2, 1] = 255
    out = moe.moe_forward_mx4(x, sx, logits, *weights, k)
    assert bool(torch.isnan(out[2]).all())
    keep = torch.arange(T, device="cuda") != 2
    assert torch.equal(out[keep], clean[keep])


# ------------------------------------------------------------------ as a program uses them


def layer_step(x, residual, norm_w, router, experts, k):
    h, n, q, s = moe.moe_add_rmsnorm(x, norm_w, 1e-6, residual=residual, quantize=True)
    logits = n.float() @ router
    return h, moe.moe_forward_mx4(q, s, logits, *experts, k)


def test_norm_quantize_and_layer_together():
    """Weights quantised at load time, then two layers' worth of norm, routing and experts."""
    T, E, k, H, I = 48, 16, 4, 512, 256
    g = gen(21)
    w13, w2 = wl.make_weights(wl.custom("run", T, E, k, H, I), seed=21, device="cuda")
    q13, s13 = moe.moe_quantize_mx(w13)
    q2, s2 = moe.moe_quantize_mx(w2)
    router = randn(H, E, g=g) / H ** 0.5
    norm_w = (1 + 0.1 * randn(H, g=g)).to(BF16)
    x, res = randn(T, H, g=g).to(BF16), randn(T, H, g=g).to(BF16)
    for _ in range(2):
        h, out = layer_step(x, res, norm_w, router, (q13, s13, q2, s2), k)
        want_h, n, _ = ref.rmsnorm(x, res, norm_w, 1e-6)
        assert torch.equal(h, want_h)
        _, nb, q, s = moe.moe_add_rmsnorm(x, norm_w, 1e-6, residual=res, quantize=True)
        ids, wts = moe.moe_route(nb.float() @ router, k)
        off, rows = moe.moe_permute(ids, E)
        y, tol = ref.grouped_ffn(ref.decode(q, s, "e4m3"), q13, s13, q2, s2, off, rows, k)
        p = wts.to(ref.F64).unsqueeze(-1)
        want = (p * y.view(T, k, H)).sum(1)
        # k fp32 products and sums, then one rounding to bf16
        mag = (p * (y.abs() + tol).view(T, k, H)).sum(1)
        bound = (p * tol.view(T, k, H)).sum(1) + 2 * k * ref.FP32_STEP * mag
        ref.assert_within(out, want, bound + ref.BF16_HALF_STEP * (want.abs() + bound), "out")
        x, res = out, h


@pytest.mark.parametrize("T", [5, 700])
def test_captured_step_replays_on_new_inputs(T):
    E, k, H, I = 16, 8, 256, 128
    g = gen(31)
    w13, w2 = wl.make_weights(wl.custom("cap", T, E, k, H, I), seed=31, device="cuda")
    experts = (*moe.moe_quantize_mx(w13), *moe.moe_quantize_mx(w2))
    router = randn(H, E, g=g) / H ** 0.5
    norm_w = (1 + 0.1 * randn(H, g=g)).to(BF16)
    x, res = randn(T, H, g=g).to(BF16), randn(T, H, g=g).to(BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer_step(x, res, norm_w, router, experts, k)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, out = layer_step(x, res, norm_w, router, experts, k)
    for i in range(3):
        x.copy_(randn(T, H, g=g))
        res.copy_(randn(T, H, g=g))
        graph.replay()
        graph.replay()
        want_h, want = layer_step(x, res, norm_w, router, experts, k)
        assert torch.equal(h, want_h) and torch.equal(out, want), i


def test_two_streams_with_workspaces_of_their_own():
    T, E, k, H, I = 200, 8, 2, 256, 256
    sets = [draw_ffn(T, E, k, H, I, seed=s) for s in (41, 42)]
    want = [moe.moe_forward_mx4(o[0], o[1], lg, *o[2:], k) for lg, o in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (lg, o) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                got[i].append(moe.moe_forward_mx4(o[0], o[1], lg, *o[2:], k))
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(w, o) for o in outs)


def guarded(shape, dtype, fill=0xA5, band=4096):
    n = torch.empty(shape, dtype=dtype, device="meta").nbytes
    buf = torch.full((n + 2 * band,), fill, dtype=U8, device="cuda")
    return buf, buf[band:band + n].view(dtype).view(*shape)


def intact(buf, band=4096, fill=0xA5):
    return bool((buf[:band] == fill).all()) and bool((buf[-band:] == fill).all())


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 256, 384), (9, 37, 3, 384, 128), (300, 4, 2, 640, 256)])
def test_calls_write_only_their_buffers(T, E, k, H, I):
    logits, (x, sx, *weights) = draw_ffn(T, E, k, H, I, seed=51)
    ids, _ = moe.moe_route(logits, k)
    off, rows = moe.moe_permute(ids, E)
    bufs = []

    def take(*shape, dtype):
        b, t = guarded(shape, dtype)
        bufs.append(b)
        return t

    ws = take(moe.moe_mx4_workspace_size(T, E, k, H, I), dtype=U8)
    moe.moe_grouped_ffn_mx4(x, sx, *weights, off, rows, k, ws=ws, y=take(T * k, H, dtype=BF16))
    moe.moe_forward_mx4(x, sx, logits, *weights, k, ws=ws, out=take(T, H, dtype=BF16))
    R, N = T * k, 2 * I - 8
    w = weights[0][:, :N].contiguous()
    sw = weights[1][:, :N].contiguous()
    xr, sxr = x[rows.long() // k].contiguous(), sx[rows.long() // k].contiguous()
    wsm = take(moe.moe_grouped_mm_workspace_size(R, E, N, H), dtype=U8)
    moe.moe_grouped_mm_mx4(xr, sxr, w, sw, off, ws=wsm, y=take(R, N, dtype=BF16))
    src = randn(T, H, g=gen(52)).to(BF16)
    moe.moe_quantize_mx(src, "e2m1", take(T, H // 2, dtype=U8), take(T, H // 32, dtype=U8))
    moe.moe_quantize_mx(src, "e4m3", take(T, H, dtype=U8), take(T, H // 32, dtype=U8))
    moe.moe_add_rmsnorm(src, src[0].contiguous(), residual=src.clone(), quantize=True,
                        sum_out=take(T, H, dtype=BF16), out=take(T, H, dtype=BF16),
                        codes=take(T, H, dtype=U8), scales=take(T, H // 32, dtype=U8))
    torch.cuda.synchronize()
    assert all(intact(b) for b in bufs)
