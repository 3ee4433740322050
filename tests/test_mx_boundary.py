"""The microscaled entry points refuse bad calls on the host, and the formats' 64-bit
reference agrees with torch's own E4M3 rounding.  As in test_boundary.py the calls pass
made-up device addresses in a child process that sees no GPU."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import mixture_experts_layer_logits_b200 as moe

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import mx_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NO_DEVICE = os.environ.get("CUDA_VISIBLE_DEVICES") == ""
A = ctypes.c_void_p(0x7f0000001000)
A16 = ctypes.c_void_p(0x7f0000001010)  # 16-byte aligned only
MIS = ctypes.c_void_p(0x7f0000001004)
NUL = None


@pytest.mark.skipif(NO_DEVICE, reason="this is the child process")
def test_boundary_checks_in_a_process_without_a_device():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        "-m", "not gpu", os.path.abspath(__file__)],
                       env=env, cwd=ROOT, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and " failed" not in r.stdout, r.stdout[-2000:]


@pytest.fixture(scope="module")
def lib():
    if not NO_DEVICE:
        pytest.skip("runs in the child process without a device")
    from mixture_experts_layer_logits_b200 import build

    build.build()
    return moe.load_library()


def variants(args, at, value):
    for i in at:
        bad = list(args)
        bad[i] = value
        yield bad


def test_quantize_validation(lib):
    f = lib.moe_quantize_mx
    ok = [A, 0, 4, 64, 0, A, A, None]
    for bad in variants(ok, (0, 5, 6), NUL):
        assert f(*bad) == moe.MOE_ERR_INVALID_ARG
    for bad in variants(ok, (0, 5, 6), MIS):
        assert f(*bad) == moe.MOE_ERR_MISALIGNED
    for i, value in ((1, 2), (1, -1), (4, 2), (4, -1)):
        assert f(*next(variants(ok, (i,), value))) == moe.MOE_ERR_INVALID_ARG
    for i, value in ((2, 0), (2, -1), (3, 0), (3, 16), (3, 40), (3, -32), (2, 1 << 38)):
        assert f(*next(variants(ok, (i,), value))) == moe.MOE_ERR_UNSUPPORTED_SHAPE


def test_norm_validation(lib):
    f = lib.moe_add_rmsnorm
    ok = [A, A, A, 4, 64, 1e-6, A, A, A, A, None]
    for bad in variants(ok, (0, 2, 1, 6, 8, 9), NUL):   # 1 / 6 and 8 / 9 go in pairs
        assert f(*bad) == moe.MOE_ERR_INVALID_ARG
    none = list(ok)
    none[7] = none[8] = none[9] = NUL
    assert f(*none) == moe.MOE_ERR_INVALID_ARG
    for bad in variants(ok, (0, 1, 2, 6, 7, 8, 9), MIS):
        assert f(*bad) == moe.MOE_ERR_MISALIGNED
    for i, value in ((3, 0), (3, -1), (4, 0), (4, 16), (4, 48), (4, 65568)):
        assert f(*next(variants(ok, (i,), value))) == moe.MOE_ERR_UNSUPPORTED_SHAPE
    for eps in (-1e-6, float("nan")):
        assert f(*next(variants(ok, (5,), eps))) == moe.MOE_ERR_INVALID_ARG


def M(R=64, E=8, N=256, K=256):
    return moe.MmShape(R, E, N, K)


def test_grouped_mm_validation(lib):
    f = lib.moe_grouped_mm_mx4
    n = lib.moe_grouped_mm_workspace_size(M())
    assert n > 0 and n % 256 == 0
    ok = [A, A, A, A, A, M(), A, A, n, None]
    for bad in variants(ok, (0, 1, 2, 3, 4, 6, 7), NUL):
        assert f(*bad) == moe.MOE_ERR_INVALID_ARG
    for bad in variants(ok, (0, 1, 2, 3, 4, 6, 7), MIS):
        assert f(*bad) == moe.MOE_ERR_MISALIGNED
    assert f(*next(variants(ok, (2,), A16))) == moe.MOE_ERR_MISALIGNED
    assert f(*next(variants(ok, (8,), n - 1))) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    for s in (M(R=0), M(E=0), M(E=1025), M(N=0), M(N=12), M(K=0), M(K=64), M(K=192), M(R=-1),
              M(R=(1 << 30) + 1), M(E=1024, N=1 << 22), M(R=1 << 30, N=2048)):
        assert f(*next(variants(ok, (5,), s))) == moe.MOE_ERR_UNSUPPORTED_SHAPE
        assert lib.moe_grouped_mm_workspace_size(s) == 0


def S(T=8, E=128, k=8, H=2048, I=768):
    return moe.Shape(T, E, k, H, I)


BAD_SHAPES = (S(H=200), S(I=100), S(H=0), S(E=0), S(T=0), S(k=17), S(E=4, k=5), S(E=1025))


def test_grouped_ffn_mx4_validation(lib):
    f = lib.moe_grouped_ffn_mx4
    n = lib.moe_mx4_workspace_size(S())
    assert n > 0 and n % 256 == 0
    ok = [A] * 8 + [S(), A, A, n, None]
    pointers = (0, 1, 2, 3, 4, 5, 6, 7, 9, 10)
    for bad in variants(ok, pointers, NUL):
        assert f(*bad) == moe.MOE_ERR_INVALID_ARG
    for bad in variants(ok, pointers, MIS):
        assert f(*bad) == moe.MOE_ERR_MISALIGNED
    for bad in variants(ok, (2, 4), A16):
        assert f(*bad) == moe.MOE_ERR_MISALIGNED
    for s in BAD_SHAPES:
        assert f(*next(variants(ok, (8,), s))) == moe.MOE_ERR_UNSUPPORTED_SHAPE
        assert lib.moe_mx4_workspace_size(s) == 0
    assert f(*next(variants(ok, (11,), n - 1))) == moe.MOE_ERR_WORKSPACE_TOO_SMALL


def test_forward_mx4_validation(lib):
    f = lib.moe_forward_mx4
    n = lib.moe_mx4_workspace_size(S())
    ok = [A] * 7 + [S(), A, NUL, NUL, NUL, NUL, A, n, None]
    needed = (0, 1, 2, 3, 4, 5, 6, 8, 13)
    for bad in variants(ok, needed, NUL):
        assert f(*bad) == moe.MOE_ERR_INVALID_ARG
    for bad in variants(ok, needed + (9, 10, 11, 12), MIS):
        assert f(*bad) == moe.MOE_ERR_MISALIGNED
    for bad in variants(ok, (3, 5), A16):
        assert f(*bad) == moe.MOE_ERR_MISALIGNED
    for s in BAD_SHAPES:
        assert f(*next(variants(ok, (7,), s))) == moe.MOE_ERR_UNSUPPORTED_SHAPE
    assert f(*next(variants(ok, (14,), n - 1))) == moe.MOE_ERR_WORKSPACE_TOO_SMALL


def test_bindings_refuse_tensors(lib):
    """The Python calls refuse host tensors and wrong types, shapes and strides."""
    u8, bf = torch.uint8, torch.bfloat16
    x = torch.zeros(4, 256, dtype=bf)
    with pytest.raises(ValueError):
        moe.moe_quantize_mx(x)                                    # not on a GPU
    with pytest.raises(ValueError):
        moe.moe_quantize_mx(x, "e5m2")
    with pytest.raises(ValueError):
        moe.moe_quantize_mx(x.half())
    with pytest.raises(ValueError):
        moe.moe_quantize_mx(x.t())
    with pytest.raises(moe.MoeError):
        moe.moe_quantize_mx(torch.zeros(4, 40, dtype=bf))
    with pytest.raises(moe.MoeError):
        moe.moe_quantize_mx(torch.zeros(0, 64, dtype=bf))
    with pytest.raises(ValueError):
        moe.moe_quantize_mx(x, codes=torch.zeros(4, 256, dtype=u8))
    w = torch.zeros(256, dtype=bf)
    with pytest.raises(ValueError):
        moe.moe_add_rmsnorm(x, w)                                 # not on a GPU
    with pytest.raises(ValueError):
        moe.moe_add_rmsnorm(x, w[:128])
    with pytest.raises(ValueError):
        moe.moe_add_rmsnorm(x, w, residual=x.float())
    with pytest.raises(ValueError):
        moe.moe_add_rmsnorm(x, w, sum_out=x.clone())
    with pytest.raises(ValueError):
        moe.moe_add_rmsnorm(x, w, codes=torch.zeros(4, 256, dtype=u8))
    with pytest.raises(moe.MoeError):
        moe.moe_add_rmsnorm(x[:, :40].contiguous(), w[:40])
    a, sa = torch.zeros(6, 256, dtype=u8), torch.zeros(6, 8, dtype=u8)
    b, sb = torch.zeros(2, 64, 128, dtype=u8), torch.zeros(2, 64, 8, dtype=u8)
    off = torch.zeros(3, dtype=torch.int32)
    for args in ((a, sa, b, sb, off), (a, sa[:5], b, sb, off), (a, sa, b[:, :, :64], sb, off),
                 (a, sa, b, sb[:1], off), (a, sa, b, sb, off.long()), (a, sa, b, sb, off[:2])):
        with pytest.raises(ValueError):
            moe.moe_grouped_mm_mx4(*args)
    with pytest.raises(moe.MoeError):
        moe.moe_grouped_mm_mx4(a[:, :64].contiguous(), sa[:, :2].contiguous(),
                               b[:, :, :32].contiguous(), sb[:, :, :2].contiguous(), off)


def test_e4m3_reference_against_torch():
    """The reference's E4M3 rounding, ties included, is torch's own saturating cast; an E2M1 tie goes
    to the even code."""
    v = torch.arange(0, 65536, dtype=torch.int32).to(torch.uint16).view(torch.bfloat16)
    v = v[torch.isfinite(v) & (v.abs() <= 448)].to(torch.float64)
    mids = torch.tensor(ref.E4M3, dtype=ref.F64)
    v = torch.cat([v, (mids[1:] + mids[:-1]) / 2])
    value, _ = ref.round_to(v, "e4m3")
    want = v.float().to(torch.float8_e4m3fn).double().abs()
    assert torch.equal(value, want)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 100.0], dtype=ref.F64)
    assert ref.round_to(ties, "e2m1")[0].tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 6.0]


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_reference_round_trip_and_shift(fmt):
    """Decoding gives back values that are in the format, and mx_shift bounds what a perturbation
    of the given size does."""
    g = torch.Generator().manual_seed(5)
    v = torch.randn(64, 96, generator=g, dtype=ref.F64)
    q = ref.mx(v, fmt)
    assert torch.equal(ref.mx(q, fmt), q)
    err = v.abs() * 1e-2
    far = ref.mx_shift(v, err, fmt)
    for _ in range(20):
        moved = v + err * (2 * torch.rand(v.shape, generator=g, dtype=ref.F64) - 1)
        assert bool(((ref.mx(moved, fmt) - q).abs() <= far).all())
