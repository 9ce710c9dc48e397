"""The NVFP4 quantiser and products on the host (no GPU): every bad argument is
refused before any CUDA call, so fake pointers are safe; and the binding's own
checks."""
import ctypes
import random

import pytest

import norm_activation_fp8_gb300 as vg
from norm_activation_fp8_gb300 import build

OK, NULL, SHAPE, ALIGN = 0, 1, 2, 3
A = 0x10000  # a 16-byte aligned fake device address (never dereferenced)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return vg.load()


def quantize(lib, q4=A, sf=A, x=A, stride=512, gs=A, T=4, n=512):
    return lib.vg_nvfp4_quantize(q4, sf, x, stride, gs, T, n, None)


def dequantize(lib, out=A, q4=A, sf=A, gs=A, T=4, n=512):
    return lib.vg_nvfp4_dequantize(out, q4, sf, gs, T, n, None)


def gemm(lib, out=A, a=A, sa=A, w=A, sw=A, alpha=A, T=4, N=256, K=512):
    return lib.vg_nvfp4_gemm(out, a, sa, w, sw, alpha, T, N, K, None)


def gated(lib, q4=A, sf=A, a=A, sa=A, w=A, sw=A, alpha=A, gs=A, T=4, I=256, K=512):
    return lib.vg_nvfp4_gemm_silu_mul_nvfp4(q4, sf, a, sa, w, sw, alpha, gs, T, I, K, None)


def test_quantize_refusals(lib):
    for T in (-1, 2 ** 31):
        assert quantize(lib, T=T) == SHAPE and dequantize(lib, T=T) == SHAPE
    for n in (0, 8, 24, -16, 32784):
        assert quantize(lib, n=n, stride=32784) == SHAPE and dequantize(lib, n=n) == SHAPE, n
    assert quantize(lib, T=2 ** 31 - 1, n=32768, stride=32768) == SHAPE  # more CTAs than a grid has
    assert dequantize(lib, T=2 ** 31 - 1, n=32768) == SHAPE
    for stride in (504, 516, -512):
        assert quantize(lib, stride=stride) == SHAPE, stride
    for k in ("q4", "sf", "x", "gs"):
        assert quantize(lib, **{k: None}) == NULL, k
    for k in ("out", "q4", "sf", "gs"):
        assert dequantize(lib, **{k: None}) == NULL, k
    for k in ("q4", "x"):
        assert quantize(lib, **{k: A + 8}) == ALIGN, k
    for k in ("q4", "out"):
        assert dequantize(lib, **{k: A + 8}) == ALIGN, k
    assert quantize(lib, gs=A + 2) == ALIGN and dequantize(lib, gs=A + 2) == ALIGN
    assert quantize(lib, q4=None, sf=None, x=None, gs=None, T=0) == OK
    assert dequantize(lib, out=None, q4=None, sf=None, gs=None, T=0) == OK


def test_product_refusals(lib):
    for T in (-1, 2 ** 24 + 1, 2 ** 31):
        assert gemm(lib, T=T) == SHAPE and gated(lib, T=T) == SHAPE, T
    for n in (0, -8, 4, 12, 2 ** 20 + 8):
        assert gemm(lib, N=n) == SHAPE, n
    for n in (0, -64, 32, 96, 32768 + 64):
        assert gated(lib, I=n) == SHAPE, n
    for k in (0, -64, 32, 96, 4128, 32768 + 64):
        assert gemm(lib, K=k) == SHAPE and gated(lib, K=k) == SHAPE, k
    for k in ("out", "a", "sa", "w", "sw", "alpha"):
        assert gemm(lib, **{k: None}) == NULL, k
    for k in ("q4", "sf", "a", "sa", "w", "sw", "alpha", "gs"):
        assert gated(lib, **{k: None}) == NULL, k
    for k in ("out", "a", "w"):
        assert gemm(lib, **{k: A + 8}) == ALIGN, k
    for k in ("q4", "a", "w"):
        assert gated(lib, **{k: A + 8}) == ALIGN, k
    for k in ("sa", "sw", "alpha"):
        assert gemm(lib, **{k: A + 2}) == ALIGN, k
    for k in ("sf", "sa", "sw", "alpha", "gs"):
        assert gated(lib, **{k: A + 2}) == ALIGN, k
    assert gemm(lib, out=None, a=None, sa=None, w=None, sw=None, alpha=None, T=0) == OK
    assert gated(lib, q4=None, sf=None, a=None, sa=None, w=None, sw=None, alpha=None, gs=None, T=0) == OK


class GemmPlan(ctypes.Structure):
    _fields_ = [("tn", ctypes.c_int), ("splits", ctypes.c_int)]


def plan(T, N, K, gated, sms):
    """The library's own plan: (tokens a tile of the stream kernel or 0 for the
    tile kernel, ways that K is split)."""
    f = vg.load()._ZN2vg13plan_fp4_gemmElllbi
    f.restype, f.argtypes = GemmPlan, [ctypes.c_int64] * 3 + [ctypes.c_bool, ctypes.c_int]
    p = f(T, N, K, gated, sms)
    return p.tn, p.splits


def _sizes(gated, n, seed):
    r = random.Random(seed)
    unit = 64 if gated else 8
    for _ in range(n):
        yield (max(1, int(2 ** (13 * r.random()))), unit * int(2 ** ((9 if gated else 13) * r.random())),
               64 * int(2 ** (9 * r.random())))


def reachable(gated):
    return {plan(*x, gated, 152) for x in _sizes(gated, 20000, 1)}


@pytest.mark.parametrize("gated", [False, True])
def test_every_plan_can_be_launched(lib, gated):
    """A split never exceeds the stages of K or its cluster the eight CTAs that
    may form one, the grid stays within its limits, and few tokens take one
    token tile."""
    sizes = list(_sizes(gated, 5000, 2)) + [(2 ** 24, 2 ** 15, 64), (2 ** 24, 64, 32768), (1, 64, 64)]
    if not gated:
        sizes += [(1, 2 ** 20, 32768), (2 ** 24, 8, 64), (128, 2 ** 20, 64), (1, 8, 32768), (2 ** 24, 2 ** 20, 64)]
    for sms in (152, 148, 132, 16, 2, 1):
        for T, N, K in sizes:
            tn, splits = plan(T, N, K, gated, sms)
            assert 1 <= splits <= (K + 255) // 256
            if tn == 0:
                assert splits <= 4
                tiles = (T + 255) // 256 * ((N + 127) // 128 if gated else (N + 255) // 256)
                assert splits == 1 or 2 * splits * tiles < 2 ** 31
                assert tiles < 2 ** 32
            else:
                assert tn in (16, 32, 64, 128) and splits in (1, 2, 4, 8)
                assert T > 64 or tn >= T
                assert (T + tn - 1) // tn * (N // 64 if gated else (N + 127) // 128) * splits < 2 ** 31
    assert {tn for tn, _ in reachable(gated)} == {0, 16, 32, 64, 128}


def test_binding_refuses_before_the_library():
    """What the binding can tell from the tensors alone; a CPU tensor comes last."""
    import torch
    u8, f8 = torch.uint8, torch.float8_e4m3fn
    a, sa = torch.zeros((3, 64), dtype=u8), torch.zeros((3, 8), dtype=f8)
    w, sw = torch.zeros((128, 64), dtype=u8), torch.zeros((128, 8), dtype=f8)
    one, x = torch.ones(1), torch.zeros((3, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        vg.nvfp4_gemm(a, sa, w, sw, one)
    with pytest.raises(ValueError, match="a_scale"):
        vg.nvfp4_gemm(a, sa[:, :4], w, sw, one)
    with pytest.raises(ValueError, match="blocks"):
        vg.nvfp4_gemm(a[:, :60], sa, w, sw, one)
    with pytest.raises(ValueError, match="2-D"):
        vg.nvfp4_gemm(a[0], sa, w, sw, one)
    with pytest.raises(ValueError, match="CUDA"):
        vg.nvfp4_gemm_silu_mul_nvfp4(a, sa, w, sw, one, one)
    with pytest.raises(ValueError, match="CUDA"):
        vg.nvfp4_dequantize(a, sa, one)
    with pytest.raises(ValueError, match="CUDA"):
        vg.nvfp4_quantize(x, one)
    with pytest.raises(TypeError, match="x"):
        vg.nvfp4_quantize(x.float(), one)
