"""The NVFP4 quantiser and products on the host (no GPU): every bad argument is
refused before any CUDA call, so fake pointers are safe; and the binding's own
checks."""
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
    for k in ("out", "a", "sa", "w", "sw"):
        assert gemm(lib, **{k: A + 8}) == ALIGN, k
    for k in ("q4", "sf", "a", "sa", "w", "sw"):
        assert gated(lib, **{k: A + 8}) == ALIGN, k
    assert gemm(lib, alpha=A + 2) == ALIGN
    for k in ("alpha", "gs"):
        assert gated(lib, **{k: A + 2}) == ALIGN, k
    assert gemm(lib, out=None, a=None, sa=None, w=None, sw=None, alpha=None, T=0) == OK
    assert gated(lib, q4=None, sf=None, a=None, sa=None, w=None, sw=None, alpha=None, gs=None, T=0) == OK


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
