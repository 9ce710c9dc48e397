"""Operands of the products that are no matrices at all are refused like other
wrong shapes (no GPU)."""
import pytest

import norm_activation_fp8_gb300 as vg


@pytest.mark.parametrize("shape", [(), (64,), (1, 3, 64)])
def test_operands_of_other_ranks_are_refused(shape):
    import torch
    u8, f8 = torch.uint8, torch.float8_e4m3fn
    a4, s4 = torch.zeros(shape, dtype=u8), torch.zeros((3, 8), dtype=f8)
    w4, sw4, one = torch.zeros((128, 64), dtype=u8), torch.zeros((128, 8), dtype=f8), torch.ones(1)
    a8, s8 = torch.zeros(shape, dtype=f8), torch.zeros((3, 1))
    w8, sw8 = torch.zeros((256, 128), dtype=f8), torch.zeros((2, 1))
    good4, good8 = torch.zeros((3, 64), dtype=u8), torch.zeros((3, 128), dtype=f8)
    with pytest.raises(ValueError, match="2-D"):
        vg.nvfp4_gemm(a4, s4, w4, sw4, one)
    with pytest.raises(ValueError, match="2-D"):
        vg.nvfp4_gemm_silu_mul_nvfp4(a4, s4, w4, sw4, one, one)
    with pytest.raises(ValueError, match="2-D"):
        vg.nvfp4_gemm(good4, s4, a4, sw4, one)
    with pytest.raises(ValueError, match="2-D"):
        vg.nvfp4_dequantize(a4, s4, one)
    with pytest.raises(ValueError, match="2-D"):
        vg.fp8_block_gemm(a8, s8, w8, sw8)
    with pytest.raises(ValueError, match="2-D"):
        vg.fp8_block_gemm_silu_mul_fp8(a8, s8, w8, sw8)
    with pytest.raises(ValueError, match="2-D"):
        vg.fp8_block_gemm(good8, s8, a8, sw8)
