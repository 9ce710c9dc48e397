"""The sizes of test_nvfp4_forms_gpu.py take every plan on 152 SMs (no GPU)."""
import pytest

from norm_activation_fp8_gb300 import build
from test_nvfp4_forms_gpu import GATED, PLAIN
from test_nvfp4_gemm_host import plan, reachable


@pytest.mark.parametrize("gated", [False, True])
def test_sizes_take_every_form(gated):
    build.build()
    sizes = GATED if gated else PLAIN
    for whole in (False, True):  # K a multiple of 256 or not
        taken = {plan(*x, gated, 152) for x in sizes if (x[2] % 256 == 0) == whole}
        assert taken >= reachable(gated), reachable(gated) - taken
