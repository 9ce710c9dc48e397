"""The NVFP4 quantiser's forms on either side of the size where a thread takes
four blocks instead of one: rows one after the other and apart, 32-byte aligned
and not, with and without the debug build's bounds checks."""
import numpy as np
import pytest

import norm_activation_fp8_gb300 as vg
from norm_activation_fp8_gb300 import build
from test_nvfp4_gemm_gpu import one
from test_nvfp4_layer_gpu import _with
from test_nvfp4_quantize_gpu import check, randn, run

pytestmark = pytest.mark.gpu

# 2^22 chunks of 8 columns are four a thread: 4087 rows of 8208 are below, 4099 above
FORMS = [(T, pitch, off) for T in (4087, 4099) for pitch, off in ((8208, 0), (8208, 8), (8240, 16), (8216, 8))]


def rows(T, pitch, off):
    """[T, 8208] out of rows of `pitch`, `off` elements on (8: 16 bytes)."""
    flat = randn(T + 1, pitch, T + off).view(-1)
    return flat[off:off + T * pitch].view(T, pitch)[:, :8208]


@pytest.mark.parametrize("T,pitch,off", FORMS)
def test_forms(T, pitch, off):
    run(rows(T, pitch, off), 168.0)
    assert vg.vg_device_status() == 0


@pytest.mark.parametrize("T,pitch,off", FORMS)
def test_debug_builds(T, pitch, off, monkeypatch):
    import torch
    x, gs = rows(T, pitch, off), one(168.0)

    def quantised():
        q4, sf = vg.nvfp4_quantize(x, gs)
        return {"q": q4.cpu().numpy(), "scale": sf.view(torch.uint8).cpu().numpy()}

    want, _ = _with(vg.load(), quantised, monkeypatch)
    got, st = _with(vg.load(build.build_debug()), quantised, monkeypatch)
    assert st == 0 and all(np.array_equal(got[k], v) for k, v in want.items())
    got, st = _with(vg.load(build.build_debug(shrunk=True)), quantised, monkeypatch)
    assert st == vg.DEVICE_OUT_OF_BOUNDS
    assert all(np.array_equal(got[k][:-1], v[:-1]) for k, v in want.items())


def test_many_rows_with_infinities_and_nans():
    """Four blocks a thread: what is not finite stays in its own block."""
    import torch
    x = rows(4099, 8208, 0).clone()
    x[::3, 16], x[::5, 40], x[::7, 200] = float("inf"), float("nan"), float("-inf")
    q4, sf = vg.nvfp4_quantize(x, one(168.0))
    s = sf.float()
    assert bool((s[::3, 1] == 448).all()) and bool((s[::7, 12] == 448).all())
    clean = torch.where(x.isfinite(), x, 0)
    r4, rf = vg.nvfp4_quantize(clean, one(168.0))
    check(clean, r4, rf, 168.0)
    keep = x.isfinite().view(4099, -1, 16).all(-1)
    assert torch.equal(sf.view(torch.uint8)[keep], rf.view(torch.uint8)[keep])
    assert torch.equal(q4.view(4099, -1, 8)[keep], r4.view(4099, -1, 8)[keep])
