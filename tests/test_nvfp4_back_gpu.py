"""NVFP4 back to bf16, bit for bit: bf16(value * fp32(decode(sf) / gs)) with IEEE
divisions and products on the host, for every code under every scale code."""
import numpy as np
import pytest

import norm_activation_fp8_gb300 as vg
from test_nvfp4_back_host import quotient
from test_nvfp4_gemm_gpu import LEVELS

pytestmark = pytest.mark.gpu

F = np.float32


def scale_values():
    import torch
    return torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()


def expected(r):
    """bf16 bits [n, 127 * 16] of all codes times the quotients r [n, 127]."""
    import torch
    v = torch.tensor(LEVELS + tuple(-x for x in LEVELS))
    return (v * torch.from_numpy(r)[..., None]).to(torch.bfloat16).flatten(1)


def check(scales):
    """A row of all codes under all scale codes, for each tensor scale."""
    import torch
    row = torch.arange(8, device="cuda", dtype=torch.uint8)
    q4 = (2 * row | (2 * row + 1) << 4).repeat(127).view(1, -1)
    sf = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).view(1, -1)
    gs = torch.from_numpy(scales).cuda()
    out = torch.empty((len(scales), 127 * 16), dtype=torch.bfloat16, device="cuda")
    for i in range(len(scales)):
        vg.vg_nvfp4_dequantize(out[i:i + 1], q4, sf, gs[i:i + 1])
    with np.errstate(over="ignore", under="ignore"):
        want = expected(scale_values().numpy() / scales[:, None])
    got = out.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    ok = want.isnan() | (got.view(torch.int16) == want.view(torch.int16))
    assert bool(ok.all()), scales[np.flatnonzero(~ok.all(1).numpy())[:5]]
    assert vg.vg_device_status() == 0


def test_quotients_next_to_bf16_midpoints():
    """Tensor scales that put a quotient on a midpoint of two bf16 numbers or a
    rounding beside it: there its last bit decides the result."""
    import torch
    m = 1 + (2 * np.arange(128) + 1) / 256
    near = np.unique(np.concatenate([(d / m).astype(F).view(np.int32) + k
                                     for d in 1 + np.arange(8) / 8 for k in range(-2, 3)]))
    scales = near.view(F) * F(64)
    d = np.broadcast_to(scale_values().numpy(), (len(scales), 127))
    r, product = quotient(d, np.broadcast_to(scales[:, None], d.shape))
    off = expected(r).view(torch.int16) != expected(product).view(torch.int16)
    assert int(off.any(1).sum()) > 100  # a quotient off by its last bit is seen
    check(scales)


def test_far_and_near_tensor_scales():
    """Both sides of where the division itself is used, the ends of fp32 (quotients
    that are subnormal, zero or infinite), and scales in between."""
    edge = [2.0 ** -149, 2.0 ** -127, 2.0 ** -126, 2.0 ** -119, 2.0 ** -118, 1.7 * 2.0 ** -110,
            2.0 ** -100, 2.0 ** 100, 1.3 * 2.0 ** 110, 2.0 ** 126, float(np.finfo(F).max)]
    edge = np.array(edge, F)
    edge = np.concatenate([edge, np.nextafter(edge, F(1)), np.nextafter(edge[6:8], F([0, np.inf]))])
    rng = np.random.default_rng(1)
    spread = np.exp2(rng.uniform(-125, 127, 2000)).astype(F)
    check(np.concatenate([edge, spread]))
