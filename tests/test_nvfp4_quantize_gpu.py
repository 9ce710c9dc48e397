"""Rows of bf16 to NVFP4 and back, against fp64.

Quantisation is exact: gs x has 32 significant bits, so fp64 holds it, and a
quotient that is no tie is at least 2^-33 of itself from one: fp64 decides every
code.  Reading back rounds to fp32 twice (2^-24 each) and to bf16 once."""
import pytest

import norm_activation_fp8_gb300 as vg
from test_nvfp4_gemm_gpu import e4m3_grid, guarded, intact, levels, nearest, one, operand, values

pytestmark = pytest.mark.gpu

GS = (1.0, 168.0, 123.456)


def check(x, q4, sf, gs):
    """x finite."""
    import torch
    T, n = x.shape
    gs = one(gs).double()
    b = x.double().reshape(T, n // 16, 16)
    want = nearest(b.abs().amax(-1) * gs / 6, e4m3_grid())
    assert torch.equal(sf.double(), want)
    v = torch.where(want[..., None] > 0, b * gs / want[..., None].clamp_min(2.0 ** -9), 0.0)
    got = values(q4).view_as(b)
    assert torch.equal(got.abs(), nearest(v.abs(), levels()))
    sign = (torch.stack([q4 & 8, q4 >> 4 & 8], -1).flatten(1) != 0).view_as(b)
    assert torch.equal(sign, (want[..., None] > 0) & torch.signbit(b))


def run(x, gs):
    import torch
    T, n = x.shape
    qbuf, q4 = guarded((T, n // 2), torch.uint8)
    sbuf, sf = guarded((T, n // 16), torch.float8_e4m3fn)
    vg.vg_nvfp4_quantize(q4, sf, x, one(gs))
    check(x, q4, sf, gs)
    assert intact(qbuf) and intact(sbuf)
    return q4, sf


def randn(T, n, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, n), generator=g, device="cuda")
    return (x * (1 + 100 * (torch.rand((T, n), generator=g, device="cuda") < 0.001))).bfloat16()


@pytest.mark.parametrize("T,n", [(1, 16), (1, 8192), (3, 48), (7, 8208), (64, 4096), (333, 1040),
                                 (1, 32768), (1025, 16), (4099, 2048), (2048, 14336)])
@pytest.mark.parametrize("gs", GS)
def test_shapes(T, n, gs):
    run(randn(T, n, T + n), gs)
    assert vg.vg_device_status() == 0


@pytest.mark.parametrize("T,n,pitch,off", [(1, 64, 128, 8), (5, 48, 64, 16), (300, 4096, 6144, 1024),
                                           (1000, 16, 24, 0), (129, 2064, 2080, 8)])
def test_strided_rows(T, n, pitch, off):
    base = randn(T, pitch, T + n)
    run(base[:, off:off + n], 168.0)


@pytest.mark.parametrize("gs", [1.0, 6.0, 0.75, 168.0, 3.0 * 2.0 ** -20, 2.0 ** 100, 2.0 ** -100])
def test_every_finite_bf16_value(gs):
    """All finite bf16 patterns, in blocks of their own and beside a larger one:
    with scales like these many quotients are ties."""
    import torch
    i = torch.arange(-32768, 32768, device="cuda")
    p = i.to(torch.int16).view(torch.bfloat16)
    p = p[torch.isfinite(p.float())]
    x = torch.zeros((len(p), 16), dtype=torch.bfloat16, device="cuda")
    x[:, 3] = p
    run(x, gs)
    x[:, 11] = 6 * torch.roll(p, 129)
    x = x[torch.isfinite(x.float()).all(1)]
    run(x.contiguous(), gs)


def test_ties():
    """Values on midpoints of either grid, and one bf16 step beside them."""
    import torch
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    x = torch.zeros((7 * 3 * 15, 16), device="cuda")
    x[:, 0] = 6.0  # the block's scale is its power of two
    i = torch.arange(len(x), device="cuda")
    x[:, 5] = mids[i % 7] * (1 + (i // 7 % 3 - 1) * 2.0 ** -7)
    x[:, 6] = -x[:, 5]
    run((x * 2.0 ** (i // 21 - 8.0)[:, None]).bfloat16(), 1.0)
    grid = e4m3_grid().float()
    m = ((grid[1:] + grid[:-1]) / 2 * 6)[:, None]  # amax / 6 on a midpoint of E4M3
    for step in (-1, 0, 1):
        y = torch.zeros((126, 16), device="cuda")
        y[:, 9:10] = m * (1 + step * 2.0 ** -7)
        run(y.bfloat16(), 1.0)


def test_not_finite():
    import torch
    x = randn(6, 32, 1)
    x[0, 3], x[1, 3], x[2, 3] = float("nan"), float("inf"), float("-inf")
    x[3, :16] = float("nan")
    x[4, 3], x[4, 4] = float("inf"), float("nan")
    q4, sf = vg.nvfp4_quantize(x, one(168.0))
    keep = x[5:]
    check(keep, q4[5:], sf[5:], 168.0)
    check(x[:3, 16:], q4[:3, 8:], sf[:3, 1:], 168.0)
    v, s = values(q4), sf.float()
    clean = x[0:1].clone()
    clean[0, 3] = 0
    assert float(s[0, 0]) == float(vg.nvfp4_quantize(clean, one(168.0))[1].float()[0, 0])
    assert abs(float(v[0, 3])) == 6
    assert float(s[1, 0]) == 448 and float(v[1, 3]) == 6 and float(v[2, 3]) == -6
    assert float(s[3, 0]) == 0 and bool((q4[3, :8] == 0).all())
    assert float(s[4, 0]) == 448 and float(v[4, 3]) == 6 and abs(float(v[4, 4])) == 6


@pytest.mark.parametrize("T,n", [(1, 16), (1, 8192), (3, 48), (333, 1040), (2048, 14336), (5, 32768)])
@pytest.mark.parametrize("gs", GS)
def test_back(T, n, gs):
    import torch
    q4, sf = operand(T, n, T + n)
    buf, out = guarded((T, n), torch.bfloat16)
    vg.vg_nvfp4_dequantize(out, q4, sf, one(gs))
    want = values(q4) * (sf.double() / one(gs).double()).repeat_interleave(16, 1)
    assert bool(((out.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -22) * want.abs()).all())
    assert intact(buf)
    # what was read back quantises to the same tensor where its block's largest code is 6
    x = vg.nvfp4_dequantize(q4, sf, one(1.0))
    r4, rf = vg.nvfp4_quantize(x, one(1.0))
    full = (values(q4).abs().view(T, n // 16, 16).amax(-1) == 6) & (sf.float() > 0)
    assert torch.equal(rf.float()[full], sf.float()[full])
    same = (values(r4) == values(q4)).view(T, n // 16, 16).all(-1)
    assert bool(same[full].all())


def test_back_nan_scale():
    import torch
    q4, sf = operand(2, 32, 1)
    sf.view(torch.uint8)[0, 1] = 0x7F
    out = vg.nvfp4_dequantize(q4, sf, one(2.0))
    assert bool(torch.isnan(out[0, 16:]).all()) and bool(torch.isfinite(out[0, :16]).all())
    assert bool(torch.isfinite(out[1]).all())


def test_no_tokens():
    import torch
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    q4, sf = vg.nvfp4_quantize(x, one(1.0))
    assert q4.shape == (0, 32) and sf.shape == (0, 4)
    assert vg.nvfp4_dequantize(q4, sf, one(1.0)).shape == (0, 64)


@pytest.mark.parametrize("pitch", [32768, 32776])
def test_offsets_past_32_bits(pitch):
    """More than 2^31 elements, rows one after the other and apart; rows sampled."""
    import torch
    T, n = 70001, 32768
    base = randn(997, n, 3)
    x = torch.empty((T, pitch), dtype=torch.bfloat16, device="cuda")[:, :n]
    for t in range(0, T, 997):
        x[t:t + 997] = base[:min(997, T - t)]
    q4, sf = vg.nvfp4_quantize(x, one(168.0))
    back = vg.nvfp4_dequantize(q4, sf, one(168.0))
    rows = torch.tensor([0, 65535, 65536, 65537, 69999, 70000], device="cuda")
    few = sf.view(torch.uint8)[rows].view(sf.dtype)
    check(x[rows], q4[rows], few, 168.0)
    assert torch.equal(back[rows], vg.nvfp4_dequantize(q4[rows], few, one(168.0)))


def test_unaligned_slices_and_refusals():
    """Rows that start at 16 but not at 32 bytes; what the binding refuses."""
    import torch
    x = randn(40, 2048, 1)
    run(x.view(-1)[8:8 + 39 * 2048].view(39, 2048), 168.0)
    gs = one(1.0)
    with pytest.raises(ValueError, match="contiguous rows"):
        vg.nvfp4_quantize(x.t(), gs)
    with pytest.raises(TypeError, match="x"):
        vg.nvfp4_quantize(x.float(), gs)
    with pytest.raises(ValueError, match="blocks"):
        vg.nvfp4_quantize(x[:, :24], gs)
    with pytest.raises(vg.VgError, match="MISALIGNED"):
        vg.nvfp4_quantize(x[:, 4:20], gs)
    with pytest.raises(vg.VgError, match="BAD_SHAPE"):
        vg.nvfp4_quantize(x[:1, :16].expand(5, 16), gs)
    with pytest.raises(TypeError, match="global_scale"):
        vg.nvfp4_quantize(x, gs.double())
    with pytest.raises(ValueError, match="global_scale"):
        vg.nvfp4_quantize(x, gs.cpu())
    with pytest.raises(ValueError, match="global_scale"):
        vg.nvfp4_quantize(x, torch.ones(2, device="cuda"))
    q4, sf = vg.nvfp4_quantize(x, gs)
    with pytest.raises(ValueError, match="both or neither"):
        vg.vg_nvfp4_quantize(q4, None, x, gs)
    with pytest.raises(ValueError, match="q4"):
        vg.vg_nvfp4_quantize(q4[:, :512].contiguous(), sf, x, gs)
    with pytest.raises(ValueError, match="block_scale"):
        vg.vg_nvfp4_quantize(q4, sf[:5], x, gs)
    with pytest.raises(TypeError, match="q4"):
        vg.nvfp4_dequantize(q4.view(torch.int8), sf, gs)
    with pytest.raises(ValueError, match="contiguous"):
        vg.nvfp4_dequantize(q4[:, ::2][:, :8], sf[:, :1], gs)
    with pytest.raises(ValueError, match="out"):
        vg.vg_nvfp4_dequantize(torch.empty((40, 16), dtype=torch.bfloat16, device="cuda"), q4, sf, gs)
    with pytest.raises(TypeError, match="out"):
        vg.vg_nvfp4_dequantize(torch.empty((40, 2048), device="cuda"), q4, sf, gs)
