"""The NVFP4 product and the gated projection against fp64, at the sizes where a
tile, a split or a tail can go wrong.

Tolerances, derived (u = 2^-24, S = the sum of |products|, scaled, alpha in):
  c    a product of two codes and two scales is exact in fp32 (12 significant
       bits); the 64 of one instruction are summed by fp32 additions in any
       order, each off by at most 2u of the running magnitude (2u, not u: the
       tensor cores may truncate), the K / 64 sums and alpha add K / 64 + 2
       roundings.  |dc| <= E = 2u (K / 64 + 66) S.
  out  bf16(c): E + 2^-8 (|c| + E)
  y    |d silu| <= 1.1 |dg| (its largest slope), so |dy| <= Ey = 1.1 Eg (|u| +
       Eu) + |silu(g)| Eu + 2^-21 |y|
  sf   between the codes of gs (amax -+ max Ey) / 6, 2^-21 of it
  q    between the codes of gs (y -+ Ey) / sf (its own sf), 2^-21 of it
Small integer codes under power-of-two scales make every sum exact: there the
result has to be the correctly rounded one, bit for bit."""
import numpy as np
import pytest

import norm_activation_fp8_gb300 as vg

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def levels():
    import torch
    return torch.tensor(LEVELS, dtype=torch.float64, device="cuda")


def values(q4):
    """fp64 values of packed codes."""
    import torch
    q = q4.long()
    c = torch.stack([q & 15, q >> 4], -1).flatten(1)
    v = levels()[c & 7]
    return torch.where(c >= 8, -v, v)


def packed(code):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()


def scaled(q4, sf):
    return values(q4) * sf.double().repeat_interleave(16, 1)


def nearest(x, grid):
    """The grid's value nearest to x >= 0 (ascending grid of codes), ties to the even code."""
    import torch
    mid = (grid[1:] + grid[:-1]) / 2
    at = torch.searchsorted(mid, x.contiguous())
    here = at.clamp_max(len(grid) - 2)
    return grid[at + ((x == mid[here]) & (here % 2 == 1)).long()]


def e4m3_grid():
    import torch
    return torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()


def operand(rows, K, seed, exact=False):
    """Codes [rows, K / 2] and scales [rows, K / 16] of a random operand."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    if exact:  # values 0, +-1, +-2 (codes 0, 2, 4), scales 1, 2: |sum| <= 16 K <= 2^19
        c = torch.randint(0, 3, (rows, K), generator=g, device="cuda") * 2
        sf = 2.0 ** torch.randint(0, 2, (rows, K // 16), generator=g, device="cuda").float()
    else:  # every code, every kind of scale: subnormal, zero, largest
        c = torch.randint(0, 8, (rows, K), generator=g, device="cuda")
        bits = torch.randint(0, 127, (rows, K // 16), generator=g, device="cuda").to(torch.uint8)
        sf = bits.view(torch.float8_e4m3fn)
    c = c | torch.randint(0, 2, (rows, K), generator=g, device="cuda") << 3
    return packed(c.to(torch.uint8)), sf.to(torch.float8_e4m3fn)


def one(v):
    import torch
    return torch.full((1,), v, device="cuda")


def guarded(shape, dtype):
    """A tensor between bands that must stay as they are."""
    import torch
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((n + 512,), 0xAB, dtype=torch.uint8, device="cuda")
    return buf, buf[256:256 + n].view(dtype).view(shape)


def intact(buf):
    return bool((buf[:256] == 0xAB).all()) and bool((buf[-256:] == 0xAB).all())


def product_error(A, W, K):
    return 2 * U * (K // 64 + 66) * (A.abs() @ W.abs().t())


PLAIN = [  # T, N, K
    (1, 128, 64), (1, 8, 128), (1, 6144, 4096), (2, 136, 256), (3, 1000, 384), (8, 4096, 14336),
    (15, 512, 1024), (16, 520, 704), (17, 2048, 512), (31, 384, 960), (33, 1024, 2048), (64, 4096, 1152),
    (65, 640, 256), (100, 264, 32768), (127, 136, 576), (128, 256, 128), (129, 384, 1024),
    (200, 4096, 4096), (256, 4096, 2048), (257, 248, 448), (300, 6144, 1024), (513, 1032, 512),
    (1000, 2056, 832), (2049, 4096, 640), (4100, 264, 256), (512, 1024, 8192),
    (130, 10248, 192), (700, 9736, 448), (4100, 2056, 64), (385, 8192, 16384), (2304, 5120, 1088),
]


@pytest.mark.parametrize("T,N,K", PLAIN)
def test_gemm(T, N, K):
    import torch
    a, sa = operand(T, K, T + N + K)
    w, sw = operand(N, K, T + N + K + 1)
    buf, out = guarded((T, N), torch.bfloat16)
    vg.vg_nvfp4_gemm(out, a, sa, w, sw, one(0.37))
    A, W = scaled(a, sa), scaled(w, sw) * float(np.float32(0.37))
    c, e = A @ W.t(), product_error(A, W, K)
    assert bool(((out.double() - c).abs() <= e + 2.0 ** -8 * (c.abs() + e)).all())
    assert intact(buf)
    # exact sums: the correctly rounded result
    a, sa = operand(T, K, T, exact=True)
    w, sw = operand(N, K, N, exact=True)
    vg.vg_nvfp4_gemm(out, a, sa, w, sw, one(0.25))
    assert torch.equal(out, (scaled(a, sa) @ (0.25 * scaled(w, sw)).t()).to(torch.bfloat16))
    assert intact(buf)
    assert vg.vg_device_status() == 0


GATED = [  # T, I, K
    (1, 64, 64), (1, 14336, 512), (2, 256, 384), (7, 384, 4096), (15, 128, 256), (16, 512, 1024),
    (17, 192, 128), (33, 1024, 704), (57, 2048, 2048), (64, 384, 32768), (65, 320, 512), (127, 640, 256),
    (128, 128, 384), (129, 1152, 576), (200, 14336, 256), (256, 2048, 1024), (300, 64, 896),
    (513, 1024, 512), (1000, 960, 640), (2049, 2048, 256), (4100, 192, 128),
    (300, 14400, 256), (515, 4160, 1088), (4100, 1344, 64), (257, 8192, 2048),
]


def check_gated(q4, sf, g, u, eg, eu, gs):
    import torch
    T, I = g.shape
    silu = g * torch.sigmoid(g)
    y = silu * u
    ey = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + 2.0 ** -21 * y.abs()
    block = lambda x: x.view(T, I // 16, 16)  # noqa: E731
    amax, ea = block(y.abs()).amax(-1), block(ey).amax(-1)
    grid, near = e4m3_grid(), 2.0 ** -21
    lo = nearest(((amax - ea).clamp_min(0) * gs / 6 * (1 - near)), grid)
    hi = nearest((amax + ea) * gs / 6 * (1 + near), grid)
    s = sf.double()
    assert bool(((s >= lo) & (s <= hi)).all())
    got, s = block(values(q4)), s[..., None]
    v, ev = block(y) * gs / s, block(ey) * gs / s
    signed = lambda x: torch.sign(x) * nearest(x.abs(), levels())  # noqa: E731
    ok = (got >= signed(v - ev - near * v.abs())) & (got <= signed(v + ev + near * v.abs()))
    assert bool(torch.where(s > 0, ok, got == 0).all())


@pytest.mark.parametrize("T,I,K", GATED)
def test_gated(T, I, K):
    import torch
    a, sa = operand(T, K, T + I + K)
    w, sw = operand(2 * I, K, T + I + K + 1)
    alpha = float(np.float32(2e-5 / K ** 0.5))
    qbuf, q4 = guarded((T, I // 2), torch.uint8)
    sbuf, sf = guarded((T, I // 16), torch.float8_e4m3fn)
    A, W = scaled(a, sa), scaled(w, sw) * alpha
    c, e = A @ W.t(), product_error(A, W, K)
    for gs in (100.0, 1e4):
        vg.vg_nvfp4_gemm_silu_mul_nvfp4(q4, sf, a, sa, w, sw, one(alpha), one(gs))
        check_gated(q4, sf, c[:, :I], c[:, I:], e[:, :I], e[:, I:], gs)
        assert intact(qbuf) and intact(sbuf)
    assert vg.vg_device_status() == 0
