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
    # the plans that the sizes above do not take
    (1677, 936, 4928), (1090, 624, 12672), (460, 1432, 13440), (1, 24, 14080), (20, 16, 192),
    (18, 16, 3392), (24, 16, 8704), (140, 15832, 256), (75, 1456, 13824),
]


def test_sizes_take_every_plan():
    """On 152 SMs the sizes of these tests run every kernel with every split that
    some size takes."""
    import test_nvfp4_gemm_host as host
    for sizes, gated in ((PLAIN, False), (GATED, True)):
        assert {host.plan(*x, gated, 152) for x in sizes} >= host.reachable(gated)


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
    (604, 960, 6592), (985, 448, 10304), (337, 704, 18176), (1, 64, 24704), (31, 64, 704),
    (32, 64, 2624), (25, 128, 5504), (59, 128, 3584), (3205, 64, 4096), (69, 768, 19264),
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


@pytest.mark.parametrize("T,N,K", [
    (1, 8, 64), (1, 6144, 4096), (20, 96, 128), (31, 384, 960), (50, 2056, 512), (70, 3800, 6912),
    (196, 3704, 6912), (1000, 2056, 896), (2049, 4096, 640)])
def test_sums_are_held_in_fp32(T, N, K):
    """Every K of 64 has +96^2 and -96^2, in it or with the one beside it, and
    products that are multiples of 2^-8: their sum has to come out exact.  Every
    partial sum, in whatever order, is a multiple of 2^-8 below 2 * 96^2 + 2^-4 K
    < 2^16, so it has at most 24 bits; an accumulator of fewer, or products
    aligned to fewer, loses some."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T + N)
    f8 = torch.float8_e4m3fn
    for apart in (False, True):
        # values 0, +-0.5, +-1 (codes 0 to 2) under scales of 2^-3
        ca = torch.randint(0, 3, (T, K), generator=g, device="cuda") | torch.randint(0, 2, (T, K), generator=g, device="cuda") << 3
        cw = torch.randint(0, 3, (N, K), generator=g, device="cuda") | torch.randint(0, 2, (N, K), generator=g, device="cuda") << 3
        sa, sw = torch.full((T, K // 16), 0.125, device="cuda"), torch.full((N, K // 16), 0.125, device="cuda")
        st = torch.randint(0, 2, (T, 1), generator=g, device="cuda") * 8
        sn = torch.randint(0, 2, (N, 1), generator=g, device="cuda") * 8
        for k in range(0, K, 64 if not apart else 128):
            # two blocks of 16 that hold one code 6 under a scale of 16 each
            first, second = k, k + 48 if not apart else min(k + 64, K - 16)
            if first == second:
                continue
            for b in (first, second):
                ca[:, b:b + 16], cw[:, b:b + 16] = 0, 0
                sa[:, b // 16], sw[:, b // 16] = 16.0, 16.0
                ca[:, [b + 5]], cw[:, [b + 5]] = 7 | st, 7 | (sn if b == first else sn ^ 8)
        a, w = packed(ca.to(torch.uint8)), packed(cw.to(torch.uint8))
        want = scaled(a, sa) @ scaled(w, sw).t()
        assert float(want.abs().max()) <= 2.0 ** -6 * K
        out = vg.nvfp4_gemm(a, sa.to(f8), w, sw.to(f8), one(1.0))
        assert torch.equal(out, want.to(torch.bfloat16))


def test_outputs_past_32_bit_offsets():
    """Outputs of more than 2^31 elements: rows sampled over all of them."""
    import torch
    T, N, K = 70001, 32768, 64
    a, sa = operand(T, K, 5, exact=True)
    w, sw = operand(N, K, 6, exact=True)
    rows = torch.tensor([0, 127, 128, 40000, 65535, 65536, 65537, 69999, 70000], device="cuda")
    out = vg.nvfp4_gemm(a, sa, w, sw, one(1.0))
    W = scaled(w, sw)
    assert torch.equal(out[rows], (scaled(a[rows], sa.view(torch.uint8)[rows].view(sa.dtype)) @ W.t()).to(torch.bfloat16))
    del out
    w2, sw2 = torch.cat([w, w]), torch.cat([sw.view(torch.uint8)] * 2).view(sw.dtype)
    q4, sf = vg.nvfp4_gemm_silu_mul_nvfp4(a, sa, w2, sw2, one(0.1), one(10.0))
    few = vg.nvfp4_gemm_silu_mul_nvfp4(a[rows], sa.view(torch.uint8)[rows].view(sa.dtype), w2, sw2, one(0.1), one(10.0))
    # the sums are exact in either kernel, and the same steps follow
    assert torch.equal(q4[rows], few[0])
    assert torch.equal(sf.view(torch.uint8)[rows], few[1].view(torch.uint8))


@pytest.mark.parametrize("T,N,K", [(2 ** 24, 8, 64), (1, 2 ** 20, 64), (130, 2 ** 20, 64), (5, 8, 32768)])
def test_largest_sizes(T, N, K):
    import torch
    a, sa = operand(T, K, 1, exact=True)
    w, sw = operand(N, K, 2, exact=True)
    out = vg.nvfp4_gemm(a, sa, w, sw, one(1.0))
    at = lambda n: torch.tensor(sorted({0, n // 3, n // 2, n - 1}), device="cuda")  # noqa: E731
    pick = lambda q, s, i: scaled(q[i], s.view(torch.uint8)[i].view(s.dtype))  # noqa: E731
    want = pick(a, sa, at(T)) @ pick(w, sw, at(N)).t()
    assert torch.equal(out[at(T)][:, at(N)], want.to(torch.bfloat16))
    if T == 2 ** 24:
        w, sw = operand(128, K, 3, exact=True)
        q4, sf = vg.nvfp4_gemm_silu_mul_nvfp4(a, sa, w, sw, one(0.1), one(10.0))
        few = vg.nvfp4_gemm_silu_mul_nvfp4(a[at(T)], sa.view(torch.uint8)[at(T)].view(sa.dtype), w, sw, one(0.1), one(10.0))
        assert torch.equal(q4[at(T)], few[0])
        assert torch.equal(sf.view(torch.uint8)[at(T)], few[1].view(torch.uint8))


@pytest.mark.parametrize("T,N", [(3, 262160), (262160, 16)])
def test_operands_past_32_bit_offsets(T, N):
    """A weight, then activations, of more than 2^32 bytes of codes; rows sampled."""
    import torch
    K, big = 32768, max(T, N)
    few, sfew = operand(min(T, N), K, 1, exact=True)
    base, sbase = operand(997, K, 2, exact=True)
    many = base.repeat(big // 997 + 1, 1)[:big].contiguous()
    smany = sbase.view(torch.uint8).repeat(big // 997 + 1, 1)[:big].contiguous().view(sbase.dtype)
    a, sa, w, sw = (few, sfew, many, smany) if T < N else (many, smany, few, sfew)
    out = vg.nvfp4_gemm(a, sa, w, sw, one(1.0))
    at = torch.tensor([0, 127, 131071, 131072, 131073, 262143, 262144, big - 1], device="cuda")
    rows = torch.arange(T, device="cuda") if T < N else at
    cols = at if T < N else torch.arange(N, device="cuda")
    pick = lambda q, s, i: scaled(q[i], s.view(torch.uint8)[i].view(s.dtype))  # noqa: E731
    assert torch.equal(out[rows][:, cols], (pick(a, sa, rows) @ pick(w, sw, cols).t()).to(torch.bfloat16))


@pytest.mark.parametrize("T", [1, 40, 300, 700])
def test_gated_zero_rows_and_saturated_gates(T):
    """A zero token gives zero scales and codes, and is no slower for it; gates far
    on either side: silu(g) = g, or 0; an output scale that saturates the blocks."""
    import torch
    I, K = 256, 256
    a, sa = operand(T, K, T)
    w, sw = operand(2 * I, K, T + 1)
    a[T // 2] = 0
    alpha = float(np.float32(1e-4))
    A, W = scaled(a, sa), scaled(w, sw) * alpha
    c, e = A @ W.t(), product_error(A, W, K)
    assert T == 1 or float(c[:, :I].abs().max()) > 90  # exp() over- and underflows
    for gs in (1e-3, 1.0, 1e6):
        q4, sf = vg.nvfp4_gemm_silu_mul_nvfp4(a, sa, w, sw, one(alpha), one(gs))
        assert not bool(q4[T // 2].any()) and not bool(sf.view(torch.uint8)[T // 2].any())
        check_gated(q4, sf, c[:, :I], c[:, I:], e[:, :I], e[:, I:], gs)


@pytest.mark.parametrize("T", [1, 40, 700])
def test_infinite_factors_follow_ieee_arithmetic(T):
    import torch
    N, K = 256, 256
    a, sa = operand(T, K, 8, exact=True)
    w, sw = operand(N, K, 9, exact=True)
    c = scaled(a, sa) @ scaled(w, sw).t()
    out = vg.nvfp4_gemm(a, sa, w, sw, one(float("inf"))).float()
    want = torch.where(c == 0, float("nan"), c.sign() * float("inf")).float()
    assert torch.equal(out.nan_to_num(7.0, 8.0, 9.0), want.nan_to_num(7.0, 8.0, 9.0))
    assert bool(vg.nvfp4_gemm(a, sa, w, sw, one(float("nan"))).isnan().all())


@pytest.mark.parametrize("T", [1, 40, 700])
def test_gated_not_finite(T):
    """Infinite and NaN gates and ups, and blocks of NaNs alone."""
    import torch
    I, K = 256, 256
    a, sa = operand(T, K, 8, exact=True)
    w, sw = operand(2 * I, K, 9, exact=True)
    w[32:48], w[I + 64:I + 80] = 0, 0  # zero sums: NaN with an infinite alpha
    q4, sf = vg.nvfp4_gemm_silu_mul_nvfp4(a, sa, w, sw, one(float("inf")), one(1.0))
    c = (scaled(a, sa) @ scaled(w, sw).t() * float("inf"))
    g, u = c[:, :I], c[:, I:]
    y = torch.where(g == -float("inf"), float("nan"), g) * u
    block = lambda x: x.view(T, I // 16, 16)  # noqa: E731
    inf = torch.isinf(block(y)).any(-1)
    assert torch.equal(sf.float(), torch.where(inf, 448.0, 0.0).float())
    got = block(values(q4))
    assert bool((got[~inf] == 0).all()) and bool((got[inf].abs() == 6).all())
    at = torch.isinf(block(y))
    assert torch.equal(got[at].sign(), block(y)[at].sign())


@pytest.mark.parametrize("K", [64, 192, 256, 448, 512])
@pytest.mark.parametrize("T,N", [(5, 72), (300, 10240)])
def test_rows_of_larger_tensors(T, N, K):
    """Operands and outputs that are some rows of larger tensors, at any row, and
    scales that are 4-byte aligned only."""
    import torch
    a, sa = operand(T + 9, K, 1, exact=True)
    w, sw = operand(N + 64, K, 2, exact=True)
    for i, j in ((1, 3), (8, 64)):
        buf = torch.zeros((T + 9, N), dtype=torch.bfloat16, device="cuda")
        vg.vg_nvfp4_gemm(buf[i:i + T], a[i:i + T], sa[i:i + T], w[j:j + N], sw[j:j + N], one(1.0))
        want = (scaled(a[i:i + T], sa[i:i + T]) @ scaled(w[j:j + N], sw[j:j + N]).t()).to(torch.bfloat16)
        assert torch.equal(buf[i:i + T], want)
        assert not bool(buf[:i].any()) and not bool(buf[i + T:].any())
    odd = torch.zeros(sa.numel() + 4, dtype=torch.uint8, device="cuda")[4:].view(sa.dtype).view(sa.shape)
    odd.copy_(sa)
    assert torch.equal(vg.nvfp4_gemm(a, odd, w, sw, one(1.0)), vg.nvfp4_gemm(a, sa, w, sw, one(1.0)))


@pytest.mark.parametrize("T", [1, 50, 200, 700])
def test_captured_calls_and_two_streams(T):
    """Captured calls follow their inputs, and calls on two streams at once do not
    disturb each other: there is no workspace to share."""
    import torch
    N, K = 4096, 2048
    sets = [(*operand(T, K, 10 + k), *operand(N, K, 20 + k), one(1e-4 * (k + 1))) for k in range(2)]
    xs = [torch.randn((T, K), device="cuda", generator=torch.Generator(device="cuda").manual_seed(k)).bfloat16()
          for k in range(2)]

    def run(s, x):
        q4, sf = vg.nvfp4_quantize(x, s[4])
        g4, gf = vg.nvfp4_gemm_silu_mul_nvfp4(*s, s[4])
        return (vg.nvfp4_gemm(*s), q4, sf.view(torch.uint8), vg.nvfp4_dequantize(q4, sf, s[4]), g4,
                gf.view(torch.uint8))
    want = [run(s, x) for s, x in zip(sets, xs)]
    live, x = [t.clone() for t in sets[0]], xs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(live, x)
    for k in (1, 0):
        for dst, src in zip((*live, x), (*sets[k], xs[k])):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want[k]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k].append(run(sets[k], xs[k]))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(p, q) for r in got[k] for p, q in zip(r, want[k]))
