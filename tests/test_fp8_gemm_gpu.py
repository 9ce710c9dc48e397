"""The block-scaled FP8 product and the gated feed-forward projection against
fp64, at the sizes where a tile, a split or a tail can go wrong.

Tolerances, derived (u = 2^-24, S = the sum of |products|, scaled):
  c    a block's 128 products are exact in fp32 and summed by fp32 additions
       in any order, each off by at most 2u of the running magnitude (2u, not
       u: the tensor cores may truncate); the two scales and the sum over the
       K/128 blocks add at most K/128 + 2 roundings.  |dc| <= E = 2u (K/128 +
       130) S.
  out  bf16(c): E + 2^-8 (|c| + E)
  y    |d silu| <= 1.1 |dg| (its largest slope), so |dy| <= Ey = 1.1 Eg (|u| +
       Eu) + |silu(g)| Eu + 2^-20 |y|  (exp, reciprocal: a few ulps)
  s    max Ey of the group / 448, and 2^-22 of its own
  q s  Ey + 2^-4 (|y| + Ey) + 2^-10 s (half a step, normal or subnormal)
Integer codes under power-of-two scales make every sum exact: there the result
has to be the correctly rounded one, bit for bit."""
import numpy as np
import pytest

import norm_activation_fp8_gb300 as vg

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BLOCK = 128


def operands(T, rows, K, seed, colmajor=False, exact=False):
    """a, a_scale (as passed), w, w_scale and the fp64 factors."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    kb, nb = K // BLOCK, (rows + BLOCK - 1) // BLOCK
    if exact:  # |sum| < 4 * 4 * 128 * 2^3 * K / 128 < 2^24 for K <= 32768
        a = torch.randint(-2, 3, (T, K), generator=g, device="cuda").float()
        w = torch.randint(-2, 3, (rows, K), generator=g, device="cuda").float()
        sa = 2.0 ** torch.randint(-1, 2, (T, kb), generator=g, device="cuda").float()
        sw = 2.0 ** torch.randint(-1, 2, (nb, kb), generator=g, device="cuda").float()
    else:
        a = torch.randn((T, K), generator=g, device="cuda") * 100
        w = torch.randn((rows, K), generator=g, device="cuda") * 100
        sa = torch.rand((T, kb), generator=g, device="cuda") * 0.02 + 1e-3
        sw = torch.rand((nb, kb), generator=g, device="cuda") * 1e-3 + 1e-5
    a, w = (x.clamp(-448, 448).to(torch.float8_e4m3fn) for x in (a, w))
    s = sa
    if colmajor:
        s = torch.full((kb, (T + 3) // 4 * 4), float("nan"), device="cuda")
        s[:, :T] = sa.t()
    A = a.double() * sa.double().repeat_interleave(BLOCK, 1)
    W = w.double() * sw.double().repeat_interleave(BLOCK, 0)[:rows].repeat_interleave(BLOCK, 1)
    return a, s, w, sw, A, W


def guarded(shape, dtype):
    """A tensor between bands that must stay as they are."""
    import torch
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((n + 512,), 0xAB, dtype=torch.uint8, device="cuda")
    return buf, buf[256:256 + n].view(dtype).view(shape)


def intact(buf):
    return bool((buf[:256] == 0xAB).all()) and bool((buf[-256:] == 0xAB).all())


def product_error(A, W, K):
    return 2 * U * (K // BLOCK + 130) * (A.abs() @ W.abs().t())


PLAIN = [  # T, N, K
    (1, 128, 128), (1, 8, 128), (1, 6144, 4096), (2, 136, 256), (3, 1000, 384), (8, 4096, 14336),
    (15, 512, 1024), (16, 520, 640), (17, 2048, 512), (31, 384, 896), (33, 1024, 2048), (64, 4096, 1152),
    (65, 640, 256), (100, 264, 32768), (127, 136, 512), (128, 256, 128), (129, 384, 1024),
    (200, 4096, 4096), (256, 4096, 2048), (257, 248, 384), (300, 6144, 1024), (513, 1032, 512),
    (1000, 2056, 896), (2049, 4096, 640), (4100, 264, 256),
    # the plans that the sizes above do not take
    (384, 4096, 4096), (196, 3704, 6912), (1465, 504, 29056), (20, 96, 128), (23, 744, 256),
    (24, 72, 13312), (69, 28872, 128), (70, 3800, 6912),
]


def test_sizes_take_every_plan():
    """On 152 SMs the sizes above run every kernel with every split that some
    size takes."""
    import test_layer_ops_host as host
    for sizes, gated in ((PLAIN, False), (GATED, True)):
        assert {host.plan(*x, gated, 152) for x in sizes} >= host.reachable(gated)


@pytest.mark.parametrize("T,N,K", PLAIN)
def test_gemm(T, N, K):
    import torch
    for colmajor in (False, True):
        a, s, w, sw, A, W = operands(T, N, K, T + N + K, colmajor)
        buf, out = guarded((T, N), torch.bfloat16)
        vg.vg_fp8_block_gemm(out, a, s, w, sw, vg.COLUMN_MAJOR if colmajor else 0)
        c = A @ W.t()
        e = product_error(A, W, K)
        assert bool(((out.double() - c).abs() <= e + 2.0 ** -8 * (c.abs() + e)).all())
        assert intact(buf)
        # exact sums: the correctly rounded result
        a, s, w, sw, A, W = operands(T, N, K, T, colmajor, exact=True)
        vg.vg_fp8_block_gemm(out, a, s, w, sw, vg.COLUMN_MAJOR if colmajor else 0)
        assert torch.equal(out, (A @ W.t()).to(torch.bfloat16))
        assert intact(buf)
    assert vg.vg_device_status() == 0


GATED = [  # T, I, K
    (1, 128, 128), (1, 14336, 512), (2, 256, 384), (7, 384, 4096), (15, 128, 256), (16, 512, 1024),
    (17, 128, 128), (33, 1024, 640), (57, 2048, 2048), (64, 384, 32768), (65, 256, 512), (127, 640, 256),
    (128, 128, 384), (129, 1152, 512), (200, 14336, 256), (256, 2048, 1024), (300, 128, 896),
    (513, 1024, 512), (1000, 896, 640), (2049, 2048, 256), (4100, 128, 128),
    (1738, 384, 18048), (609, 640, 11904), (812, 384, 25728), (22, 1152, 256), (25, 896, 512), (25, 256, 9472),
    (83, 23936, 256),
]


@pytest.mark.parametrize("T,I,K", GATED)
def test_gated(T, I, K):
    import torch
    for colmajor, ue8m0 in ((False, False), (True, False), (True, True)):
        a, s, w, sw, A, W = operands(T, 2 * I, K, T + I + K, colmajor)
        oo = (vg.COLUMN_MAJOR if colmajor else 0) | (vg.UE8M0 if ue8m0 else 0)
        qbuf, q = guarded((T, I), torch.float8_e4m3fn)
        t4 = (T + 3) // 4 * 4
        sbuf, scale = guarded((I // BLOCK, t4) if colmajor else (T, I // BLOCK), torch.float32)
        vg.vg_fp8_block_gemm_silu_mul_fp8(q, scale, a, s, w, sw, vg.COLUMN_MAJOR if colmajor else 0, oo)
        sc = scale[:, :T].t() if colmajor else scale
        if colmajor and t4 > T:  # padding columns are not written
            assert bool((scale[:, T:].contiguous().view(torch.uint8) == 0xAB).all())
        c, e = A @ W.t(), product_error(A, W, K)
        g, u, eg, eu = c[:, :I], c[:, I:], e[:, :I], e[:, I:]
        silu = g * torch.sigmoid(g)
        y = silu * u
        ey = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + 2.0 ** -20 * y.abs()
        grp = lambda x: x.view(T, I // BLOCK, BLOCK)  # noqa: E731
        amax, ea = grp(y.abs()).amax(-1), grp(ey).amax(-1)
        if ue8m0:
            lo, hi = (torch.exp2(torch.ceil(torch.log2(((amax + k * (ea + 2.0 ** -22 * amax)).clamp_min(1e-10)) / 448)))
                      for k in (-1, 1))
            assert bool(((sc.double() == lo) | (sc.double() == hi)).all())
        else:
            want = amax.clamp_min(1e-10) / 448
            assert bool(((sc.double() - want).abs() <= ea / 448 + 2.0 ** -22 * want).all())
        s64 = sc.double()[..., None]
        got = grp(q.double()) * s64
        tol = grp(ey) + 2.0 ** -4 * (grp(y.abs()) + grp(ey)) + 2.0 ** -10 * s64
        assert bool(((got - grp(y)).abs() <= tol).all())
        assert intact(qbuf) and intact(sbuf)
    assert vg.vg_device_status() == 0


@pytest.mark.parametrize("T,N,K", [(70001, 32768, 128), (70001, 32768, 256)])
def test_outputs_past_32_bit_offsets(T, N, K):
    """Outputs of more than 2^31 elements: rows sampled over all of them."""
    import torch
    a, s, w, sw, A, W = operands(T, N, K, 5, exact=True)
    rows = torch.tensor([0, 127, 128, 40000, 65535, 65536, 65537, 69999, 70000], device="cuda")
    out = vg.fp8_block_gemm(a, s, w, sw)
    assert torch.equal(out[rows], (A[rows] @ W.t()).to(torch.bfloat16))
    del out
    if K == 128:
        w2 = torch.cat([w.view(torch.uint8), w.view(torch.uint8)]).view(torch.float8_e4m3fn)
        q, sc = vg.fp8_block_gemm_silu_mul_fp8(a, s, w2, torch.cat([sw, sw]))
        few = vg.fp8_block_gemm_silu_mul_fp8(a.view(torch.uint8)[rows].view(torch.float8_e4m3fn), s[rows],
                                             w2, torch.cat([sw, sw]))
        # the sums are exact in either kernel, and the same steps follow
        assert torch.equal(q.view(torch.uint8)[rows], few[0].view(torch.uint8))
        assert torch.equal(sc[rows], few[1])


def test_weights_and_activations_past_32_bit_offsets():
    """A weight, then activations, of more than 2^32 codes; rows sampled."""
    import torch
    K = 32768
    for T, N in ((3, 131080), (131080, 16)):
        big = max(T, N)
        g = torch.Generator(device="cuda").manual_seed(T)
        base = torch.randint(-2, 3, (997, K), generator=g, device="cuda").to(torch.float8_e4m3fn)
        many = base.view(torch.uint8).repeat(big // 997 + 1, 1)[:big].view(torch.float8_e4m3fn)
        few = torch.randint(-2, 3, (min(T, N), K), generator=g, device="cuda").to(torch.float8_e4m3fn)
        a, w = (few, many) if T < N else (many, few)
        sa = 2.0 ** torch.randint(-1, 2, (T, K // BLOCK), generator=g, device="cuda").float()
        sw = 2.0 ** torch.randint(-1, 2, ((N + 127) // 128, K // BLOCK), generator=g, device="cuda").float()
        out = vg.fp8_block_gemm(a, sa, w, sw)
        at = torch.tensor([0, 127, 65535, 65536, 65537, 131071, 131072, big - 1], device="cuda")
        rows = torch.arange(T, device="cuda") if T < N else at
        cols = at if T < N else torch.arange(N, device="cuda")
        A = a.view(torch.uint8)[rows].view(torch.float8_e4m3fn).double() * sa[rows].double().repeat_interleave(BLOCK, 1)
        W = w.view(torch.uint8)[cols].view(torch.float8_e4m3fn).double()
        W = W * sw[cols // BLOCK].double().repeat_interleave(BLOCK, 1)
        assert torch.equal(out[rows][:, cols], (A @ W.t()).to(torch.bfloat16))


@pytest.mark.parametrize("T", [1, 40, 300])
def test_infinite_scales_follow_ieee_arithmetic(T):
    """An infinite token scale: its row is infinite or NaN where the products
    say so; the others do not notice.  Gated: infinite activations give the
    group an infinite scale and NaN codes there, zeros beside them."""
    import torch
    N, K = 256, 256
    a, s, w, sw, A, W = operands(T, N, K, 8, exact=True)
    t = T // 2
    s2 = s.clone()
    s2[t, 1] = float("inf")
    out, ref = vg.fp8_block_gemm(a, s2, w, sw), vg.fp8_block_gemm(a, s, w, sw)
    part = a[t, BLOCK:].double() @ w[:, BLOCK:].double().t()  # inf * part, then + finite
    want = torch.where(part == 0, float("nan"), part.sign() * float("inf")).float()
    assert torch.equal(out[t].float().nan_to_num(7.0, 8.0, 9.0), want.nan_to_num(7.0, 8.0, 9.0))
    keep = torch.arange(T, device="cuda") != t
    assert torch.equal(out[keep], ref[keep])
    q, sc = vg.fp8_block_gemm_silu_mul_fp8(a, s2, w, sw)
    q0, sc0 = vg.fp8_block_gemm_silu_mul_fp8(a, s, w, sw)
    assert torch.equal(q.view(torch.uint8)[keep], q0.view(torch.uint8)[keep]) and torch.equal(sc[keep], sc0[keep])
    assert not bool(torch.isfinite(sc[t]).all()) or bool((q[t].view(torch.uint8) & 0x7F == 0x7F).any())


def test_gated_zero_rows_and_saturated_gates():
    """A zero token: zero codes under the floor scale.  Gates far on either
    side: silu(g) = g, or -0."""
    import torch
    T, I, K = 40, 256, 256
    a, s, w, sw, A, W = operands(T, 2 * I, K, 1)
    az = a.clone().view(torch.uint8)
    az[3] = 0
    az[17] = 0
    big = s.clone()
    big[5:9] *= 1e4
    q, sc = vg.fp8_block_gemm_silu_mul_fp8(az.view(torch.float8_e4m3fn), big, w, sw)
    floor = torch.tensor(1e-10, dtype=torch.float32, device="cuda") / 448
    for t in (3, 17):
        assert bool((q[t].view(torch.uint8) & 0x7F == 0).all())
        assert bool(((sc[t] - floor).abs() <= 2.0 ** -22 * floor).all())
    A2 = A.clone()
    A2[5:9] *= 1e4
    g, u = (A2 @ W[:I].t()), (A2 @ W[I:].t())
    y = (g * torch.sigmoid(g) * u).view(T, I // BLOCK, BLOCK)[5:9]
    got = q.double().view(T, I // BLOCK, BLOCK)[5:9] * sc[5:9].double()[..., None]
    tol = 2.0 ** -4 * y.abs() * 1.01 + 1e-3 * y.abs().amax(-1, keepdim=True)
    assert bool(((got - y).abs() <= tol).all())


@pytest.mark.parametrize("T", [1, 40, 300])
def test_nan_codes_stay_in_their_row_and_column(T):
    """A NaN code of a makes its row NaN, one of w its column; a NaN among a
    group's activations leaves its scale the others' and its code NaN."""
    import torch
    N, K = 384, 512
    a, s, w, sw, A, W = operands(T, N, K, 3)
    a, w = a.view(torch.uint8).clone(), w.view(torch.uint8).clone()
    w[130, 200] = 0x7F
    if T > 1:
        a[T // 2, 77] = 0xFF
    f8 = torch.float8_e4m3fn
    out = vg.fp8_block_gemm(a.view(f8), s, w.view(f8), sw)
    nan = torch.zeros((T, N), dtype=torch.bool, device="cuda")
    nan[:, 130] = True
    if T > 1:
        nan[T // 2] = True
    assert torch.equal(out.isnan(), nan)
    # gated: w row 130 is up row 2 of an inter of 128 (rows 0..127 gate, 128.. up)
    q, sc = vg.fp8_block_gemm_silu_mul_fp8(a.view(f8), s, w.view(f8)[:256], sw[:2])
    want = torch.zeros((T, 128), dtype=torch.bool, device="cuda")
    want[:, 2] = True
    if T > 1:
        want[T // 2] = True
    assert torch.equal(q.view(torch.uint8) & 0x7F == 0x7F, want)
    assert bool(torch.isfinite(sc).all())


@pytest.mark.parametrize("T", [1, 50, 700])
def test_captured_calls_and_two_streams(T):
    """A captured product follows its inputs, and calls on two streams at once
    do not disturb each other: there is no workspace to share."""
    import torch
    N, K = 4096, 2048
    sets = [operands(T, N, K, 10 + k)[:4] for k in range(2)]
    want = [vg.fp8_block_gemm(*x) for x in sets]
    gated = [vg.fp8_block_gemm_silu_mul_fp8(*x) for x in sets]
    live = [x.clone() for x in sets[0]]
    for _ in range(2):
        vg.fp8_block_gemm(*live)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = vg.fp8_block_gemm(*live)
        q, sc = vg.fp8_block_gemm_silu_mul_fp8(*live)
    for k in (1, 0):
        for dst, src in zip(live, sets[k]):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[k])
        assert torch.equal(q.view(torch.uint8), gated[k][0].view(torch.uint8))
        assert torch.equal(sc, gated[k][1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k].append(vg.fp8_block_gemm(*sets[k]))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(x, want[k]) for x in got[k])


@pytest.mark.parametrize("big,step", [(256.0, 2.0 ** -4), (448.0, 2.0 ** -3)])
@pytest.mark.parametrize("T,N,K", [
    (1, 8, 128), (1, 6144, 4096), (20, 96, 128), (31, 384, 896), (50, 2056, 512), (69, 28872, 128),
    (70, 3800, 6912), (196, 3704, 6912), (1000, 2056, 896), (2049, 4096, 640)])
def test_block_sums_are_held_in_fp32(T, N, K, big, step):
    """Blocks with +big^2 and -big^2, in one product of 32 codes or in two,
    beside products that are multiples of 2^-3 step: their sum has to come out
    exact.  Every partial sum, in whatever order, is a multiple of 2^-3 step
    (2^-7, 2^-6) below big^2 + 126 * 2^-1 step < 2^17 (2^18), so it has at most
    24 bits; an accumulator of fewer, or products aligned to fewer, loses some."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T + N)
    kb = K // BLOCK
    for apart in (False, True):
        a = torch.randint(-2, 3, (T, K), generator=g, device="cuda") * 2.0 ** -3
        w = torch.randint(-2, 3, (N, K), generator=g, device="cuda") * step
        st = torch.randint(0, 2, (T, 1), generator=g, device="cuda") * 2.0 - 1
        sn = torch.randint(0, 2, (N, 1), generator=g, device="cuda") * 2.0 - 1
        for b in range(kb):
            p = int(torch.randint(0, 128, (1,), generator=g, device="cuda"))
            q = (p + 32 + 32 * (b % 3)) % 128 if apart else p ^ (1 + b % 31)
            p, q = b * BLOCK + p, b * BLOCK + q
            a[:, [p, q]] = big * st
            w[:, [p]], w[:, [q]] = big * sn, -big * sn
        f8 = torch.float8_e4m3fn
        assert bool((a.to(f8).float() == a).all()) and bool((w.to(f8).float() == w).all())
        want = a.double() @ w.double().t()
        assert float(want.abs().max()) < 4 * kb and (K == 128 or float(want.abs().max()) > 0)
        sa = torch.ones((T, kb), device="cuda")
        sw = torch.ones(((N + BLOCK - 1) // BLOCK, kb), device="cuda")
        out = vg.fp8_block_gemm(a.to(f8), sa, w.to(f8), sw)
        assert torch.equal(out, want.to(torch.bfloat16))
