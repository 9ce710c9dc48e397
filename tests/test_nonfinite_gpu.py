"""NaN and infinity inputs: the CUDA path against the oracle (GPU).

The reading both sides follow: every formula is evaluated in IEEE
arithmetic as written, and the amax of a row or group is the largest |y|
among its non-NaN elements (0 when there is none).  So a NaN in r makes the
whole row NaN (codes 0x7F, dynamic scales at the floor); an infinity in r
gives inv = 0, codes +-0 at the finite elements and 0x7F at the infinite
one; an infinite SiLU activation saturates under a static scale and makes
its row's or group's dynamic scale +inf.  The oracle's side is pinned by
check_nonfinite_norm / check_nonfinite_silu.  Both the register kernels
(few rows) and the pipelined kernels (many rows) are covered.
"""
from __future__ import annotations

import numpy as np
import pytest

import gen
import norm_activation_fp8_gb300 as vg
import parity

pytestmark = pytest.mark.gpu

STATIC, PER_TOKEN, PER_GROUP = 0, 1, 2
UE8M0, COL_MAJOR = parity.UE8M0, parity.COL_MAJOR
NAN16, PINF16, NINF16 = 0x7FC0, 0x7F80, 0xFF80


@pytest.fixture(scope="module", autouse=True)
def cuda_library():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from norm_activation_fp8_gb300 import build
    build.build()
    import norm_activation_fp8_gb300 as vg
    vg.load()


def plant_norm(x, res, rng, with_inf=True):
    """NaN / +-inf at random places of a few rows; returns the planted rows."""
    T, H = x.shape
    rows = rng.permutation(T)[:28]
    cols = rng.integers(0, H, rows.size)
    kinds = ["x_nan", "res_nan", "x_inf", "res_ninf", "inf_minus_inf"] if with_inf \
        else ["x_nan", "res_nan"]
    for i, (t, j) in enumerate(zip(rows, cols)):
        k = kinds[i % len(kinds)]
        if k == "x_nan":
            x[t, j] = NAN16
        elif k == "res_nan" and res is not None:
            res[t, j] = NAN16
        elif k == "x_inf":
            x[t, j] = PINF16
        elif k == "res_ninf" and res is not None:
            res[t, j] = NINF16
        elif k == "inf_minus_inf" and res is not None:
            x[t, j], res[t, j] = PINF16, NINF16
        else:
            x[t, j] = NAN16 if i % 2 else PINF16
    return rows


NORM_MODES = [(STATIC, 128), (PER_TOKEN, 128), (PER_GROUP, 128), (PER_GROUP, 64),
              (PER_GROUP | COL_MAJOR, 128), (PER_GROUP | UE8M0, 128)]


@pytest.mark.parametrize("T,H", [(64, 4096), (1024, 4096)], ids=["register", "pipelined"])
@pytest.mark.parametrize("mode,G", NORM_MODES, ids=lambda v: str(v))
@pytest.mark.parametrize("fused", [True, False], ids=["fused_add", "plain"])
def test_nonfinite_norm(T, H, mode, G, fused):
    rng = np.random.default_rng(T + mode + G)
    d = gen.norm_inputs(T, H, seed=5)
    x, w = d["x"].copy(), d["weight"]
    res = d["residual"].copy() if fused else None
    # an infinite amax has no power-of-two scale: UE8M0 gets NaN rows only
    rows = plant_norm(x, res, rng, with_inf=not (mode & UE8M0))
    g = parity.gpu_norm(x, res, w, 1e-5, mode, G, scale=0.05)
    o = parity.oracle_norm(x, res, w, 1e-5, mode, G, scale=0.05)
    parity.check_norm(g, o, mode & 0xFF)
    assert np.any(g["q"][rows] == 0x7F)


@pytest.mark.parametrize("mode,G", [(STATIC, 128), (PER_TOKEN, 128), (PER_GROUP, 128)],
                         ids=lambda v: str(v))
@pytest.mark.parametrize("T", [64, 1024], ids=["register", "pipelined"])
def test_nan_weight_and_zero_rows_without_eps(T, mode, G):
    """A NaN weight column turns only that column into NaN; with eps = 0 an
    all-zero row is 0 * (1/0) = NaN everywhere (the other rows are defined)."""
    H = 4096
    d = gen.norm_inputs(T, H, seed=6)
    w = d["weight"].copy()
    w[[3, 1000, 4095]] = NAN16
    g = parity.gpu_norm(d["x"], d["residual"], w, 1e-5, mode, G, scale=0.05)
    o = parity.oracle_norm(d["x"], d["residual"], w, 1e-5, mode, G, scale=0.05)
    parity.check_norm(g, o, mode)
    assert np.all(g["q"][:, [3, 1000, 4095]] == 0x7F)
    x = d["x"].copy()
    x[[0, T // 2, T - 1]] = 0
    g = parity.gpu_norm(x, None, d["weight"], 0.0, mode, G, scale=0.05)
    o = parity.oracle_norm(x, None, d["weight"], 0.0, mode, G, scale=0.05)
    parity.check_norm(g, o, mode)
    assert np.all(g["q"][[0, T // 2, T - 1]] == 0x7F)


def plant_silu(gu, rng, with_inf=True):
    T, two_i = gu.shape
    I = two_i // 2
    rows = rng.permutation(T)[:30]
    cols = rng.integers(0, I, rows.size)
    kinds = ["gate_nan", "up_nan", "gate_ninf", "up_inf", "gate_inf"] if with_inf \
        else ["gate_nan", "up_nan"]
    for i, (t, j) in enumerate(zip(rows, cols)):
        k = kinds[i % len(kinds)]
        if k == "gate_nan":
            gu[t, j] = NAN16
        elif k == "up_nan":
            gu[t, I + j] = NAN16
        elif k == "gate_ninf":
            gu[t, j] = NINF16           # silu(-inf) = -inf / inf = NaN
        elif k == "up_inf":
            gu[t, I + j] = PINF16       # +-inf, or NaN where the gate is 0
        else:
            gu[t, j] = PINF16           # silu(inf) = inf, times up
    return rows


SILU_MODES = [(STATIC, 128), (PER_TOKEN, 128), (PER_GROUP, 128), (PER_GROUP, 64),
              (PER_GROUP | COL_MAJOR, 128), (PER_GROUP | UE8M0, 128)]


@pytest.mark.parametrize("T,I", [(64, 4096), (400, 4096)], ids=["register", "pipelined"])
@pytest.mark.parametrize("mode,G", SILU_MODES, ids=lambda v: str(v))
def test_nonfinite_silu(T, I, mode, G):
    rng = np.random.default_rng(T + mode + G + 1)
    gu = gen.silu_inputs(T, I, seed=7)["gate_up"].copy()
    rows = plant_silu(gu, rng, with_inf=not (mode & UE8M0))
    g = parity.gpu_silu(gu, mode, G, scale=0.1)
    o = parity.oracle_silu(gu, mode, G, scale=0.1)
    parity.check_silu(g, o, mode & 0xFF)
    assert np.any(g["q"][rows] == 0x7F)


# T, I, K that take every form of the gated projection: streams of 16 to 128
# tokens, tiles, tiles with K shared
GATED = [(1, 256, 256), (20, 256, 256), (50, 256, 256), (83, 23936, 256), (2049, 2048, 256), (609, 640, 11904)]


def test_gated_sizes_take_every_form():
    import test_layer_ops_host as host
    plans = {host.plan(*x, True, 152) for x in GATED}
    assert {tn for tn, _ in plans} == {0, 16, 32, 64, 128} and {(0, 1), (0, 3)} <= plans


def _gated(sa, n, m, codes, I, K):
    """Operands with g[t, i] = codes[t] n[i] sa[t, 0], u[t, i] = codes[t] m[i]
    sa[t, 1] (each exactly, or an overflow) in the first columns and zeros in
    the others, and these g and u as fp32 tensors.  (+ 0.0: a sum with other,
    positive zeros among its terms is not -0.)"""
    import torch
    T, cols = sa.shape[0], n.shape[0]
    a, w = torch.zeros((T, K), device="cuda"), torch.zeros((2 * I, K), device="cuda")
    a[:, 0] = a[:, 128] = codes
    w[:cols, 0], w[I:I + cols, 128] = n, m
    f8 = torch.float8_e4m3fn
    scales = torch.ones((T, K // 128), device="cuda")
    scales[:, :2] = sa
    sw = torch.ones((2 * I // 128, K // 128), device="cuda")
    g, u = codes[:, None] * n * sa[:, :1] + 0.0, codes[:, None] * m * sa[:, 1:] + 0.0
    return (a.to(f8), scales, w.to(f8), sw), g, u


def _run_gated(args, ue8m0):
    """Codes of the first two groups [T, 2, 128] and their scales."""
    import torch
    q, s = vg.fp8_block_gemm_silu_mul_fp8(*args, 0, vg.UE8M0 if ue8m0 else 0)
    return q.view(torch.uint8)[:, :256].reshape(-1, 2, 128), s[:, :2]


def _codes(v):
    import torch
    return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _signed(y, plus, minus):
    import torch
    return torch.where(y.signbit(), minus, plus).to(torch.uint8)


@pytest.mark.parametrize("T,I,K", GATED)
def test_nonfinite_gated_projection(T, I, K):
    """Activations beyond fp32, element by element: the group's scale is +inf,
    codes there NaN and signed zeros beside them; with UE8M0 the scale is 2^120
    (the largest that a finite amax takes) and the codes there +-448.  Groups
    without one do not notice, and vg_silu_mul_fp8 says the same of the same
    activations."""
    import torch
    g_ = torch.Generator(device="cuda").manual_seed(T)
    n, m = (torch.randint(-2, 3, (256,), generator=g_, device="cuda").float() for _ in range(2))
    m[128:] = m[128:].clamp(-1, 1)       # |g u| <= 2^127 in the second group
    n[:4], m[:4] = torch.tensor([2., 2, -2, -2]), torch.tensor([2., -2, 2, -2])
    n[130:132], m[130:132] = torch.tensor([2., -2]), torch.tensor([1., 1])
    sa = torch.full((T, 2), 2.0 ** 63, device="cuda")
    sa[1::3] = 1.0                       # tokens of ordinary size
    codes = torch.ones(T, device="cuda")
    codes[2::3] = -1.0                   # the other gates vanish
    big = torch.arange(T, device="cuda") % 3 != 1
    args, g, u = _gated(sa, n, m, codes, I, K)
    y = (g / (1 + torch.exp(-g)) * u).view(T, 2, 128)
    amax = y.abs().amax(-1)
    assert bool(amax[big, 0].isinf().all()) and bool((amax[big, 1] == 2.0 ** 127).all())
    for ue8m0 in (False, True):
        q, s = _run_gated(args, ue8m0)
        y0, q0 = y[big, 0], q[big, 0]
        inf = y0.isinf()
        if ue8m0:
            k = torch.ceil(torch.log2(amax.double() / 448)).clamp_max(120)
            assert torch.equal(s.double(), torch.exp2(k))
            assert torch.equal(q0[inf], _signed(y0[inf], 0x7E, 0xFE))
            assert torch.equal(q0[~inf], _codes(y0[~inf] * 2.0 ** -120))
            assert torch.equal(q[big, 1], _codes(y[big, 1] / s[big, 1, None]))
        else:
            ok = ~amax.isinf()
            assert torch.equal(s.isinf(), ~ok)
            assert bool(((s - amax / 448)[ok].abs() <= 2.0 ** -20 * s[ok]).all())
            assert bool((q0[inf] & 0x7F == 0x7F).all())
            assert torch.equal(q0[~inf], _signed(y0[~inf], 0, 0x80))
            # 0, 2^126 and 2^127 under 2^127 / 448: codes 0, 224, 448
            assert torch.equal(q[big, 1], _codes(y[big, 1] * 2.0 ** -127 * 448))
        if I == 256:  # the same activations (exact as bf16) through the unfused op
            q2, s2 = vg.silu_mul_fp8(torch.cat([g, u], 1).bfloat16(), vg.PER_GROUP | (vg.UE8M0 if ue8m0 else 0))
            assert torch.equal(q[big], q2.view(torch.uint8).view(T, 2, 128)[big])
            assert torch.equal(s2[big].isinf(), s[big].isinf()) and (not ue8m0 or torch.equal(s2[big], s[big]))


@pytest.mark.parametrize("one_block", [False, True], ids=["two", "one"])
@pytest.mark.parametrize("T,I,K", GATED)
def test_infinite_token_scales_gated_projection(T, I, K, one_block):
    """An infinite scale of a.  With the gates' and the up values' products in
    the one block that has it, g and u are +-inf, or NaN where their product is
    zero; silu(-inf) is NaN; a NaN never wins the amax.  With either's in a
    block of its own, and both scales infinite, each meets a zero product of
    the other block: inf * 0, NaN throughout, under the floor scale."""
    import torch
    t = T // 2
    g_ = torch.Generator(device="cuda").manual_seed(T)
    n, m = (torch.randint(-2, 3, (256,), generator=g_, device="cuda").float() for _ in range(2))
    n[128:] = -n[128:].abs()             # the second group: NaN throughout
    one = torch.ones(T, device="cuda")
    clean, g, u = _gated(torch.ones((T, 2), device="cuda"), n, m, one, I, K)
    if one_block:
        w = clean[2].view(torch.uint8)
        w[I:, 0] = w[I:, 128]
        w[I:, 128] = 0
    scales = clean[1].clone()
    scales[t, :1 if one_block else 2] = float("inf")
    args = (clean[0], scales, *clean[2:])
    inf = torch.tensor(float("inf"), device="cuda")
    g, u = (g[t] * inf, u[t] * inf) if one_block else (g[t] * inf + 0 * inf, u[t] * inf + 0 * inf)
    y = (g / (1 + torch.exp(-g)) * u).view(2, 128)
    is_inf = y[0].isinf()
    assert bool(is_inf.any()) == one_block and bool(y[0].isnan().any()) and bool(y[1].isnan().all())
    keep = torch.arange(T, device="cuda") != t
    for ue8m0 in (False, True):
        floor = 2.0 ** -42 if ue8m0 else 1e-10 / 448  # 2^-43 < 1e-10 / 448 < 2^-42
        q, s = _run_gated(args, ue8m0)
        q1, s1 = _run_gated(clean, ue8m0)
        assert torch.equal(q[keep], q1[keep]) and torch.equal(s[keep], s1[keep])
        assert bool((q[t][y.isnan()] & 0x7F == 0x7F).all())
        for k in range(2):
            if k == 0 and one_block:
                assert float(s[t, k]) == (2.0 ** 120 if ue8m0 else float("inf"))
            else:
                assert abs(float(s[t, k]) / floor - 1) < 2.0 ** -21
        if ue8m0:
            assert torch.equal(q[t, 0][is_inf], _signed(y[0][is_inf], 0x7E, 0xFE))
        else:
            assert bool((q[t, 0][is_inf] & 0x7F == 0x7F).all())


@pytest.mark.parametrize("T,I,K", GATED)
def test_gated_activation_within_the_stated_bound(T, I, K):
    """One active column a group, so that the scale shows y to fp32: gates from
    -85 to 85 with up values that keep y in range.  |dy| <= (5 + 1.2 |g|) 2^-23
    |y|: __expf is off by 2 + 1.173 |g| ulps, the sum and the product with u by
    half an ulp each, __fdividef by two; the scale adds 2^-23 (1 / 448 and the
    product, half an ulp each)."""
    import torch
    g = torch.linspace(-85, 85, T, device="cuda") if T > 1 else torch.tensor([-60.0], device="cuda")
    g[T // 3] = -0.375
    g[T // 2] = -60.5
    u = torch.exp2(torch.round(torch.where(g < 0, -g, -torch.ones_like(g)) * 1.45))  # about e^-g, a power of two
    n = torch.zeros(256, device="cuda")
    n[77] = 1.0
    args, _, _ = _gated(torch.stack([g, u], 1), n, n, torch.ones(T, device="cuda"), I, K)
    q, s = _run_gated(args, False)
    gd, ud = g.double(), u.double()
    y = (gd / (1 + torch.exp(-gd)) * ud).abs()
    err = (s[:, 0].double() * 448 - y).abs() / y
    tol = (6 + 1.2 * gd.abs()) * 2.0 ** -23
    assert bool((err <= tol).all()), float((err / tol).max())
    assert torch.equal(q[:, 0, 77], _signed(g, 0x7E, 0xFE))
    q[:, 0, 77] = 0
    assert bool((q & 0x7F == 0).all())
