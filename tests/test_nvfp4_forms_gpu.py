"""Every kernel form of the NVFP4 products: each token tile with each split of K,
plain and gated, rows of scales of whole 16 bytes (K a multiple of 256) and not.
The sums of each form are held in fp32, and the debug build, which checks every
access against its tensor, gives the same results and finds nothing.

Tolerance: none.  The plain results are the correctly rounded ones, and what the
gated form's codes may be follows from check_gated() with exact g and u."""
import numpy as np
import pytest

import norm_activation_fp8_gb300 as vg
from norm_activation_fp8_gb300 import build
from test_nvfp4_gemm_gpu import check_gated, one, packed, scaled
from test_nvfp4_layer_gpu import _gated, _gemm, _with

pytestmark = pytest.mark.gpu

PLAIN = [  # T, N, K
    (1691, 1224, 704), (1155, 2000, 512), (757, 2784, 896), (742, 2720, 1024), (1116, 712, 9792),
    (861, 872, 10752), (907, 752, 12608), (766, 952, 11264), (1, 136, 64), (3, 136, 256), (1, 136, 320),
    (15, 136, 512), (1, 136, 1600), (7, 136, 1792), (2, 136, 5184), (1, 136, 5376), (17, 136, 64),
    (31, 136, 256), (17, 136, 320), (25, 136, 512), (17, 136, 1600), (29, 136, 1792), (19, 136, 5184),
    (17, 136, 5376), (33, 136, 64), (63, 136, 256), (33, 136, 320), (50, 136, 512), (33, 136, 1600),
    (57, 136, 1792), (35, 136, 5184), (33, 136, 5376), (475, 4016, 192), (1089, 1384, 256), (325, 2680, 448),
    (742, 1208, 512), (474, 984, 1984), (734, 616, 2048), (73, 1448, 12224), (84, 1488, 10240),
]
GATED = [  # T, I, K
    (1283, 1600, 64), (1419, 832, 512), (482, 2112, 960), (450, 2112, 1024), (897, 448, 10176),
    (837, 448, 9984), (730, 448, 13248), (726, 448, 12288), (1, 192, 64), (3, 192, 256), (1, 192, 320),
    (15, 192, 512), (1, 192, 1600), (7, 192, 1792), (2, 192, 5184), (1, 192, 5376), (17, 192, 64),
    (31, 192, 256), (17, 192, 320), (25, 192, 512), (17, 192, 1600), (29, 192, 1792), (19, 192, 5184),
    (17, 192, 5376), (33, 192, 64), (63, 192, 256), (33, 192, 320), (50, 192, 512), (33, 192, 1600),
    (57, 192, 1792), (35, 192, 5184), (33, 192, 5376), (1269, 832, 192), (1091, 704, 256), (577, 832, 448),
    (771, 576, 512), (742, 320, 2752), (458, 448, 2048), (472, 192, 18368), (455, 192, 18432),
]


def cancelling(T, N, K, pairs, seed):
    """Operands whose products are multiples of 2^-8, at most 2^-6 each, but for a
    +96^2 and a -96^2 at each of `pairs` (columns of K, multiples of 16)."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    draw = lambda *a: torch.randint(*a, generator=g, device="cuda")  # noqa: E731
    # values 0, +-0.5, +-1 (codes 0 to 2) under scales of 2^-3
    ca, cw = draw(0, 3, (T, K)) | draw(0, 2, (T, K)) << 3, draw(0, 3, (N, K)) | draw(0, 2, (N, K)) << 3
    sa, sw = torch.full((T, K // 16), 0.125, device="cuda"), torch.full((N, K // 16), 0.125, device="cuda")
    st, sn = draw(0, 2, (T, 1)) * 8, draw(0, 2, (N, 1)) * 8
    for at, sign in ((0, 0), (1, 8)) if pairs else ():
        # a block of 16 with one code 6 under a scale of 16
        b = torch.tensor([p[at] for p in pairs], device="cuda")
        inside = (b[:, None] + torch.arange(16, device="cuda")).flatten()
        ca[:, inside], cw[:, inside] = 0, 0
        sa[:, b // 16], sw[:, b // 16] = 16.0, 16.0
        ca[:, b + 5], cw[:, b + 5] = 7 | st, 7 | (sn ^ sign)
    f8 = torch.float8_e4m3fn
    return packed(ca.to(torch.uint8)), sa.to(f8), packed(cw.to(torch.uint8)), sw.to(f8)


def arrangements(K):
    """Where the large products and what cancels them lie: in one instruction (a K
    of 64), in neighbouring ones, in the first and the last share of K."""
    yield [(k, k + 48) for k in range(0, K, 64)]
    yield [(k, k + 64) for k in range(0, K - 64, 128)]
    yield [(0, K - 64)] if K >= 128 else []


# Every partial sum, in whatever order and of whichever share, is a multiple of
# 2^-8 below 96^2 + 2^-6 K < 2^14: fp32 holds it, and whatever has fewer than
# 22 bits loses some.

@pytest.mark.parametrize("T,N,K", PLAIN)
def test_sums_are_held_in_fp32(T, N, K):
    import torch
    for i, pairs in enumerate(arrangements(K)):
        a, sa, w, sw = cancelling(T, N, K, pairs, T + N + i)
        want = scaled(a, sa) @ scaled(w, sw).t()
        assert float(want.abs().max()) <= 2.0 ** -6 * K
        assert torch.equal(vg.nvfp4_gemm(a, sa, w, sw, one(1.0)), want.to(torch.bfloat16))
    assert vg.vg_device_status() == 0


@pytest.mark.parametrize("T,I,K", GATED)
def test_gated_sums_are_held_in_fp32(T, I, K):
    """Exact sums times a power of two near one over their deviation: g and u are
    of order one, and an error of 2^-8 in a sum is some percent of it."""
    alpha = 1.0
    while alpha * 0.0065 * K ** 0.5 < 1:  # a product's deviation: (0 + 1/4 + 1) / 3 * 2^-6
        alpha *= 2
    for i, pairs in enumerate(arrangements(K)):
        a, sa, w, sw = cancelling(T, 2 * I, K, pairs, T + I + i)
        c = scaled(a, sa) @ scaled(w, sw).t() * alpha
        q4, sf = vg.nvfp4_gemm_silu_mul_nvfp4(a, sa, w, sw, one(alpha), one(100.0))
        zero = c.new_zeros(())
        check_gated(q4, sf, c[:, :I], c[:, I:], zero, zero, 100.0)
    assert vg.vg_device_status() == 0


def test_the_gated_check_sees_a_lost_bit():
    """The same check refuses codes where the expected sums are one unit off."""
    T, I, K, alpha = 33, 192, 512, 8.0
    a, sa, w, sw = cancelling(T, 2 * I, K, [(0, 48)], 1)
    c = scaled(a, sa) @ scaled(w, sw).t() * alpha
    q4, sf = vg.nvfp4_gemm_silu_mul_nvfp4(a, sa, w, sw, one(alpha), one(100.0))
    zero = c.new_zeros(())
    check_gated(q4, sf, c[:, :I], c[:, I:], zero, zero, 100.0)
    for off in (c + alpha * 2.0 ** -8, c - alpha * 2.0 ** -8):
        with pytest.raises(AssertionError):
            check_gated(q4, sf, off[:, :I], off[:, I:], zero, zero, 100.0)


FORMS = [(_gemm, *x) for x in PLAIN] + [(_gated, *x) for x in GATED]
IDS = [f"{f.__name__[1:]}-{T}-{N}-{K}" for f, T, N, K in FORMS]


@pytest.mark.parametrize("op,T,N,K", FORMS, ids=IDS)
def test_debug_build_matches_and_reports_nothing(op, T, N, K, monkeypatch):
    run = op(T, N, K)
    want, st0 = _with(vg.load(), run, monkeypatch)
    got, st = _with(vg.load(build.build_debug()), run, monkeypatch)
    assert st0 == 0 and st == 0, (st0, st)
    for k, v in want.items():
        assert np.array_equal(got[k], v), k


@pytest.mark.parametrize("op,T,N,K", FORMS, ids=IDS)
def test_out_of_range_accesses_are_flagged_and_skipped(op, T, N, K, monkeypatch):
    """With every tensor of tokens reported one row short: the last token's scale
    reads and the stores of its row are flagged, the other rows stay."""
    run = op(T, N, K)
    want, _ = _with(vg.load(), run, monkeypatch)
    got, st = _with(vg.load(build.build_debug(shrunk=True)), run, monkeypatch)
    assert st == vg.DEVICE_OUT_OF_BOUNDS, st
    for k, v in want.items():
        assert np.array_equal(got[k][:-1], v[:-1]), k
