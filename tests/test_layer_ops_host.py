"""The FP8 products and the rotary cache entry points on the host (no GPU):
every bad argument is refused before any CUDA call, so fake pointers are
safe; and the binding's own checks."""
import ctypes

import pytest

import norm_activation_fp8_gb300 as vg
from norm_activation_fp8_gb300 import build

OK, NULL, SHAPE, ALIGN, MODE, GROUP = 0, 1, 2, 3, 4, 5
A = 0x10000  # a 16-byte aligned fake device address (never dereferenced)
COL, POW2 = 0x200, 0x100


@pytest.fixture(scope="module")
def lib():
    build.build()
    return vg.load()


def gemm(lib, out=A, a=A, sa=A, w=A, sw=A, T=4, N=256, K=512, opt=0):
    return lib.vg_fp8_block_gemm(out, a, sa, w, sw, T, N, K, opt, None)


def gated(lib, q=A, s=A, a=A, sa=A, w=A, sw=A, T=4, I=256, K=512, opt=0, oopt=0):
    return lib.vg_fp8_block_gemm_silu_mul_fp8(q, s, a, sa, w, sw, T, I, K, opt, oopt, None)


def test_gemm_refusals(lib):
    for T in (-1, 2 ** 24 + 1, 2 ** 31):
        assert gemm(lib, T=T) == SHAPE and gated(lib, T=T) == SHAPE, T
    for n in (0, -8, 4, 12, 2 ** 20 + 8):
        assert gemm(lib, N=n) == SHAPE, n
    for n in (0, -128, 100, 32768 + 128):
        assert gated(lib, I=n) == SHAPE, n
    for k in (0, -128, 32768 + 128):
        assert gemm(lib, K=k) == SHAPE and gated(lib, K=k) == SHAPE, k
    for k in (64, 192, 4104):
        assert gemm(lib, K=k) == GROUP and gated(lib, K=k) == GROUP, k
    assert gated(lib, I=200) == GROUP
    for opt in (1, 2, POW2, COL | POW2, 0x400, -1):
        assert gemm(lib, opt=opt) == MODE and gated(lib, opt=opt) == MODE, opt
    for opt in (1, 2, 0x400, -1):
        assert gated(lib, oopt=opt) == MODE, opt
    for k in ("out", "a", "sa", "w", "sw"):
        assert gemm(lib, **{k: None}) == NULL, k
    for k in ("q", "s", "a", "sa", "w", "sw"):
        assert gated(lib, **{k: None}) == NULL, k
    for k in ("out", "a", "w"):
        assert gemm(lib, **{k: A + 8}) == ALIGN, k
    for k in ("q", "a", "w"):
        assert gated(lib, **{k: A + 8}) == ALIGN, k
    for k in ("sa", "sw"):
        assert gemm(lib, **{k: A + 2}) == ALIGN, k
    for k in ("s", "sa", "sw"):
        assert gated(lib, **{k: A + 1}) == ALIGN, k
    assert gemm(lib, out=None, a=None, sa=None, w=None, sw=None, T=0) == OK
    assert gated(lib, q=None, s=None, a=None, sa=None, w=None, sw=None, T=0) == OK


class GemmPlan(ctypes.Structure):
    _fields_ = [("tn", ctypes.c_int), ("splits", ctypes.c_int)]


def plan(T, N, K, gated, sms):
    """The library's own plan: (tokens a tile of the stream kernel or 0 for the
    tile kernel, ways that K is split)."""
    f = vg.load()._ZN2vg9plan_gemmElllbi
    f.restype, f.argtypes = GemmPlan, [ctypes.c_int64] * 3 + [ctypes.c_bool, ctypes.c_int]
    p = f(T, N, K, gated, sms)
    return p.tn, p.splits


def _sizes(gated, n, seed):
    import random
    r = random.Random(seed)
    unit = 128 if gated else 8
    for _ in range(n):
        yield (max(1, int(2 ** (13 * r.random()))), unit * int(2 ** ((8 if gated else 13) * r.random())),
               128 * int(2 ** (8 * r.random())))


def reachable(gated):
    return {plan(*x, gated, 152) for x in _sizes(gated, 20000, 1)}


@pytest.mark.parametrize("gated", [False, True])
def test_every_plan_can_be_launched(lib, gated):
    """A split never exceeds the scale blocks or its cluster the eight CTAs
    that may form one, the grid stays within its limits, and few tokens take
    one token tile."""
    sizes = list(_sizes(gated, 5000, 2)) + [(2 ** 24, 2 ** 15, 128), (2 ** 24, 128, 32768), (1, 128, 128)]
    if not gated:
        sizes += [(1, 2 ** 20, 32768), (2 ** 24, 8, 128), (128, 2 ** 20, 128), (1, 8, 32768)]
    for sms in (152, 148, 132, 16, 2, 1):
        for T, N, K in sizes:
            tn, splits = plan(T, N, K, gated, sms)
            assert 1 <= splits <= K // 128
            if tn == 0:
                assert splits <= 4
                tiles = (T + 255) // 256 * (N // 128 if gated else (N + 255) // 256)
                assert splits == 1 or 2 * splits * tiles < 2 ** 31
                assert tiles < 2 ** 32
            else:
                assert tn in (16, 32, 64, 128) and splits * (2 if gated else 1) in (1, 2, 4, 8)
                assert (T + tn - 1) // tn <= 65535
                assert T > 64 or tn >= T
    assert {tn for tn, _ in reachable(gated)} == {0, 16, 32, 64, 128}


def _sec(sections):
    return None if sections is None else (ctypes.c_int32 * len(sections))(*sections)


def mrope(lib, qkv=A, qw=A, kw=A, cache=A, pos=A, sec=(24, 20, 20), axes=3, T=4, hq=32, hkv=8,
          D=128, maxp=4096, inter=0):
    return lib.vg_fused_qk_norm_mrope(qkv, qw, kw, cache, pos, _sec(sec), axes, T, hq, hkv, D, maxp,
                                      1e-6, 1, inter, None)


def append(lib, qkv=A, kc=A, vc=A + 0x100000, qw=A, kw=A, cache=A, pos=A, slots=A, ks=None, vs=None, sec=None,
           axes=1, T=4, hq=32, hkv=8, D=128, maxp=4096, pages=64, page=16, ps=16 * 1024, ts=1024,
           hs=128, inter=0):
    return lib.vg_fused_qk_norm_rope_append(qkv, kc, vc, qw, kw, cache, pos, slots, ks, vs,
                                            _sec(sec), axes, T, hq, hkv, D, maxp, pages, page, ps,
                                            ts, hs, 1e-6, 1, inter, None)


def test_mrope_refusals(lib):
    for D in (0, 32, 96, 512):
        assert mrope(lib, D=D) == SHAPE, D
    assert mrope(lib, hq=0, hkv=0) == SHAPE
    assert mrope(lib, hq=4000, hkv=100) == SHAPE
    assert mrope(lib, maxp=0) == SHAPE
    assert mrope(lib, maxp=2 ** 31 // 128) == SHAPE           # table offsets past 31 bits
    assert mrope(lib, T=-1) == SHAPE
    for axes, sec in ((0, ()), (5, (24, 10, 10, 10, 10)), (3, None), (3, (24, 20, 19)),
                      (3, (65, 0, -1)), (2, (70, -6)), (1, (63,))):
        assert mrope(lib, axes=axes, sec=sec) == SHAPE, (axes, sec)
    # taking turns, the second axis needs pairs 1, 4, .., 3 * 21 + 1 = 64: one too many
    assert mrope(lib, sec=(22, 22, 20), inter=1) == SHAPE
    for k in ("qkv", "cache", "pos"):
        assert mrope(lib, **{k: None}) == NULL, k
    assert mrope(lib, qw=None) == NULL and mrope(lib, kw=None) == NULL  # a norm for one of the two
    for k in ("qkv", "qw", "kw", "cache"):
        assert mrope(lib, **{k: A + 8}) == ALIGN, k
    assert mrope(lib, pos=A + 4) == ALIGN
    for inter in (0, 1):
        assert mrope(lib, qkv=None, qw=None, kw=None, cache=None, pos=None, T=0, inter=inter) == OK
        assert mrope(lib, axes=4, sec=(64, 0, 0, 0), T=0, inter=inter) == OK
        assert mrope(lib, axes=2, sec=(0, 64), T=0, inter=inter) == (SHAPE if inter else OK)


def test_append_refusals(lib):
    for D in (0, 32, 96, 512):
        assert append(lib, D=D) == SHAPE, D
    assert append(lib, hkv=0) == SHAPE
    assert append(lib, T=-1) == SHAPE
    assert append(lib, axes=3) == SHAPE                     # several axes need sections
    assert append(lib, axes=3, sec=(24, 20, 19)) == SHAPE
    assert append(lib, pages=0) == SHAPE and append(lib, page=0) == SHAPE
    assert append(lib, pages=2 ** 20, page=2 ** 11) == SHAPE  # 2^31 slots
    assert append(lib, hs=64) == SHAPE                      # heads overlap
    assert append(lib, hs=132) == SHAPE                     # not whole chunks
    assert append(lib, ts=512) == SHAPE                     # tokens overlap the heads
    assert append(lib, ps=8 * 1024) == SHAPE                # pages overlap
    assert append(lib, ps=-16 * 1024) == SHAPE
    assert append(lib, ps=2 ** 62) == SHAPE                 # an offset past 64 bits
    assert append(lib, vc=A) == SHAPE                       # one cache for K and V
    # heads outside tokens, an extent of one with any stride, gaps
    assert append(lib, hs=16 * 128, ts=128, T=0) == OK
    assert append(lib, pages=1, ps=3, T=0) == OK
    assert append(lib, hkv=1, hs=0, T=0) == OK
    assert append(lib, ps=2 * 16 * 1024, T=0) == OK
    for k in ("qkv", "kc", "vc", "cache", "pos", "slots"):
        assert append(lib, **{k: None}) == NULL, k
    assert append(lib, qw=None) == NULL and append(lib, kw=None) == NULL
    assert append(lib, ks=A) == NULL and append(lib, vs=A) == NULL
    for k in ("qkv", "kc", "vc", "qw", "kw", "cache"):
        assert append(lib, **{k: 2 * A + 8}) == ALIGN, k
    assert append(lib, pos=A + 4) == ALIGN and append(lib, slots=A + 4) == ALIGN
    assert append(lib, ks=A + 2, vs=A) == ALIGN
    assert append(lib, qkv=None, kc=None, vc=None, qw=None, kw=None, cache=None, pos=None,
                  slots=None, T=0) == OK


def test_binding_refuses_cpu_tensors_and_bad_shapes(lib):
    import torch
    u8, f32, i64 = torch.uint8, torch.float32, torch.int64
    a, sa = torch.zeros(4, 256, dtype=u8), torch.zeros(4, 2)
    w, sw = torch.zeros(128, 256, dtype=u8), torch.zeros(1, 2)
    with pytest.raises(ValueError, match="CUDA"):
        vg.fp8_block_gemm(a, sa, w, sw)
    with pytest.raises(ValueError, match="same number of columns"):
        vg.fp8_block_gemm(a, sa, torch.zeros(128, 128, dtype=u8), sw)
    with pytest.raises(ValueError, match="a_scale"):
        vg.fp8_block_gemm(a, sa.t().contiguous(), w, sw)
    with pytest.raises(ValueError, match="a_scale"):
        vg.fp8_block_gemm(a, sa, w, sw, vg.COLUMN_MAJOR)
    with pytest.raises(ValueError, match="w_scale"):
        vg.fp8_block_gemm(a, sa, w, torch.zeros(2, 2))
    qkv = torch.zeros(4, 4 * 64, dtype=torch.bfloat16)
    table, pos = torch.zeros(16, 64), torch.zeros(4, dtype=i64)
    with pytest.raises(ValueError, match="columns"):
        vg.vg_fused_qk_norm_mrope(qkv, None, None, table, pos.view(1, 4), (32,), 1, 1, 64, 1e-6)
    with pytest.raises(ValueError, match="one row per axis"):
        vg.vg_fused_qk_norm_mrope(qkv, None, None, table, pos, (16, 16), 2, 1, 64, 1e-6)
    with pytest.raises(ValueError, match="number of tokens"):
        vg.vg_fused_qk_norm_mrope(qkv, None, None, table, pos[:3].view(1, 3), (32,), 2, 1, 64, 1e-6)
    with pytest.raises(ValueError, match="head_dim columns"):
        vg.vg_fused_qk_norm_mrope(qkv, None, None, table[:, :32], pos.view(1, 4), (32,), 2, 1, 64,
                                  1e-6)
    cache = torch.zeros(4, 16, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        vg.vg_fused_qk_norm_rope_append(qkv, cache, cache, None, None, table, pos, pos, 2, 1, 64, 1e-6)
