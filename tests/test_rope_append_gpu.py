"""QK norm + rotation with several position axes, and on the way into a paged
cache: the CUDA path against fp64.

The rotation of one token only reads that token's cos/sin values, so a
multi-axis rotation equals the one-axis op on a table whose row t holds the
values token t takes from its axes; the oracle runs on that table.  Tolerances
are the one-axis op's: a bf16 value is the correctly rounded one, or one ulp
from it within 2^-19 of a midpoint.  An FP8 cache follows the code rule (the
kernel's fp32 value and its reciprocal scale are within 2^-19 of the exact
quotient; a code may differ by one where the quotient is that near a
midpoint).  A rotation without a norm is compared with fp64 numpy."""
import numpy as np
import pytest

import gen
import oracle
import parity
import norm_activation_fp8_gb300 as vg

pytestmark = pytest.mark.gpu

EPS = 1e-6
MAXP = 2048


def axis_of_pair(half, sections, interleaved):
    """The definition, pair by pair."""
    if not interleaved:
        return np.repeat(np.arange(len(sections)), sections)
    n = len(sections)
    return np.array([i % n if i // n < sections[i % n] else 0 for i in range(half)])


def inputs(T, hq, hkv, D, sections=None, interleaved=False, seed=0):
    d = gen.qk_inputs(T, hq, hkv, D, MAXP, seed=seed)
    rng = np.random.default_rng(seed + 77)
    if sections is None:
        d["token_table"] = d["cos_sin_cache"][d["positions"]]
        return d
    d["positions"] = rng.integers(0, MAXP, (len(sections), T)).astype(np.int64)
    axis = axis_of_pair(D // 2, sections, interleaved)
    i = np.arange(D // 2)
    rows = d["positions"][axis].T  # [T, D/2]
    d["token_table"] = np.concatenate([d["cos_sin_cache"][rows, i], d["cos_sin_cache"][rows, D // 2 + i]], 1)
    return d


def turned(d, hq, hkv, D, neox, norm):
    """(qkv after an in-place turn, the fp64 values of the Q and K heads)."""
    T = d["qkv"].shape[0]
    if norm:
        e = dict(d, cos_sin_cache=d["token_table"], positions=np.arange(T))
        return parity.oracle_qk(e, hq, hkv, D, EPS, neox)
    x = oracle.bf16_decode(d["qkv"][:, :(hq + hkv) * D]).astype(np.float64).reshape(T, hq + hkv, D)
    c = d["token_table"][:, None, :D // 2].astype(np.float64)
    s = d["token_table"][:, None, D // 2:].astype(np.float64)
    a, b = (np.s_[..., :D // 2], np.s_[..., D // 2:]) if neox else (np.s_[..., 0::2], np.s_[..., 1::2])
    o = np.empty_like(x)
    o[a] = x[a] * c - x[b] * s
    o[b] = x[b] * c + x[a] * s
    o = o.reshape(T, -1)
    out = d["qkv"].copy()
    out[:, :o.shape[1]] = oracle.bf16_encode(o)
    return out, o


def cuda(a):
    import torch
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


SECTIONS = {64: (12, 10, 10), 128: (24, 20, 20), 256: (56, 36, 36)}


@pytest.mark.parametrize("neox", [True, False], ids=["neox", "gptj"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["runs", "turns"])
@pytest.mark.parametrize("T,hq,hkv,D,sections", [
    (1, 32, 8, 128, None), (7, 4, 2, 64, None), (333, 32, 8, 128, None), (65, 8, 1, 256, None),
    (33, 5, 0, 128, None), (17, 0, 3, 64, None), (9, 150, 5, 64, None),
    (50, 4, 2, 128, (40, 24)), (50, 4, 2, 128, (28, 12, 12, 12)), (50, 4, 2, 128, (64,)),
    (50, 4, 2, 128, (64, 0, 0)), (50, 4, 2, 64, (11, 11, 10)),
    # many tokens: three heads a lane group, the last groups with fewer or none
    (640, 32, 8, 128, None), (611, 28, 4, 128, (28, 12, 12, 12)), (700, 1, 1, 64, None),
    (613, 23, 2, 64, None), (609, 7, 1, 256, None), (650, 0, 5, 128, (64,)), (620, 70, 3, 256, None),
])
def test_mrope(T, hq, hkv, D, sections, interleaved, neox):
    sections = sections or SECTIONS[D]
    d = inputs(T, hq, hkv, D, sections, interleaved, seed=T + D)
    for norm in (True, False):
        qkv = cuda(d["qkv"]).clone()
        w = (cuda(d["q_weight"]), cuda(d["k_weight"])) if norm else (None, None)
        vg.vg_fused_qk_norm_mrope(qkv, *w, cuda(d["cos_sin_cache"]), cuda(d["positions"]), sections,
                                  hq, hkv, D, EPS, neox, interleaved)
        g = qkv.cpu().numpy().view(np.uint16)
        parity.check_qk(g, turned(d, hq, hkv, D, neox, norm), d["qkv"], hq, hkv, D)
    assert vg.vg_device_status() == 0


def test_one_axis_sections_equal_the_plain_op():
    """All pairs on one axis: the bits of vg_fused_qk_norm_rope."""
    d = inputs(100, 8, 2, 128, (64, 0, 0), seed=5)
    want = cuda(d["qkv"]).clone()
    tail = (8, 2, 128, EPS)
    w = cuda(d["q_weight"]), cuda(d["k_weight"]), cuda(d["cos_sin_cache"])
    vg.vg_fused_qk_norm_rope(want, *w, cuda(np.ascontiguousarray(d["positions"][0])), *tail)
    got = cuda(d["qkv"]).clone()
    vg.vg_fused_qk_norm_mrope(got, *w, cuda(d["positions"]), (64, 0, 0), *tail)
    assert bool((want == got).all())


def test_mrope_bad_position_on_any_axis():
    T, hq, hkv, D = 8, 4, 2, 128
    d = inputs(T, hq, hkv, D, (24, 20, 20), seed=6)
    bad = d["positions"].copy()
    bad[0, 1], bad[1, 3], bad[2, 6] = MAXP, -1, 2 ** 40
    vg.vg_device_status(reset=True)
    qkv = cuda(d["qkv"]).clone()
    vg.vg_fused_qk_norm_mrope(qkv, cuda(d["q_weight"]), cuda(d["k_weight"]), cuda(d["cos_sin_cache"]),
                              cuda(bad), (24, 20, 20), hq, hkv, D, EPS)
    assert vg.vg_device_status(reset=True) == vg.DEVICE_BAD_POSITION
    g = qkv.cpu().numpy().view(np.uint16)
    good = np.ones(T, bool)
    good[[1, 3, 6]] = False
    assert np.array_equal(g[~good], d["qkv"][~good])
    out, o = turned(d, hq, hkv, D, True, True)
    parity.check_qk(g[good], (out[good], o[good]), d["qkv"][good], hq, hkv, D)


def paged(layout, pages, page, hkv, D, dtype):
    """k_cache, v_cache [pages, page, hkv, D] filled with a pattern, in one of
    three memory orders."""
    import torch
    n = torch.arange(2 * pages * page * hkv * D, device="cuda", dtype=torch.int64)
    raw = (n % 113).to(torch.uint8 if dtype == torch.uint8 else torch.int16)
    if layout == "heads":       # [2, pages, page, heads, D]
        k, v = raw.view(2, pages, page, hkv, D)
    elif layout == "tokens":    # [2, pages, heads, page, D]: pages in head-major order
        k, v = raw.view(2, pages, hkv, page, D).transpose(2, 3)
    else:                       # [pages, 2, page, heads, D]: K and V of a page together
        x = raw.view(pages, 2, page, hkv, D)
        k, v = x[:, 0], x[:, 1]
    return k, v


def run_append(d, T, hq, hkv, D, fp8, norm, neox, sections, interleaved, layout, page, slots, pages):
    import torch
    k, v = paged(layout, pages, page, hkv, D, torch.uint8 if fp8 else torch.int16)
    before = k.cpu().numpy().copy(), v.cpu().numpy().copy()
    qkv = cuda(d["qkv"]).clone()
    w = (cuda(d["q_weight"]), cuda(d["k_weight"])) if norm else (None, None)
    scales = [torch.tensor([x], device="cuda") for x in (0.02, 0.015)] if fp8 else [None, None]
    vg.vg_fused_qk_norm_rope_append(qkv, k, v, *w, cuda(d["cos_sin_cache"]), cuda(d["positions"]),
                                    cuda(slots), hq, hkv, D, EPS, neox, sections, interleaved, *scales)
    return qkv.cpu().numpy().view(np.uint16), before, (k.cpu().numpy(), v.cpu().numpy())


def check_append(d, got, slots, T, hq, hkv, D, fp8, norm, neox, page):
    g, before, after = got
    out, o = turned(d, hq, hkv, D, neox, norm)
    nq = hq * D
    if hq:
        parity.compare_bf16(g[:, :nq], out[:, :nq], o[:, :nq], "q heads")
    assert np.array_equal(g[:, nq:], d["qkv"][:, nq:])  # K and V of the row itself stay
    live = slots >= 0
    at = slots[live] // page, slots[live] % page
    k, v = (x[at].reshape(int(live.sum()), hkv * D) for x in after)
    ko = o[live][:, nq:]
    vbits = d["qkv"][live][:, (hq + hkv) * D:]
    if fp8:
        for codes, value, s in ((k, ko, 0.02), (v, oracle.bf16_decode(vbits).astype(np.float64), 0.015)):
            q = value / float(np.float32(s))
            parity.compare_codes(codes, oracle.e4m3_encode(q).reshape(q.shape), q, "cache")
    else:
        parity.compare_bf16(k.view(np.uint16), out[live][:, nq:(hq + hkv) * D], ko, "k cache")
        assert np.array_equal(v.view(np.uint16), vbits)
    for x, y in zip(before, after):  # every other slot as it was
        x[at] = y[at]
        assert np.array_equal(x, y)


@pytest.mark.parametrize("layout", ["heads", "tokens", "together"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("T,hq,hkv,D,page,axes,norm,neox", [
    (1, 32, 8, 128, 16, 1, True, True),
    (1, 4, 1, 64, 1, 3, False, True),
    (7, 8, 1, 256, 96, 1, False, False),
    (333, 32, 8, 128, 16, 1, True, True),
    (333, 28, 4, 128, 16, 3, True, True),
    (130, 5, 3, 64, 1, 1, True, False),
    (77, 0, 2, 128, 64, 1, True, True),
    (601, 64, 8, 128, 128, 1, False, True),
    # many tokens: three heads a lane group, Q, K and V in one warp
    (640, 32, 8, 128, 16, 1, True, True), (611, 5, 1, 64, 1, 3, True, False),
    (700, 64, 8, 128, 64, 1, False, True), (609, 3, 2, 256, 96, 3, True, True),
    (650, 0, 5, 128, 16, 1, False, True), (1201, 28, 4, 128, 128, 3, True, True),
])
def test_append(T, hq, hkv, D, page, axes, norm, neox, fp8, layout):
    sections = SECTIONS[D] if axes == 3 else None
    d = inputs(T, hq, hkv, D, sections, False, seed=T + hq + page)
    rng = np.random.default_rng(T)
    pages = T // page + 3
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    if T > 4:
        slots[::5] = -1
        slots[2] = -2 ** 40
    got = run_append(d, T, hq, hkv, D, fp8, norm, neox, sections, False, layout, page, slots, pages)
    check_append(d, got, slots, T, hq, hkv, D, fp8, norm, neox, page)
    assert vg.vg_device_status() == 0


def test_append_bad_slots_and_positions():
    """A slot past the cache or a bad position: reported, nothing appended; a
    bad slot's Q is still turned, a bad position's token stays."""
    T, hq, hkv, D, page, pages = 12, 4, 2, 128, 8, 3
    d = inputs(T, hq, hkv, D, seed=9)
    slots = np.arange(T, dtype=np.int64)
    slots[3], slots[5] = pages * page, 2 ** 62
    d["positions"][7] = MAXP
    vg.vg_device_status(reset=True)
    got = run_append(d, T, hq, hkv, D, False, True, True, None, False, "heads", page, slots, pages)
    assert vg.vg_device_status(reset=True) == vg.DEVICE_BAD_SLOT | vg.DEVICE_BAD_POSITION
    g, before, after = got
    assert np.array_equal(g[7], d["qkv"][7])
    keep = np.arange(T) != 7
    e = {k: (v[keep] if k in ("qkv", "positions", "token_table") else v) for k, v in d.items()}
    s = slots[keep].copy()
    s[s >= pages * page] = -1
    check_append(e, (g[keep], before, after), s, T - 1, hq, hkv, D, False, True, True, page)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_append_offsets_past_32_bits(fp8):
    """Slots whose element offset passes 2^32 (a cache of 9 or 4.5 GB each)."""
    import torch
    T, hq, hkv, D, page = 40, 2, 8, 128, 64
    pages = 70000
    d = inputs(T, hq, hkv, D, seed=3)
    k, v = (torch.zeros((pages, page, hkv, D), dtype=torch.uint8 if fp8 else torch.int16, device="cuda")
            for _ in range(2))
    slots = np.arange(T, dtype=np.int64)
    slots[20:] = pages * page - 1 - slots[20:]
    assert int(slots[20]) * hkv * D > 2 ** 32
    qkv = cuda(d["qkv"]).clone()
    scales = [torch.ones(1, device="cuda")] * 2 if fp8 else [None, None]
    vg.vg_fused_qk_norm_rope_append(qkv, k, v, cuda(d["q_weight"]), cuda(d["k_weight"]),
                                    cuda(d["cos_sin_cache"]), cuda(d["positions"]), cuda(slots), hq,
                                    hkv, D, EPS, True, None, False, *scales)
    vbits = d["qkv"][:, (hq + hkv) * D:]
    rows = v.view(-1, hkv * D)[torch.from_numpy(slots).cuda()].cpu().numpy()
    if fp8:
        q = oracle.bf16_decode(vbits).astype(np.float64)
        parity.compare_codes(rows, oracle.e4m3_encode(q).reshape(q.shape), q, "v cache")
    else:
        assert np.array_equal(rows.view(np.uint16), vbits)
    for x in (k, v):
        assert int((x.view(-1, hkv * D) != 0).any(1).sum()) == T


def test_append_captured_and_replayed():
    """A captured append takes each replay's slots and positions."""
    import torch
    T, hq, hkv, D, page, pages = 6, 8, 2, 128, 16, 8
    d = inputs(T, hq, hkv, D, seed=4)
    k, v = paged("heads", pages, page, hkv, D, torch.int16)
    args = [cuda(d[n]) for n in ("q_weight", "k_weight", "cos_sin_cache")]
    src, pos = cuda(d["qkv"]), cuda(d["positions"]).clone()
    qkv, slots = src.clone(), torch.zeros(T, dtype=torch.int64, device="cuda")

    def step():
        qkv.copy_(src)
        vg.vg_fused_qk_norm_rope_append(qkv, k, v, *args, pos, slots, hq, hkv, D, EPS)

    slots.copy_(torch.arange(T))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for shift in (20, 61):
        before = k.cpu().numpy().copy(), v.cpu().numpy().copy()
        slots.copy_(torch.arange(T) + shift)
        pos.copy_((cuda(d["positions"]) + shift) % MAXP)
        e = dict(d, positions=(d["positions"] + shift) % MAXP)
        e["token_table"] = e["cos_sin_cache"][e["positions"]]
        graph.replay()
        got = qkv.cpu().numpy().view(np.uint16), before, (k.cpu().numpy(), v.cpu().numpy())
        check_append(e, got, np.arange(T) + shift, T, hq, hkv, D, False, True, True, page)


def with_infinities(d, hq, hkv, D, seed):
    """d with infinities of either sign in Q, K and V heads, alone in a pair and
    on both sides of it, some at position 0, whose sines are zero."""
    rng = np.random.default_rng(seed)
    T, heads = d["qkv"].shape[0], hq + 2 * hkv
    x = d["qkv"].copy().reshape(T, heads, D)
    for n in range(6 * heads):
        t, h, i = rng.integers(T), n % heads, rng.integers(D // 2)
        kind = n // heads % 3  # one side of a neox pair, of a gptj pair, both sides of both
        at = ((i, i), (2 * i, 2 * i), (i, i + D // 2, i ^ 1))[kind]
        x[t, h, list(at)] = np.where(rng.random(len(at)) < 0.5, 0x7F80, 0xFF80)
    d["qkv"] = x.reshape(T, -1)
    d["positions"][::3] = 0
    d["token_table"] = d["cos_sin_cache"][d["positions"]]
    return d


def near_codes(codes, q):
    """Every code is q's, or its neighbour where q lies within 2^-19 of their
    midpoint: the rotation is off by at most 2 ulps (2^-22), the reciprocal and
    the product by half an ulp each (2^-24).  No cap on the neighbours' number:
    at position 0 K passes unchanged, and bf16 values as common as 0.5 lie at
    0.5 / fp32(0.02) = 25 (1 + 2.2e-8), beside the midpoint of 24 and 26."""
    want = oracle.e4m3_encode(q).reshape(q.shape)
    at = codes != want
    a, b, v = codes[at], want[at], np.abs(q[at])
    assert ((a & 0x80) == (b & 0x80)).all() and (np.abs((a & 0x7F).astype(int) - (b & 0x7F)) == 1).all()
    mid = (np.abs(oracle.e4m3_decode(a).astype(np.float64)) + np.abs(oracle.e4m3_decode(b))) / 2
    assert (np.abs(v - mid) <= 2.0 ** -19 * mid).all()


@pytest.mark.parametrize("neox", [True, False], ids=["neox", "gptj"])
@pytest.mark.parametrize("T,hq,hkv,D", [(40, 4, 2, 128), (170, 3, 1, 64), (700, 5, 2, 128), (650, 2, 1, 256)])
def test_infinities_without_a_norm_follow_the_formula(T, hq, hkv, D, neox):
    """x = inf: a c - b s is that infinity, NaN only where IEEE arithmetic says
    so (inf - inf, inf * 0), and an FP8 cache saturates it as it does V's."""
    d = with_infinities(inputs(T, hq, hkv, D, seed=T), hq, hkv, D, T)
    with np.errstate(invalid="ignore"):
        out, o = turned(d, hq, hkv, D, neox, False)
    assert np.isinf(o).any() and np.isnan(o).any()

    def check(bits, want, exact, what):
        v = oracle.bf16_decode(bits).astype(np.float64)
        assert np.array_equal(np.isnan(v), np.isnan(exact)), what
        inf = np.isinf(exact)
        assert np.array_equal(v[inf], exact[inf]), what
        ok = np.isfinite(exact)
        parity.compare_bf16(bits[ok], want[ok], exact[ok], what)

    qkv = cuda(d["qkv"]).clone()
    vg.vg_fused_qk_norm_mrope(qkv, None, None, cuda(d["cos_sin_cache"]), cuda(d["positions"][None]), (D // 2,),
                              hq, hkv, D, EPS, neox)
    g = qkv.cpu().numpy().view(np.uint16)
    n = (hq + hkv) * D
    check(g[:, :n], out[:, :n], o, "in place")
    assert np.array_equal(g[:, n:], d["qkv"][:, n:])
    slots = np.arange(T, dtype=np.int64)
    for fp8 in (False, True):
        g, _, (k, v) = run_append(d, T, hq, hkv, D, fp8, False, neox, None, False, "heads", 16, slots, T // 16 + 1)
        k, v = (x.reshape(-1, hkv * D)[:T] for x in (k, v))
        check(g[:, :hq * D], out[:, :hq * D], o[:, :hq * D], "q heads")
        ko, vbits = o[:, hq * D:], d["qkv"][:, n:]
        if not fp8:
            check(k.view(np.uint16), out[:, hq * D:n], ko, "k cache")
            assert np.array_equal(v.view(np.uint16), vbits)
            continue
        for codes, value, s in ((k, ko, 0.02), (v, oracle.bf16_decode(vbits).astype(np.float64), 0.015)):
            assert np.array_equal(codes & 0x7F == 0x7F, np.isnan(value))
            assert (codes[value == np.inf] == 0x7E).all() and (codes[value == -np.inf] == 0xFE).all()
            ok = np.isfinite(value)
            near_codes(codes[ok], value[ok] / float(np.float32(s)))
    assert vg.vg_device_status() == 0


@pytest.mark.parametrize("neox", [True, False], ids=["neox", "gptj"])
@pytest.mark.parametrize("T", [30, 640])
def test_infinities_under_a_norm(T, neox):
    """x = inf makes its head's mean square infinite and 1 / rms zero: NaN in
    the pairs that hold it, zeros beside them, other heads as they are."""
    hq, hkv, D = 4, 2, 128
    clean = inputs(T, hq, hkv, D, seed=T)
    d = with_infinities(inputs(T, hq, hkv, D, seed=T), hq, hkv, D, T)
    x = oracle.bf16_decode(d["qkv"]).reshape(T, -1, D)[:, :hq + hkv]
    inf = np.isinf(x)
    pair = inf | (np.roll(inf, D // 2, -1) if neox else inf[..., np.arange(D) ^ 1])
    hit = inf.any(-1)
    clean["positions"] = d["positions"]
    qkv, ref = cuda(d["qkv"]).clone(), cuda(clean["qkv"]).clone()
    w = cuda(d["q_weight"]), cuda(d["k_weight"]), cuda(d["cos_sin_cache"])
    for q in (qkv, ref):
        vg.vg_fused_qk_norm_mrope(q, *w, cuda(d["positions"][None]), (D // 2,), hq, hkv, D, EPS, neox)
    plain = cuda(d["qkv"]).clone()
    vg.vg_fused_qk_norm_rope(plain, *w, cuda(d["positions"]), hq, hkv, D, EPS, neox)
    for out in (qkv, plain):
        v = oracle.bf16_decode(out.cpu().numpy().view(np.uint16)).reshape(T, -1, D)[:, :hq + hkv]
        r = oracle.bf16_decode(ref.cpu().numpy().view(np.uint16)).reshape(T, -1, D)[:, :hq + hkv]
        assert np.array_equal(np.isnan(v), pair)
        assert (v[hit[..., None] & ~pair] == 0).all()
        assert np.array_equal(v[~hit], r[~hit])
