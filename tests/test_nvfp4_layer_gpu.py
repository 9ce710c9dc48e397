"""The NVFP4 products and the quantiser beside the framework's other ops: a
layer's run of them on one stream, eager and captured; host threads; debug builds
with bounds checks; a wait that runs out."""
import ctypes

import numpy as np
import pytest

import gen
import norm_activation_fp8_gb300 as vg
from norm_activation_fp8_gb300 import build
from test_nvfp4_gemm_gpu import check_gated, one, operand, product_error, scaled

pytestmark = pytest.mark.gpu

H, HQ, HKV, D, I, PAGE = 1024, 6, 1, 128, 1152, 16


class Layer:
    """norm -> qkv product -> QK norm, rotation, append -> (the rotated Q heads
    stand for the attention's output) -> quantiser -> output product -> residual
    norm -> gated projection -> down product, twice.  Every call reads what the
    one before it wrote."""

    def __init__(self, torch, T, seed=0):
        self.torch, self.T = torch, T
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.x0 = torch.randn((T, H), generator=g, device="cuda").bfloat16()
        self.res0 = torch.randn((T, H), generator=g, device="cuda").bfloat16()
        self.norm_w = torch.ones(H, device="cuda").bfloat16()
        self.head_w = torch.ones(D, device="cuda").bfloat16()
        self.gs = one(200.0)  # of every activation
        self.weights = {}
        for name, n, k in (("qkv", (HQ + 2 * HKV) * D, H), ("out", H, HQ * D), ("up", 2 * I, H), ("down", H, I)):
            w = (torch.randn((n, k), generator=g, device="cuda") / k ** 0.5).bfloat16()
            gs = (2688.0 / w.float().abs().max()).view(1)
            self.weights[name] = *vg.nvfp4_quantize(w, gs), 1 / (gs * self.gs)
        self.table = torch.from_numpy(gen.rope_cache(256, D)).cuda()
        self.positions = torch.arange(T, device="cuda") % 256
        pages = T // PAGE + 1
        self.slots = torch.randperm(pages * PAGE, generator=g, device="cuda")[:T]
        e = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
        codes = lambda n: (e(T, n // 2, dtype=torch.uint8), e(T, n // 16, dtype=torch.float8_e4m3fn))  # noqa: E731
        self.x, self.res, self.o, self.qkv = e(T, H), e(T, H), e(T, H), e(T, (HQ + 2 * HKV) * D)
        self.h4, self.a4, self.g4 = codes(H), codes(HQ * D), codes(I)
        self.k_cache, self.v_cache = e(pages, PAGE, HKV, D), e(pages, PAGE, HKV, D)

    def run(self, after=lambda: None):
        W, gs = self.weights, self.gs
        self.x.copy_(self.x0)
        self.res.copy_(self.res0)
        for _ in range(2):
            vg.vg_fused_add_rms_norm_nvfp4(*self.h4, self.res, self.x, self.res, self.norm_w, gs, 1e-5)
            after()
            vg.vg_nvfp4_gemm(self.qkv, *self.h4, *W["qkv"])
            after()
            vg.vg_fused_qk_norm_rope_append(self.qkv, self.k_cache, self.v_cache, self.head_w, self.head_w,
                                            self.table, self.positions, self.slots, HQ, HKV, D, 1e-6)
            after()
            vg.vg_nvfp4_quantize(*self.a4, self.qkv[:, :HQ * D], gs)
            after()
            vg.vg_nvfp4_gemm(self.o, *self.a4, *W["out"])
            after()
            vg.vg_fused_add_rms_norm_nvfp4(*self.h4, self.res, self.o, self.res, self.norm_w, gs, 1e-5)
            after()
            vg.vg_nvfp4_gemm_silu_mul_nvfp4(*self.g4, *self.h4, *W["up"], gs)
            after()
            vg.vg_nvfp4_gemm(self.x, *self.g4, *W["down"])
            after()

    def outputs(self):
        self.torch.cuda.synchronize()
        u8 = self.torch.uint8
        return [t.clone() for t in (self.x, self.res, self.o, self.qkv, self.k_cache, self.v_cache, self.g4[0],
                                    self.g4[1].view(u8), self.a4[0], self.a4[1].view(u8))]


def same(torch, a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T", [1, 37, 100, 300, 1500])
def test_layer_eager_and_captured_equal_the_synchronised_calls(T):
    import torch
    layers = [Layer(torch, T, seed) for seed in range(2)]
    want = []
    for x in layers:
        x.run(torch.cuda.synchronize)
        want.append(x.outputs())
        assert bool(torch.isfinite(x.x).all()) and float(x.x.float().abs().max()) > 0
        # what the last two products read is there: they are right
        w4, ws, alpha = x.weights["up"]
        A, Wt = scaled(*x.h4), scaled(w4, ws) * alpha.double()
        c, e = A @ Wt.t(), product_error(A, Wt, H)
        check_gated(*x.g4, c[:, :I], c[:, I:], e[:, :I], e[:, I:], 200.0)
        w4, ws, alpha = x.weights["down"]
        A, Wt = scaled(*x.g4), scaled(w4, ws) * alpha.double()
        c, e = A @ Wt.t(), product_error(A, Wt, I)
        assert bool(((x.x.double() - c).abs() <= e + 2.0 ** -8 * (c.abs() + e)).all())
    for x, w in zip(layers, want):  # no synchronisation between the calls, another stream
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            x.run()
        assert same(torch, x.outputs(), w)
    graphs = []
    for x in layers:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            x.run()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(3):  # two graphs, one after the other and at once on two streams
        for g in graphs:
            g.replay()
        for x, w in zip(layers, want):
            assert same(torch, x.outputs(), w)
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        for x, w in zip(layers, want):
            assert same(torch, x.outputs(), w)
    assert vg.vg_device_status() == 0


def test_arguments_on_the_gpu():
    """Refusals that need a CUDA tensor, and an explicit stream."""
    import torch
    f8 = torch.float8_e4m3fn
    a, sa = operand(4, 512, 1)
    w, sw = operand(128, 256, 2)
    al, a2, sa2 = one(1.0), a[:, :128].contiguous(), sa[:, :16].contiguous()
    with pytest.raises(ValueError, match="contiguous"):
        vg.nvfp4_gemm(a[:, :128], sa2, w, sw, al)
    with pytest.raises(ValueError, match="columns"):
        vg.nvfp4_gemm(a, sa, w, sw, al)
    with pytest.raises(ValueError, match="w_scale"):
        vg.nvfp4_gemm(a2, sa2, w, sw[:64], al)
    with pytest.raises(TypeError, match="w_scale"):
        vg.nvfp4_gemm(a2, sa2, w, sw.float(), al)
    with pytest.raises(TypeError, match="a:"):
        vg.nvfp4_gemm(a2.view(f8), sa2, w, sw, al)
    with pytest.raises(TypeError, match="alpha"):
        vg.nvfp4_gemm(a2, sa2, w, sw, al.double())
    with pytest.raises(ValueError, match="alpha"):
        vg.nvfp4_gemm(a2, sa2, w, sw, 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        vg.nvfp4_gemm(a2, sa2, w, sw.cpu(), al)
    with pytest.raises(TypeError, match="out"):
        vg.vg_nvfp4_gemm(torch.zeros((4, 128), device="cuda"), a2, sa2, w, sw, al)
    with pytest.raises(ValueError, match="out"):
        vg.vg_nvfp4_gemm(torch.zeros((4, 64), device="cuda").bfloat16(), a2, sa2, w, sw, al)
    with pytest.raises(vg.VgError, match="BAD_SHAPE"):
        vg.nvfp4_gemm(a2, sa2, w[:12], sw[:12], al)
    with pytest.raises(vg.VgError, match="BAD_SHAPE"):
        vg.nvfp4_gemm(*operand(4, 96, 1), *operand(8, 96, 2), al)  # K no multiple of 64
    with pytest.raises(ValueError, match="both or neither"):
        vg.vg_nvfp4_gemm_silu_mul_nvfp4(None, sa, a2, sa2, w, sw, al, al)
    with pytest.raises(ValueError, match="q4"):
        vg.vg_nvfp4_gemm_silu_mul_nvfp4(a, sa, a2, sa2, w, sw, al, al)
    with pytest.raises(ValueError, match="global_scale"):
        vg.nvfp4_gemm_silu_mul_nvfp4(a2, sa2, w, sw, al, torch.ones(2, device="cuda"))
    with pytest.raises(vg.VgError, match="BAD_SHAPE"):
        vg.nvfp4_gemm_silu_mul_nvfp4(a2, sa2, w[:96], sw[:96], al, al)  # an inter of 48
    want = vg.nvfp4_gemm(a2, sa2, w, sw, al)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = vg.nvfp4_gemm(a2, sa2, w, sw, al, stream=st)
    q4, sf = vg.nvfp4_gemm_silu_mul_nvfp4(a2, sa2, w, sw, al, al, stream=st)
    x = vg.nvfp4_dequantize(q4, sf, al, stream=st)
    r4, rf = vg.nvfp4_quantize(x, al, stream=st)
    st.synchronize()
    assert torch.equal(out, want)
    assert torch.equal(vg.nvfp4_dequantize(r4, rf, al), vg.nvfp4_dequantize(*vg.nvfp4_quantize(x, al), al))


def test_no_tokens():
    import torch
    a, sa = torch.zeros((0, 128), dtype=torch.uint8, device="cuda"), torch.zeros((0, 16), device="cuda").to(torch.float8_e4m3fn)
    w, sw = operand(128, 256, 2)
    assert vg.nvfp4_gemm(a, sa, w, sw, one(1.0)).shape == (0, 128)
    q4, sf = vg.nvfp4_gemm_silu_mul_nvfp4(a, sa, w, sw, one(1.0), one(1.0))
    assert q4.shape == (0, 32) and sf.shape == (0, 4)


FIRST_CALL = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
import norm_activation_fp8_gb300 as vg
from test_nvfp4_gemm_gpu import operand, scaled, one
sets = [(*operand(T, K, 1, exact=True), *operand(N, K, 2, exact=True)) for T, N, K in
        ((1, 1024, 512), (50, 640, 512), (460, 1432, 13440), (600, 8192, 512))]
outs = [torch.zeros((s[0].shape[0], s[2].shape[0]), dtype=torch.bfloat16, device="cuda") for s in sets]
al, x = one(1.0), torch.randn((9, 64), device="cuda").bfloat16()
q4, sf = torch.zeros((9, 32), dtype=torch.uint8, device="cuda"), torch.zeros((9, 4), dtype=torch.uint8, device="cuda")
back = torch.zeros_like(x)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for o, s in zip(outs, sets):
        vg.vg_nvfp4_gemm(o, *s, al)
    vg.vg_nvfp4_quantize(q4, sf.view(torch.float8_e4m3fn), x, al)
    vg.vg_nvfp4_dequantize(back, q4, sf.view(torch.float8_e4m3fn), al)
g.replay()
torch.cuda.synchronize()
for o, s in zip(outs, sets):
    assert torch.equal(o, (scaled(*s[:2]) @ scaled(*s[2:]).t()).to(torch.bfloat16))
assert (back - x).abs().max() < 1 and back.any()
print("captured first calls ok")
"""


def test_first_calls_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", FIRST_CALL.format(root=root)], capture_output=True, text=True,
                       cwd=root, timeout=300)
    assert p.returncode == 0 and "captured first calls ok" in p.stdout, p.stdout + p.stderr


def test_threads_that_call_at_once():
    """Host threads, each with its first call of CUDA here, on streams of their own."""
    import threading
    import torch
    sets = [(*operand(T, 1024, T, exact=True), *operand(1024, 1024, T + 1, exact=True), one(0.5))
            for T in (1, 20, 60, 200, 300, 700)]
    want = [(0.5 * scaled(*s[:2]) @ scaled(*s[2:4]).t()).to(torch.bfloat16) for s in sets]
    gated = [vg.nvfp4_gemm_silu_mul_nvfp4(*s[:4], one(1e-2), one(10.0))[0] for s in sets]
    streams, small, ten = [torch.cuda.Stream() for _ in sets], one(1e-2), one(10.0)
    torch.cuda.synchronize()
    done = []

    def work(i):
        outs = [vg.nvfp4_gemm(*sets[i], stream=streams[i]) for _ in range(30)]
        q4s = [vg.nvfp4_gemm_silu_mul_nvfp4(*sets[i][:4], small, ten, stream=streams[i])[0] for _ in range(10)]
        streams[i].synchronize()
        if all(torch.equal(o, want[i]) for o in outs) and all(torch.equal(q, gated[i]) for q in q4s):
            done.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert sorted(done) == list(range(len(sets)))


def _gemm(T, N, K):
    import torch
    x = (*operand(T, K, T), *operand(N, K, N), one(1e-3))
    return lambda: {"out": vg.nvfp4_gemm(*x).view(torch.int16).cpu().numpy()}


def _gated(T, n, K):
    import torch
    x = (*operand(T, K, T), *operand(2 * n, K, n), one(1e-5), one(100.0))

    def run():
        q4, sf = vg.nvfp4_gemm_silu_mul_nvfp4(*x)
        return {"q": q4.cpu().numpy(), "scale": sf.view(torch.uint8).cpu().numpy()}
    return run


def _quantize(T, n, pitch):
    import torch
    x = torch.randn((T, pitch), device="cuda", generator=torch.Generator(device="cuda").manual_seed(T)).bfloat16()[:, :n]

    def run():
        q4, sf = vg.nvfp4_quantize(x, one(100.0))
        return {"q": q4.cpu().numpy(), "scale": sf.view(torch.uint8).cpu().numpy()}
    return run


def _back(T, n):
    import torch
    x = (*operand(T, n, T), one(3.0))
    return lambda: {"out": vg.nvfp4_dequantize(*x).view(torch.int16).cpu().numpy()}


# every kernel form: stream tiles of 16 to 128 tokens, split and not; the tile
# kernel, split and not, rows of whole and of broken groups of scales
CASES = {
    "gemm-1": lambda: _gemm(1, 1032, 1024), "gemm-20": lambda: _gemm(20, 96, 192),
    "gemm-50": lambda: _gemm(50, 2056, 512), "gemm-70": lambda: _gemm(70, 3800, 6912),
    "gemm-460-tile-split": lambda: _gemm(460, 1432, 13440), "gemm-700-tile": lambda: _gemm(700, 8200, 512),
    "gemm-700-tile-odd": lambda: _gemm(700, 8200, 576), "gated-1": lambda: _gated(1, 256, 1024),
    "gated-40": lambda: _gated(40, 1152, 512), "gated-604-tile-split": lambda: _gated(604, 960, 6592),
    "gated-700-tile": lambda: _gated(700, 4032, 512), "quantize-9": lambda: _quantize(9, 4112, 4112),
    "quantize-700-apart": lambda: _quantize(700, 4112, 4136), "quantize-1000": lambda: _quantize(1000, 16384, 16384),
    "back-9": lambda: _back(9, 4112), "back-700": lambda: _back(700, 4112),
}


def _with(lib, run, monkeypatch):
    with monkeypatch.context() as m:
        m.setattr(vg, "_lib", lib)
        vg.vg_device_status(reset=True)
        return run(), vg.vg_device_status(reset=True)


@pytest.mark.parametrize("case", sorted(CASES))
def test_debug_build_matches_and_reports_nothing(case, monkeypatch):
    run = CASES[case]()
    want, st0 = _with(vg.load(), run, monkeypatch)
    got, st = _with(vg.load(build.build_debug()), run, monkeypatch)
    assert st0 == 0 and st == 0, (st0, st)
    for k, v in want.items():
        assert np.array_equal(got[k], v), k


@pytest.mark.parametrize("case", sorted(CASES))
def test_out_of_range_accesses_are_flagged_and_skipped(case, monkeypatch):
    """With every tensor of tokens reported one row short: the last token's scale
    reads and the stores of its row are flagged, the other rows stay."""
    run = CASES[case]()
    want, _ = _with(vg.load(), run, monkeypatch)
    got, st = _with(vg.load(build.build_debug(shrunk=True)), run, monkeypatch)
    assert st == vg.DEVICE_OUT_OF_BOUNDS, st
    for k, v in want.items():
        assert np.array_equal(got[k][:-1], v[:-1]), k


@pytest.mark.parametrize("T,N,K", [(1, 1024, 1024), (460, 1536, 13440), (600, 8192, 512)],
                         ids=["stream", "tile-split", "tile"])
def test_forced_wait_timeout_is_reported_and_context_survives(T, N, K):
    """The test copy's product warps also wait on a barrier that nothing arrives
    on: the wait gives up, every other wait runs out after it, the status says
    so, and the product library runs the same call right after."""
    import torch
    lib = vg.load(build.build_wait_test())

    def status(reset):
        flags = ctypes.c_uint32(0)
        assert lib.vg_device_status(ctypes.byref(flags), reset) == 0
        return flags.value

    a, sa = operand(T, K, 1, exact=True)
    w, sw = operand(N, K, 2, exact=True)
    out, al = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda"), one(1.0)
    status(1)
    ptrs = [x.data_ptr() for x in (a, sa, w, sw, al)]
    assert lib.vg_nvfp4_gemm(out.data_ptr(), *ptrs, T, N, K, None) == 0
    torch.cuda.synchronize()
    assert status(1) & vg.DEVICE_WAIT_TIMEOUT
    assert status(0) == 0
    q4, sf = torch.zeros((T, N // 4), dtype=torch.uint8, device="cuda"), torch.zeros((T, N // 32), dtype=torch.uint8, device="cuda")
    assert lib.vg_nvfp4_gemm_silu_mul_nvfp4(q4.data_ptr(), sf.data_ptr(), *ptrs, al.data_ptr(), T, N // 2, K, None) == 0
    torch.cuda.synchronize()
    assert status(1) & vg.DEVICE_WAIT_TIMEOUT
    vg.vg_device_status(reset=True)
    assert torch.equal(vg.nvfp4_gemm(a, sa, w, sw, al), (scaled(a, sa) @ scaled(w, sw).t()).to(torch.bfloat16))
    assert vg.vg_device_status() == 0
