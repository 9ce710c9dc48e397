"""The FP8 products and the rotary cache append beside the framework's other
ops: a layer's run of them on one stream, eager and captured; debug builds with
bounds checks; a wait that runs out."""
import ctypes

import numpy as np
import pytest

import gen
import norm_activation_fp8_gb300 as vg
from norm_activation_fp8_gb300 import build

pytestmark = pytest.mark.gpu

H, HQ, HKV, D, I, PAGE = 1024, 6, 1, 128, 1152, 16
COL = vg.COLUMN_MAJOR


class Layer:
    """norm -> qkv product -> QK norm, rotation, append -> (the rotated Q heads
    stand for the attention's output) -> norm -> output product -> residual
    norm -> gated projection -> down product, twice.  Every call reads what the
    one before it wrote."""

    def __init__(self, torch, T, options, seed=0):
        self.torch, self.T, self.options = torch, T, options
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.x0 = torch.randn((T, H), generator=g, device="cuda").bfloat16()
        self.res0 = torch.randn((T, H), generator=g, device="cuda").bfloat16()
        self.norm_w = torch.ones(H, device="cuda").bfloat16()
        self.attn_w = torch.ones(HQ * D, device="cuda").bfloat16()
        self.head_w = torch.ones(D, device="cuda").bfloat16()
        self.weights = {}
        for name, n, k in (("qkv", (HQ + 2 * HKV) * D, H), ("out", H, HQ * D), ("up", 2 * I, H), ("down", H, I)):
            w = (torch.randn((n, k), generator=g, device="cuda") * 100).clamp(-448, 448)
            s = torch.rand((n // 128, k // 128), generator=g, device="cuda") * 1e-3 / k ** 0.5 + 1e-5
            self.weights[name] = w.to(torch.float8_e4m3fn), s
        self.table = torch.from_numpy(gen.rope_cache(256, D)).cuda()
        self.positions = torch.arange(T, device="cuda") % 256
        pages = T // PAGE + 1
        self.slots = torch.randperm(pages * PAGE, generator=g, device="cuda")[:T]
        e = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
        f8, f32, t4 = torch.float8_e4m3fn, torch.float32, (T + 3) // 4 * 4
        sc = (lambda n: e(n // 128, t4, dtype=f32)) if options & COL else (lambda n: e(T, n // 128, dtype=f32))
        self.x, self.res = e(T, H), e(T, H)
        self.q8, self.s8 = e(T, H, dtype=f8), sc(H)
        self.qkv, self.attn = e(T, (HQ + 2 * HKV) * D), e(T, HQ * D)
        self.a8, self.as8 = e(T, HQ * D, dtype=f8), sc(HQ * D)
        self.o = e(T, H)
        self.g8, self.gs8 = e(T, I, dtype=f8), sc(I)
        self.k_cache, self.v_cache = e(pages, PAGE, HKV, D), e(pages, PAGE, HKV, D)

    def run(self, after=lambda: None):
        mode, col = vg.PER_GROUP | self.options, self.options & COL
        W = self.weights
        self.x.copy_(self.x0)
        self.res.copy_(self.res0)
        for _ in range(2):
            vg.vg_fused_add_rms_norm_fp8(self.q8, self.res, self.s8, self.x, self.res, self.norm_w, 1e-5, mode)
            after()
            vg.vg_fp8_block_gemm(self.qkv, self.q8, self.s8, *W["qkv"], col)
            after()
            vg.vg_fused_qk_norm_rope_append(self.qkv, self.k_cache, self.v_cache, self.head_w, self.head_w,
                                            self.table, self.positions, self.slots, HQ, HKV, D, 1e-6)
            after()
            self.attn.copy_(self.qkv[:, :HQ * D])
            vg.vg_fused_add_rms_norm_fp8(self.a8, None, self.as8, self.attn, None, self.attn_w, 1e-5, mode)
            after()
            vg.vg_fp8_block_gemm(self.o, self.a8, self.as8, *W["out"], col)
            after()
            vg.vg_fused_add_rms_norm_fp8(self.q8, self.res, self.s8, self.o, self.res, self.norm_w, 1e-5, mode)
            after()
            vg.vg_fp8_block_gemm_silu_mul_fp8(self.g8, self.gs8, self.q8, self.s8, *W["up"], col, self.options)
            after()
            vg.vg_fp8_block_gemm(self.x, self.g8, self.gs8, *W["down"], col)
            after()

    def outputs(self):
        self.torch.cuda.synchronize()
        return [t.clone() for t in (self.x, self.res, self.qkv, self.k_cache, self.v_cache,
                                    self.g8.view(self.torch.uint8))]


def same(torch, a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("options", [0, COL, COL | vg.UE8M0], ids=["rows", "columns", "ue8m0-columns"])
@pytest.mark.parametrize("T", [1, 37, 100, 300, 1500])
def test_layer_eager_and_captured_equal_the_synchronised_calls(T, options):
    import torch
    layers = [Layer(torch, T, options, seed) for seed in range(2)]
    want = []
    for x in layers:
        x.run(torch.cuda.synchronize)
        want.append(x.outputs())
        assert bool(torch.isfinite(x.x).all()) and float(x.x.float().abs().max()) > 0
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
    for _ in range(3):  # two graphs, one after the other and at once on two streams
        for g in graphs:
            g.replay()
        for x, w in zip(layers, want):
            assert same(torch, x.outputs(), w)
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    for x, w in zip(layers, want):
        assert same(torch, x.outputs(), w)
    assert vg.vg_device_status() == 0


def test_arguments_on_the_gpu():
    """Refusals that need a CUDA tensor: strided operands, wrong types, a cache
    whose K and V differ, an explicit stream."""
    import torch
    f8 = torch.float8_e4m3fn
    a = torch.zeros((4, 512), dtype=torch.uint8, device="cuda").view(f8)
    sa, w = torch.ones((4, 2), device="cuda"), torch.zeros((128, 256), dtype=f8, device="cuda")
    sw = torch.ones((1, 2), device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        vg.fp8_block_gemm(a[:, :256], sa, w, sw)
    with pytest.raises(TypeError, match="w_scale"):
        vg.fp8_block_gemm(a[:, :256].contiguous(), sa, w, sw.double())
    with pytest.raises(ValueError, match="both or neither"):
        vg.vg_fp8_block_gemm_silu_mul_fp8(None, sa, a[:, :256].contiguous(), sa, w, sw)
    with pytest.raises(ValueError, match="scale"):
        vg.vg_fp8_block_gemm_silu_mul_fp8(torch.zeros((4, 128), dtype=f8, device="cuda"), sa,
                                          a[:, :256].contiguous(), sa, torch.cat([w.view(torch.uint8)] * 2),
                                          torch.cat([sw] * 2))
    with pytest.raises(TypeError, match="out"):
        vg.vg_fp8_block_gemm(torch.zeros((4, 128), device="cuda"), a[:, :256].contiguous(), sa, w, sw)
    with pytest.raises(TypeError, match="a:"):
        vg.fp8_block_gemm(a[:, :256].float(), sa, w, sw)
    with pytest.raises(ValueError, match="2-D"):
        vg.fp8_block_gemm(a[0, :256], sa, w, sw)
    with pytest.raises(ValueError, match="out"):
        vg.vg_fp8_block_gemm(torch.zeros((4, 64), device="cuda").bfloat16(), a[:, :256].contiguous(), sa, w, sw)
    with pytest.raises(ValueError, match="CUDA"):
        vg.fp8_block_gemm(a[:, :256].contiguous(), sa, w, sw.cpu())
    st = torch.cuda.Stream()
    a2 = a[:, :256].contiguous()
    torch.cuda.synchronize()
    out = vg.fp8_block_gemm(a2, sa, w, sw, stream=st)
    st.synchronize()
    assert not out.any()
    qkv = torch.zeros((4, 4 * 64), device="cuda").bfloat16()
    table, pos = torch.zeros((16, 64), device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    slots = torch.arange(4, device="cuda")
    k = torch.zeros((2, 16, 1, 64), device="cuda").bfloat16()
    tail = (None, None, table, pos, slots, 2, 1, 64, 1e-6)
    with pytest.raises(ValueError, match="same shape and strides"):
        vg.vg_fused_qk_norm_rope_append(qkv, k, k[:1], *tail)
    with pytest.raises(TypeError, match="k_cache"):
        vg.vg_fused_qk_norm_rope_append(qkv, k.float(), k.float(), *tail)
    with pytest.raises(TypeError, match="k_cache"):
        vg.vg_fused_qk_norm_rope_append(qkv, k, k, *tail, k_scale=sa[0, :1], v_scale=sa[0, :1])
    with pytest.raises(vg.VgError, match="NULL"):
        vg.vg_fused_qk_norm_rope_append(qkv, k.view(torch.uint8)[..., :64].contiguous(),
                                        k.view(torch.uint8)[..., :64].contiguous(), *tail, k_scale=sa[0, :1])
    with pytest.raises(ValueError, match="slots"):
        vg.vg_fused_qk_norm_rope_append(qkv, k, k.clone(), None, None, table, pos, slots[:3], 2, 1, 64, 1e-6)


def test_no_tokens():
    """Every call with zero tokens returns and writes nothing."""
    import torch
    f8 = torch.float8_e4m3fn
    w, sw = torch.zeros((256, 256), dtype=f8, device="cuda"), torch.ones((2, 2), device="cuda")
    for col in (0, COL):
        a = torch.zeros((0, 256), dtype=f8, device="cuda")
        sa = torch.zeros((2, 0) if col else (0, 2), device="cuda")
        assert vg.fp8_block_gemm(a, sa, w, sw, col).shape == (0, 256)
        q, s = vg.fp8_block_gemm_silu_mul_fp8(a, sa, w, sw, col, col)
        assert q.shape == (0, 128) and s.shape == ((1, 0) if col else (0, 1))
    qkv = torch.zeros((0, 4 * 64), device="cuda").bfloat16()
    table, none = torch.zeros((16, 64), device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda")
    k, v = (torch.ones((2, 16, 1, 64), device="cuda").bfloat16() for _ in range(2))
    vg.vg_fused_qk_norm_mrope(qkv, None, None, table, none.view(2, 0), (16, 16), 2, 1, 64, 1e-6)
    vg.vg_fused_qk_norm_rope_append(qkv, k, v, None, None, table, none, none, 2, 1, 64, 1e-6)
    torch.cuda.synchronize()
    assert bool((k == 1).all()) and bool((v == 1).all())


def test_a_tensor_of_another_device_is_refused():
    import torch
    x = torch.zeros(4, device="cuda")
    other = torch.cuda.current_device() + 1
    for contiguous in (True, False):
        with pytest.raises(ValueError, match="current device"):
            vg._arg(x, (torch.float32,), "x", other, contiguous)


FIRST_CALL = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
import norm_activation_fp8_gb300 as vg
from test_fp8_gemm_gpu import operands
from test_rope_append_gpu import inputs, cuda
sets = [operands(T, N, K, 1, exact=True) for T, N, K in ((1, 1024, 512), (50, 640, 512), (196, 3704, 6912), (600, 8192, 512))]
d = inputs(20, 4, 2, 128, seed=1)
args = [cuda(d[n]) for n in ("q_weight", "k_weight", "cos_sin_cache", "positions")]
qkv, k, v = cuda(d["qkv"]).clone(), *(torch.zeros((2, 16, 2, 128), dtype=torch.int16, device="cuda") for _ in range(2))
slots = torch.arange(20, device="cuda")
outs = [torch.zeros((s[0].shape[0], s[2].shape[0]), dtype=torch.bfloat16, device="cuda") for s in sets]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for o, s in zip(outs, sets):
        vg.vg_fp8_block_gemm(o, *s[:4])
    vg.vg_fused_qk_norm_rope_append(qkv, k, v, *args, slots, 4, 2, 128, 1e-6)
g.replay()
torch.cuda.synchronize()
for o, s in zip(outs, sets):
    assert torch.equal(o, (s[4] @ s[5].t()).to(torch.bfloat16))
assert (v.view(-1, 256)[:20] == cuda(d["qkv"])[:, 768:]).all()
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


def test_calls_from_several_threads():
    """Host threads that call at once, each on its own stream."""
    import threading
    import torch
    from test_fp8_gemm_gpu import operands
    sets = [operands(T, 1024, 1024, T, exact=True) for T in (1, 20, 60, 300, 700, 3)]
    want = [(x[4] @ x[5].t()).to(torch.bfloat16) for x in sets]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()) as _:
            outs = [vg.fp8_block_gemm(*sets[i][:4]) for _ in range(50)]
            torch.cuda.current_stream().synchronize()
        if not all(torch.equal(o, want[i]) for o in outs):
            bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("first", ["gemm", "gated", "append", "mrope", "norm"])
def test_first_call_of_a_thread(first):
    """A host thread whose first use of CUDA is a call of this library, into
    outputs that are there already."""
    import threading
    import torch
    from test_fp8_gemm_gpu import operands
    from test_rope_append_gpu import cuda, inputs
    sets = [operands(T, 512, 512, T, exact=True) for T in (1, 40, 300)]
    outs = [torch.zeros((x[0].shape[0], 512), dtype=torch.bfloat16, device="cuda") for x in sets]
    qs = [torch.zeros((x[0].shape[0], 256), dtype=torch.float8_e4m3fn, device="cuda") for x in sets]
    scs = [torch.zeros((x[0].shape[0], 2), device="cuda") for x in sets]
    d = inputs(20, 4, 2, 128, seed=1)
    args = [cuda(d[n]) for n in ("q_weight", "k_weight", "cos_sin_cache")]
    pos, qkv = cuda(d["positions"]), cuda(d["qkv"]).clone()
    k, v = (torch.zeros((2, 16, 2, 128), dtype=torch.int16, device="cuda") for _ in range(2))
    slots, w = torch.arange(20, device="cuda"), torch.ones(512, device="cuda").bfloat16()
    stream = torch.cuda.current_stream().cuda_stream
    calls = {
        "gemm": lambda i: vg.vg_fp8_block_gemm(outs[i], *sets[i][:4], stream=stream),
        "gated": lambda i: vg.vg_fp8_block_gemm_silu_mul_fp8(qs[i], scs[i], *sets[i][:4], stream=stream),
        "append": lambda i: vg.vg_fused_qk_norm_rope_append(qkv, k, v, *args, pos, slots, 4, 2, 128, 1e-6,
                                                            stream=stream),
        "mrope": lambda i: vg.vg_fused_qk_norm_mrope(qkv, *args, pos.view(1, 20), (64,), 4, 2, 128, 1e-6,
                                                     stream=stream),
        "norm": lambda i: vg.vg_fused_add_rms_norm_fp8(qs[i].view(-1, 256), None, scs[i], outs[i][:, :256].contiguous(),
                                                       None, w[:256], 1e-5, vg.PER_GROUP, stream=stream),
    }
    torch.cuda.synchronize()
    raised = []

    def work(i):
        try:
            calls[first](i)
        except Exception as e:  # noqa: BLE001
            raised.append(e)

    for i in range(3):
        t = threading.Thread(target=work, args=(i,))
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert not raised
    if first == "gemm":
        for o, x in zip(outs, sets):
            assert torch.equal(o, (x[4] @ x[5].t()).to(torch.bfloat16))


def test_threads_that_call_at_once_raise_nothing():
    """As above, many threads at once, each allocating on a stream of its own."""
    import threading
    import torch
    from test_fp8_gemm_gpu import operands
    sets = [operands(T, 1024, 1024, T, exact=True) for T in (1, 20, 60, 300, 700, 3)]
    want = [(x[4] @ x[5].t()).to(torch.bfloat16) for x in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    done = []

    def work(i):
        with torch.cuda.stream(streams[i]):
            outs = [vg.fp8_block_gemm(*sets[i][:4]) for _ in range(50)]
            gated = [vg.fp8_block_gemm_silu_mul_fp8(*sets[i][:4]) for _ in range(10)]
            streams[i].synchronize()
        if all(torch.equal(o, want[i]) for o in outs) and all(torch.equal(s, gated[0][1]) for _, s in gated):
            done.append(i)

    for _ in range(5):
        threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    assert sorted(done) == sorted(list(range(len(sets))) * 5)


def _gemm(T, N, K):
    import torch
    from test_fp8_gemm_gpu import operands
    x = operands(T, N, K, T)[:4]
    return lambda: {"out": vg.fp8_block_gemm(*x).view(torch.int16).cpu().numpy()}


def _gated(T, n, K):
    import torch
    from test_fp8_gemm_gpu import operands
    x = operands(T, 2 * n, K, T)[:4]

    def run():
        q, s = vg.fp8_block_gemm_silu_mul_fp8(*x)
        return {"q": q.view(torch.uint8).cpu().numpy(), "scale": s.cpu().numpy()}
    return run


def _append(T, fp8):
    from test_rope_append_gpu import inputs, run_append
    d = inputs(T, 6, 2, 128, (24, 20, 20), True, seed=T)
    slots = np.arange(T, dtype=np.int64)[::-1].copy()

    def run():
        g, _, (k, v) = run_append(d, T, 6, 2, 128, fp8, True, True, (24, 20, 20), True, "tokens", 16, slots,
                                  T // 16 + 1)
        return {"qkv": g, "k": k, "v": v}
    return run


# every kernel form: stream tiles of 16 to 128 tokens, split and not; the tile
# kernel, split and not; the append with few and many tokens
CASES = {
    "gemm-1": lambda: _gemm(1, 1032, 1024), "gemm-20": lambda: _gemm(20, 96, 128),
    "gemm-50": lambda: _gemm(50, 2056, 512), "gemm-70": lambda: _gemm(70, 3800, 6912),
    "gemm-196-tile-split": lambda: _gemm(196, 3704, 6912), "gemm-700-tile": lambda: _gemm(700, 8200, 512),
    "gated-1": lambda: _gated(1, 256, 1024), "gated-40": lambda: _gated(40, 1152, 512),
    "gated-609-tile-split": lambda: _gated(609, 640, 11904), "gated-700-tile": lambda: _gated(700, 4096, 512),
    "append-9": lambda: _append(9, False), "append-700-fp8": lambda: _append(700, True),
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


@pytest.mark.parametrize("case", ["gemm-50", "gated-40", "gemm-196-tile-split", "append-9"])
def test_out_of_range_accesses_are_flagged_and_skipped(case, monkeypatch):
    """Thread stores, with every tensor reported one row short (the tile
    kernel's own stores are clipped by their tensor map)."""
    run = CASES[case]()
    want, _ = _with(vg.load(), run, monkeypatch)
    got, st = _with(vg.load(build.build_debug(shrunk=True)), run, monkeypatch)
    assert st & vg.DEVICE_OUT_OF_BOUNDS, st
    for k, v in want.items():
        if k in ("out", "q", "qkv"):
            assert np.array_equal(got[k][:-1], v[:-1]), k


@pytest.mark.parametrize("colmajor", [False, True], ids=["rows", "columns"])
@pytest.mark.parametrize("T,N,K", [(700, 8200, 512), (300, 264, 256), (1, 512, 512), (20, 96, 128), (50, 2056, 512),
                                   (70, 3800, 6912), (196, 3704, 6912)])
def test_scale_copies_are_checked(T, N, K, colmajor, monkeypatch):
    """Scales are read by their own index arithmetic, not through a tensor map.
    Debug build: nothing is flagged and the bits are the product's.  With every
    tensor one token short, the reads of the last token's scales are flagged
    (in the tile kernel nothing else could be: its stores are clipped by their
    map) and read as zeros; the other rows stay."""
    from test_fp8_gemm_gpu import operands
    x = operands(T, N, K, T, colmajor, exact=True)[:4]
    run = lambda: vg.fp8_block_gemm(*x, COL if colmajor else 0)  # noqa: E731
    want, st0 = _with(vg.load(), run, monkeypatch)
    got, st = _with(vg.load(build.build_debug()), run, monkeypatch)
    assert st0 == 0 and st == 0
    assert bool((got == want).all())
    got, st = _with(vg.load(build.build_debug(shrunk=True)), run, monkeypatch)
    assert st == vg.DEVICE_OUT_OF_BOUNDS
    assert bool((got[:-1] == want[:-1]).all())
    if T == 700:  # the tile kernel stores the row: its scales, or by columns the last one, were zeros
        zeroed = operands(T, N, K, T, colmajor, exact=True)[:4]
        zeroed[1][-1, T - 1 if colmajor else slice(None)] = 0
        assert bool((got[-1] == vg.fp8_block_gemm(*zeroed, COL if colmajor else 0)[-1]).all())


@pytest.mark.parametrize("T,N,K", [(1, 1024, 1024), (196, 3704, 6912), (600, 8192, 512)],
                         ids=["stream", "tile-split", "tile"])
def test_forced_wait_timeout_is_reported_and_context_survives(T, N, K):
    """The test copy's product warps also wait on a barrier that nothing arrives
    on: the wait gives up, every other wait runs out after it, the status says
    so, and the product library runs the same call right after."""
    import torch
    from test_fp8_gemm_gpu import operands
    lib = vg.load(build.build_wait_test())

    def status(reset):
        flags = ctypes.c_uint32(0)
        assert lib.vg_device_status(ctypes.byref(flags), reset) == 0
        return flags.value

    a, s, w, sw, A, W = operands(T, N, K, 1, exact=True)
    out = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
    status(1)
    ptrs = [x.data_ptr() for x in (out, a, s, w, sw)]
    assert lib.vg_fp8_block_gemm(*ptrs, T, N, K, 0, None) == 0
    torch.cuda.synchronize()
    assert status(1) & vg.DEVICE_WAIT_TIMEOUT
    assert status(0) == 0
    if N % 128 == 0:
        q = torch.zeros((T, N // 2), dtype=torch.uint8, device="cuda")
        sc = torch.zeros((T, N // 256), device="cuda")
        assert lib.vg_fp8_block_gemm_silu_mul_fp8(q.data_ptr(), sc.data_ptr(), *ptrs[1:], T, N // 2, K, 0, 0,
                                                  None) == 0
        torch.cuda.synchronize()
        assert status(1) & vg.DEVICE_WAIT_TIMEOUT
    vg.vg_device_status(reset=True)
    assert torch.equal(vg.fp8_block_gemm(a, s, w, sw), (A @ W.t()).to(torch.bfloat16))
    assert vg.vg_device_status() == 0
