"""The allocating PyTorch wrappers (fused_add_rms_norm_fp8, silu_mul_fp8,
fused_add_rms_norm_pad, the NVFP4 pair) against the oracle: they pass bf16
tensors through the C ABI, allocate outputs of the right shape and dtype,
update the residual in place when asked, and return the same results as the
raw calls' parity tests require."""
import numpy as np
import pytest

import gen
import parity
import norm_activation_fp8_gb300 as vg

pytestmark = pytest.mark.gpu

OPT = vg.UE8M0 | vg.COLUMN_MAJOR


def _bf16(torch, bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def _scales(s, mode, T, n, G):
    a = s.cpu().numpy()
    if mode & vg.COLUMN_MAJOR:
        return np.ascontiguousarray(a.reshape(n // G, -1)[:, :T].T)
    return a.reshape(-1) if (mode & 0xFF) != vg.PER_GROUP else a.reshape(T, n // G)


@pytest.mark.parametrize("inplace", [True, False], ids=["in-place", "out-of-place"])
@pytest.mark.parametrize("mode,G", [(vg.STATIC, 128), (vg.PER_TOKEN, 128), (vg.PER_GROUP, 128),
                                    (vg.PER_GROUP, 64), (vg.PER_GROUP | OPT, 128)],
                         ids=["static", "per-token", "per-group128", "per-group64", "ue8m0-colmajor"])
def test_fused_add_rms_norm_fp8_wrapper(mode, G, inplace):
    import torch
    T, H = 333, 4096
    d = gen.norm_inputs(T, H, seed=11)
    x, res, w = _bf16(torch, d["x"]), _bf16(torch, d["residual"]), _bf16(torch, d["weight"])
    scale = torch.tensor([0.05], dtype=torch.float32, device="cuda") if mode == vg.STATIC else None
    res_before = res.clone()
    q, s, r_out = vg.fused_add_rms_norm_fp8(x, res, w, 1e-5, mode, G, scale=scale, inplace=inplace)
    torch.cuda.synchronize()
    assert q.dtype == torch.float8_e4m3fn and tuple(q.shape) == (T, H)
    assert (r_out is res) == inplace
    if not inplace:
        assert torch.equal(res, res_before)
    o = parity.oracle_norm(d["x"], d["residual"], d["weight"], 1e-5, mode, G, scale=0.05)
    g = {"q": q.view(torch.uint8).cpu().numpy(), "scale": _scales(s, mode, T, H, G),
         "residual_out": r_out.view(torch.int16).cpu().numpy().view(np.uint16)}
    parity.check_norm(g, o, mode)


def test_fused_add_rms_norm_fp8_wrapper_without_residual():
    import torch
    T, H = 64, 2048
    d = gen.norm_inputs(T, H, seed=12)
    q, s, r_out = vg.fused_add_rms_norm_fp8(_bf16(torch, d["x"]), None, _bf16(torch, d["weight"]),
                                           1e-6, vg.PER_TOKEN)
    torch.cuda.synchronize()
    assert r_out is None
    o = parity.oracle_norm(d["x"], None, d["weight"], 1e-6, vg.PER_TOKEN)
    parity.check_norm({"q": q.view(torch.uint8).cpu().numpy(), "scale": s.cpu().numpy(),
                       "residual_out": None}, o, vg.PER_TOKEN)


@pytest.mark.parametrize("mode,G", [(vg.STATIC, 128), (vg.PER_TOKEN, 128), (vg.PER_GROUP, 128),
                                    (vg.PER_GROUP | OPT, 128)],
                         ids=["static", "per-token", "per-group128", "ue8m0-colmajor"])
def test_silu_mul_fp8_wrapper(mode, G):
    import torch
    T, I = 400, 14336
    d = gen.silu_inputs(T, I, seed=13)
    scale = torch.tensor([0.1], dtype=torch.float32, device="cuda") if mode == vg.STATIC else None
    q, s = vg.silu_mul_fp8(_bf16(torch, d["gate_up"]), mode, G, scale=scale)
    torch.cuda.synchronize()
    assert q.dtype == torch.float8_e4m3fn and tuple(q.shape) == (T, I)
    o = parity.oracle_silu(d["gate_up"], mode, G, scale=0.1)
    parity.check_silu({"q": q.view(torch.uint8).cpu().numpy(), "scale": _scales(s, mode, T, I, G)},
                      o, mode)


def test_fused_add_rms_norm_pad_wrapper():
    import torch
    T, H, P = 300, 2880, 3072
    d = gen.norm_inputs(T, H, seed=14)
    res = _bf16(torch, d["residual"])
    out, r_out = vg.fused_add_rms_norm_pad(_bf16(torch, d["x"]), res, _bf16(torch, d["weight"]),
                                           1e-5, P)
    torch.cuda.synchronize()
    assert out.dtype == torch.bfloat16 and tuple(out.shape) == (T, P) and r_out is res
    o = parity.oracle_pad(d["x"], d["residual"], d["weight"], 1e-5, P)
    parity.check_pad({"out": out.view(torch.int16).cpu().numpy().view(np.uint16),
                      "residual_out": r_out.view(torch.int16).cpu().numpy().view(np.uint16)}, o)


def test_nvfp4_wrappers():
    import torch
    gs = torch.tensor([168.0], dtype=torch.float32, device="cuda")
    T, H = 300, 8192
    d = gen.norm_inputs(T, H, seed=15)
    q4, sf, r_out = vg.fused_add_rms_norm_nvfp4(_bf16(torch, d["x"]), _bf16(torch, d["residual"]),
                                                _bf16(torch, d["weight"]), 1e-5, gs)
    torch.cuda.synchronize()
    assert tuple(q4.shape) == (T, H // 2) and tuple(sf.shape) == (T, H // 16)
    o = parity.oracle_nvfp4_norm(d["x"], d["residual"], d["weight"], 1e-5, 168.0)
    parity.check_nvfp4({"q4": q4.cpu().numpy(), "sf": sf.view(torch.uint8).cpu().numpy(),
                        "residual_out": r_out.view(torch.int16).cpu().numpy().view(np.uint16)}, o)
    I = 14336
    ds = gen.silu_inputs(T, I, seed=16)
    q4, sf = vg.silu_mul_nvfp4(_bf16(torch, ds["gate_up"]), gs)
    torch.cuda.synchronize()
    assert tuple(q4.shape) == (T, I // 2) and tuple(sf.shape) == (T, I // 16)
    o = parity.oracle_nvfp4_silu(ds["gate_up"], 168.0)
    parity.check_nvfp4({"q4": q4.cpu().numpy(), "sf": sf.view(torch.uint8).cpu().numpy()}, o)


def _calls(torch):
    """Every allocating call: (name, function of a stream that returns its outputs)."""
    T, H = 300, 1024
    g = torch.Generator(device="cuda").manual_seed(3)
    x, res = (torch.randn((T, H), generator=g, device="cuda").bfloat16() for _ in range(2))
    gu = torch.randn((T, 2 * H), generator=g, device="cuda").bfloat16()
    w, gs = torch.ones(H, device="cuda").bfloat16(), torch.ones(1, device="cuda")
    a = torch.randint(-2, 3, (T, H), generator=g, device="cuda").to(torch.float8_e4m3fn)
    b = torch.randint(-2, 3, (H, H), generator=g, device="cuda").to(torch.float8_e4m3fn)
    sa, sb = torch.ones((T, H // 128), device="cuda"), torch.ones((H // 128, H // 128), device="cuda")
    return {
        "norm": lambda s: vg.fused_add_rms_norm_fp8(x, res, w, 1e-5, vg.PER_GROUP, inplace=False, stream=s),
        "silu": lambda s: vg.silu_mul_fp8(gu, vg.PER_GROUP | OPT, stream=s),
        "mla": lambda s: vg.mla_dual_rms_norm(x, w, res, w, 1e-5, 1e-5, stream=s),
        "mla_fp8": lambda s: vg.mla_dual_rms_norm(x, w, res, w, 1e-5, 1e-5, True, stream=s),
        "pad": lambda s: vg.fused_add_rms_norm_pad(x, res, w, 1e-5, H + 256, inplace=False, stream=s),
        "norm_nvfp4": lambda s: vg.fused_add_rms_norm_nvfp4(x, res, w, 1e-5, gs, inplace=False, stream=s),
        "silu_nvfp4": lambda s: vg.silu_mul_nvfp4(gu, gs, stream=s),
        "gemm": lambda s: (vg.fp8_block_gemm(a, sa, b, sb, stream=s),),
        "gated": lambda s: vg.fp8_block_gemm_silu_mul_fp8(a, sa, b, sb, stream=s),
    }


def _pool_stream(torch, t):
    """The stream whose pool a tensor's memory belongs to."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's memory")


@pytest.mark.parametrize("name", ["norm", "silu", "mla", "mla_fp8", "pad", "norm_nvfp4", "silu_nvfp4", "gemm",
                                  "gated"])
def test_outputs_of_a_call_on_another_stream_are_that_streams_memory(name):
    """The call's stream does not wait for the current one, so its outputs must
    not reuse a block that work queued there still writes."""
    import torch
    call = _calls(torch)[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    big = torch.randn((8192, 8192), device="cuda").bfloat16()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        # blocks of the outputs' sizes, written late on the current stream, then freed
        old = [torch.empty_like(t) for t in want]
        for _ in range(20):
            big @ big
        for t in old:
            t.view(torch.uint8).fill_(0xAB)
        del old, t
        got = call(stream)
        assert all(_pool_stream(torch, t) == side.cuda_stream for t in got)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    with torch.cuda.stream(side):  # the current stream, given by name
        got = call(side)
    assert all(_pool_stream(torch, t) == side.cuda_stream for t in got)
    for stream in (0, torch.cuda.default_stream()):
        assert all(_pool_stream(torch, t) == 0 for t in call(stream))
        with torch.cuda.stream(side):
            assert all(_pool_stream(torch, t) == 0 for t in call(stream))
    torch.cuda.synchronize()
