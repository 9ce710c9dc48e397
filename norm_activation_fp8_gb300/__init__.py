"""Fused residual-add + RMSNorm -> FP8 and SiLU-and-mul -> FP8 on GB300, the
block-scaled FP8 products that read them, and QK norm + rotation with a paged
K/V cache.

Thin Python binding over the C ABI of ``libvg_fused.so`` (declared in
``include/vg_fused.h``).  Every step of both ops runs in the library's CUDA
kernels; this module only marshals arguments: it checks dtypes, devices and
contiguity of torch tensors, passes their device pointers and the current
CUDA stream, and turns a non-zero status into ``VgError``.  There is no CPU
fallback: if the library has not been built, every call raises.

Entry points (same names and argument order as the C ABI):
  vg_fused_add_rms_norm_fp8(q, residual_out, scale, x, residual, weight,
                            eps, mode, group_size=128, stream=None)
  vg_silu_mul_fp8(q, scale, gate_up, mode, group_size=128, stream=None)
  vg_fused_add_rms_norm_pad(out, residual_out, x, residual, weight, eps, stream=None)
  vg_fused_qk_norm_rope(qkv, q_weight, k_weight, cos_sin_cache, positions,
                        num_q_heads, num_kv_heads, head_dim, eps, is_neox=True, stream=None)
  vg_fused_mla_dual_rms_norm(q_out, kv_out, q_c, q_weight, kv_c, kv_weight,
                             eps_q, eps_kv, stream=None)
  vg_fused_mla_dual_rms_norm_per_token_quant(q_fp8, q_scale, kv_out, q_c,
                             q_weight, kv_c, kv_weight, eps_q, eps_kv, stream=None)
  (the MLA inputs may be column-slice views: their row stride is passed on)
  vg_fused_add_rms_norm_nvfp4(q4, block_scale, residual_out, x, residual, weight,
                              global_scale, eps, stream=None)
  vg_silu_mul_nvfp4(q4, block_scale, gate_up, global_scale, stream=None)
  vg_fused_qk_norm_mrope(qkv, q_weight, k_weight, cos_sin_cache, positions, sections,
                         num_q_heads, num_kv_heads, head_dim, eps, is_neox=True,
                         interleaved=False, stream=None)
  vg_fused_qk_norm_rope_append(qkv, k_cache, v_cache, q_weight, k_weight, cos_sin_cache,
                         positions, slots, num_q_heads, num_kv_heads, head_dim, eps,
                         is_neox=True, sections=None, interleaved=False, k_scale=None,
                         v_scale=None, stream=None)
  vg_fp8_block_gemm(out, a, a_scale, w, w_scale, a_options=0, stream=None)
  vg_fp8_block_gemm_silu_mul_fp8(q, scale, a, a_scale, w, w_scale, a_options=0,
                         out_options=0, stream=None)
Convenience wrappers that allocate the outputs with torch (as memory of the
stream they run on):
  fused_add_rms_norm_fp8(x, residual, weight, eps, mode, ...)
  silu_mul_fp8(gate_up, mode, ...)
  fused_add_rms_norm_pad(x, residual, weight, eps, padded_hidden, ...)
  mla_dual_rms_norm(q_c, q_weight, kv_c, kv_weight, eps_q, eps_kv, q_fp8=False)
  fused_add_rms_norm_nvfp4(x, residual, weight, eps, global_scale, ...)
  silu_mul_nvfp4(gate_up, global_scale, ...)
  fp8_block_gemm(a, a_scale, w, w_scale, a_options=0)
  fp8_block_gemm_silu_mul_fp8(a, a_scale, w, w_scale, a_options=0, out_options=0)
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

from .build import LIB_PATH

STATIC, PER_TOKEN, PER_GROUP = 0, 1, 2
UE8M0, COLUMN_MAJOR = 0x100, 0x200  # per-group options, or-ed into the mode
MAX_ROW = 32768

STATUS_NAMES = {
    0: "VG_OK", 1: "VG_ERR_NULL_PTR", 2: "VG_ERR_BAD_SHAPE", 3: "VG_ERR_MISALIGNED",
    4: "VG_ERR_BAD_MODE", 5: "VG_ERR_BAD_GROUP", 6: "VG_ERR_UNSUPPORTED_DEVICE", 7: "VG_ERR_CUDA",
}

EXPORTED_SYMBOLS = ("vg_fused_add_rms_norm_fp8", "vg_silu_mul_fp8", "vg_fused_add_rms_norm_pad",
                    "vg_fused_mla_dual_rms_norm", "vg_fused_qk_norm_rope",
                    "vg_fused_mla_dual_rms_norm_per_token_quant", "vg_fused_add_rms_norm_nvfp4",
                    "vg_silu_mul_nvfp4", "vg_fused_qk_norm_mrope", "vg_fused_qk_norm_rope_append",
                    "vg_fp8_block_gemm", "vg_fp8_block_gemm_silu_mul_fp8", "vg_device_status",
                    "vg_status_string", "vg_abi_version")
DEVICE_WAIT_TIMEOUT = 1
DEVICE_BAD_POSITION = 2
DEVICE_OUT_OF_BOUNDS = 4  # debug builds (VG_DEBUG_CHECKS) only
DEVICE_BAD_SLOT = 8
BLOCK = 128  # columns of an activation scale, rows and columns of a weight scale

_lock = threading.Lock()
_lib = None


class VgError(RuntimeError):
    """A non-zero vg_status returned by the library."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def load(path: str | None = None) -> ctypes.CDLL:
    """Load the CUDA library (built by ``build.build()``); raises if absent."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or os.environ.get("VG_FUSED_LIB", LIB_PATH)
        if not os.path.exists(p):
            raise RuntimeError(
                f"CUDA library {p} is missing: build it with "
                "`python -m norm_activation_fp8_gb300.build` (no CPU fallback exists)")
        lib = ctypes.CDLL(p)
        P, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        lib.vg_fused_add_rms_norm_fp8.argtypes = [P, P, P, P, P, P, i64, i64, ctypes.c_float,
                                                  i32, i32, P]
        lib.vg_fused_add_rms_norm_fp8.restype = ctypes.c_int
        lib.vg_silu_mul_fp8.argtypes = [P, P, P, i64, i64, i32, i32, P]
        lib.vg_silu_mul_fp8.restype = ctypes.c_int
        f32 = ctypes.c_float
        lib.vg_fused_add_rms_norm_pad.argtypes = [P, P, P, P, P, i64, i64, i64, f32, P]
        lib.vg_fused_qk_norm_rope.argtypes = [P, P, P, P, P, i64, i32, i32, i32, i64, f32, i32, P]
        lib.vg_fused_qk_norm_rope.restype = ctypes.c_int
        lib.vg_fused_add_rms_norm_pad.restype = ctypes.c_int
        lib.vg_fused_mla_dual_rms_norm.argtypes = [P, P, P, i64, P, P, i64, P, i64, i64, i64,
                                                   f32, f32, P]
        lib.vg_fused_mla_dual_rms_norm.restype = ctypes.c_int
        lib.vg_fused_mla_dual_rms_norm_per_token_quant.argtypes = [P, P, P, P, i64, P, P, i64, P,
                                                                   i64, i64, i64, f32, f32, P]
        lib.vg_fused_mla_dual_rms_norm_per_token_quant.restype = ctypes.c_int
        lib.vg_fused_add_rms_norm_nvfp4.argtypes = [P, P, P, P, P, P, P, i64, i64, f32, P]
        lib.vg_fused_add_rms_norm_nvfp4.restype = ctypes.c_int
        lib.vg_silu_mul_nvfp4.argtypes = [P, P, P, P, i64, i64, P]
        lib.vg_silu_mul_nvfp4.restype = ctypes.c_int
        lib.vg_fused_qk_norm_mrope.argtypes = [P, P, P, P, P, P, i32, i64, i32, i32, i32, i64, f32,
                                               i32, i32, P]
        lib.vg_fused_qk_norm_mrope.restype = ctypes.c_int
        lib.vg_fused_qk_norm_rope_append.argtypes = [P] * 10 + [P, i32, i64, i32, i32, i32, i64, i64,
                                                                i64, i64, i64, i64, f32, i32, i32, P]
        lib.vg_fused_qk_norm_rope_append.restype = ctypes.c_int
        lib.vg_fp8_block_gemm.argtypes = [P, P, P, P, P, i64, i64, i64, i32, P]
        lib.vg_fp8_block_gemm.restype = ctypes.c_int
        lib.vg_fp8_block_gemm_silu_mul_fp8.argtypes = [P, P, P, P, P, P, i64, i64, i64, i32, i32, P]
        lib.vg_fp8_block_gemm_silu_mul_fp8.restype = ctypes.c_int
        lib.vg_status_string.argtypes = [ctypes.c_int]
        lib.vg_status_string.restype = ctypes.c_char_p
        lib.vg_abi_version.argtypes = []
        lib.vg_abi_version.restype = i32
        lib.vg_device_status.argtypes = [P, i32]
        lib.vg_device_status.restype = ctypes.c_int
        if path is None:
            _lib = lib
        return lib


def status_string(status: int) -> str:
    return load().vg_status_string(status).decode()


def _check(status: int):
    if status != 0:
        raise VgError(status, status_string(status))


# ----------------------------------------------------------- marshalling

def _ptr(t, dtypes, name):
    """Device pointer of a torch tensor (or pass an int pointer / None)."""
    if t is None or isinstance(t, int):
        return t
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, an int pointer or None")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor (there is no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _allocator(stream):
    """torch.empty for the outputs of a call: memory of the stream it runs on.
    Memory of the current stream may still be in use there by work queued
    before, which another stream does not wait for."""
    import torch
    if stream is None:
        return torch.empty
    raw = _stream(stream)
    if raw == torch.cuda.current_stream().cuda_stream:
        return torch.empty
    if not isinstance(stream, torch.cuda.Stream):
        # 0 and 1 (cudaStreamLegacy) are the default stream
        stream = torch.cuda.ExternalStream(raw) if raw > 1 else torch.cuda.default_stream()

    def empty(shape, dtype, device):
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=device)
    return empty


def _dtypes():
    import torch
    bf16 = (torch.bfloat16, torch.int16, torch.uint16)
    fp8 = (torch.float8_e4m3fn, torch.uint8, torch.int8)
    return bf16, fp8, (torch.float32,)


def _rows(t, name):
    if isinstance(t, int) or t is None:
        raise ValueError(f"{name}: shapes cannot be taken from a raw pointer; pass num_tokens")
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D [T, n] tensor")
    return t.shape[0], t.shape[1]


def vg_fused_add_rms_norm_fp8(q, residual_out, scale, x, residual, weight, eps: float,
                              mode: int, group_size: int = 128, stream=None,
                              num_tokens: int | None = None, hidden: int | None = None):
    """Residual add + RMSNorm -> FP8 through the C ABI (outputs preallocated).

    q [T,H] fp8/uint8; residual_out [T,H] bf16 (may be ``residual`` itself)
    or None with residual None; scale fp32 ([1] static input, [T] or
    [T,H/G] output); x [T,H] bf16; residual [T,H] bf16 or None; weight [H]."""
    bf16, fp8, f32 = _dtypes()
    if num_tokens is None or hidden is None:
        num_tokens, hidden = _rows(x, "x")
    st = load().vg_fused_add_rms_norm_fp8(
        _ptr(q, fp8, "q"), _ptr(residual_out, bf16, "residual_out"), _ptr(scale, f32, "scale"),
        _ptr(x, bf16, "x"), _ptr(residual, bf16, "residual"), _ptr(weight, bf16, "weight"),
        num_tokens, hidden, ctypes.c_float(eps), mode, group_size, _stream(stream))
    _check(st)


def vg_silu_mul_fp8(q, scale, gate_up, mode: int, group_size: int = 128, stream=None,
                    num_tokens: int | None = None, inter: int | None = None):
    """SiLU(gate) * up -> FP8 through the C ABI (outputs preallocated).

    q [T,I] fp8/uint8; scale fp32 ([1] static input, [T] or [T,I/G]
    output); gate_up [T,2I] bf16 with gate = columns [0,I), up = [I,2I)."""
    bf16, fp8, f32 = _dtypes()
    if num_tokens is None or inter is None:
        num_tokens, two_i = _rows(gate_up, "gate_up")
        if two_i % 2:
            raise ValueError("gate_up must have an even number of columns")
        inter = two_i // 2
    st = load().vg_silu_mul_fp8(_ptr(q, fp8, "q"), _ptr(scale, f32, "scale"),
                                _ptr(gate_up, bf16, "gate_up"), num_tokens, inter, mode,
                                group_size, _stream(stream))
    _check(st)


def vg_fused_add_rms_norm_pad(out, residual_out, x, residual, weight, eps: float, stream=None,
                              num_tokens: int | None = None, hidden: int | None = None,
                              padded_hidden: int | None = None):
    """Residual add + RMSNorm into a padded bf16 row through the C ABI.

    out [T, padded] bf16 (columns >= H come back zero); residual_out [T,H]
    (may be ``residual`` itself) or None with residual None; x [T,H]; weight [H]."""
    bf16, _, _ = _dtypes()
    if num_tokens is None or hidden is None:
        num_tokens, hidden = _rows(x, "x")
    if padded_hidden is None:
        padded_hidden = _rows(out, "out")[1]
    _check(load().vg_fused_add_rms_norm_pad(
        _ptr(out, bf16, "out"), _ptr(residual_out, bf16, "residual_out"), _ptr(x, bf16, "x"),
        _ptr(residual, bf16, "residual"), _ptr(weight, bf16, "weight"), num_tokens, hidden,
        padded_hidden, ctypes.c_float(eps), _stream(stream)))


def vg_fused_qk_norm_rope(qkv, q_weight, k_weight, cos_sin_cache, positions, num_q_heads: int,
                          num_kv_heads: int, head_dim: int, eps: float, is_neox: bool = True,
                          stream=None):
    """Per-head QK RMSNorm + rotary embedding, in place on qkv
    [T, (Hq + 2 Hkv) * D] bf16; cos_sin_cache fp32 [max_pos, D]; positions
    int64 [T]."""
    import torch
    bf16, _, f32 = _dtypes()
    T = _rows(qkv, "qkv")[0]
    max_pos = _rows(cos_sin_cache, "cos_sin_cache")[0]
    _check(load().vg_fused_qk_norm_rope(
        _ptr(qkv, bf16, "qkv"), _ptr(q_weight, bf16, "q_weight"), _ptr(k_weight, bf16, "k_weight"),
        _ptr(cos_sin_cache, f32, "cos_sin_cache"), _ptr(positions, (torch.int64,), "positions"),
        T, num_q_heads, num_kv_heads, head_dim, max_pos, ctypes.c_float(eps),
        1 if is_neox else 0, _stream(stream)))


def _rows_ptr(t, name):
    """(device pointer, row stride in elements, rows, columns) of a 2-D bf16
    CUDA tensor whose rows are contiguous (a column slice is fine)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    bf16, _, _ = _dtypes()
    if t.dtype not in bf16:
        raise TypeError(f"{name}: dtype {t.dtype} not in {bf16}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor (there is no CPU path)")
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name}: expected a 2-D [T, n] tensor with contiguous rows")
    return t.data_ptr(), t.stride(0), t.shape[0], t.shape[1]


def vg_fused_mla_dual_rms_norm(q_out, kv_out, q_c, q_weight, kv_c, kv_weight, eps_q: float,
                               eps_kv: float, stream=None):
    """MLA dual RMSNorm through the C ABI: q_out = bf16(rms_norm(q_c)),
    kv_out = bf16(rms_norm(kv_c)) in one launch (outputs preallocated,
    dense bf16; q_c / kv_c may be column slices of one projected tensor)."""
    bf16, _, _ = _dtypes()
    qp, qs, T, q_dim = _rows_ptr(q_c, "q_c")
    kp, ks, T2, kv_dim = _rows_ptr(kv_c, "kv_c")
    if T2 != T:
        raise ValueError("q_c and kv_c must have the same number of rows")
    _check(load().vg_fused_mla_dual_rms_norm(
        _ptr(q_out, bf16, "q_out"), _ptr(kv_out, bf16, "kv_out"), qp, qs,
        _ptr(q_weight, bf16, "q_weight"), kp, ks, _ptr(kv_weight, bf16, "kv_weight"),
        T, q_dim, kv_dim, ctypes.c_float(eps_q), ctypes.c_float(eps_kv), _stream(stream)))


def vg_fused_mla_dual_rms_norm_per_token_quant(q_fp8, q_scale, kv_out, q_c, q_weight, kv_c,
                                               kv_weight, eps_q: float, eps_kv: float,
                                               stream=None):
    """The per-token-quant variant: q to FP8 with q_scale [T] fp32, kv bf16."""
    bf16, fp8, f32 = _dtypes()
    qp, qs, T, q_dim = _rows_ptr(q_c, "q_c")
    kp, ks, T2, kv_dim = _rows_ptr(kv_c, "kv_c")
    if T2 != T:
        raise ValueError("q_c and kv_c must have the same number of rows")
    _check(load().vg_fused_mla_dual_rms_norm_per_token_quant(
        _ptr(q_fp8, fp8, "q_fp8"), _ptr(q_scale, f32, "q_scale"), _ptr(kv_out, bf16, "kv_out"),
        qp, qs, _ptr(q_weight, bf16, "q_weight"), kp, ks, _ptr(kv_weight, bf16, "kv_weight"),
        T, q_dim, kv_dim, ctypes.c_float(eps_q), ctypes.c_float(eps_kv), _stream(stream)))


def vg_fused_add_rms_norm_nvfp4(q4, block_scale, residual_out, x, residual, weight,
                                global_scale, eps: float, stream=None,
                                num_tokens: int | None = None, hidden: int | None = None):
    """Residual add + RMSNorm -> NVFP4 through the C ABI (outputs preallocated).

    q4 [T,H/2] uint8 (two E2M1 codes a byte, column 2i in the low nibble);
    block_scale [T,H/16] uint8 E4M3 codes; residual_out as for the FP8 op;
    global_scale fp32 [1] on the device."""
    import torch
    bf16, fp8, f32 = _dtypes()
    u8 = (torch.uint8,)
    if num_tokens is None or hidden is None:
        num_tokens, hidden = _rows(x, "x")
    _check(load().vg_fused_add_rms_norm_nvfp4(
        _ptr(q4, u8, "q4"), _ptr(block_scale, fp8, "block_scale"),
        _ptr(residual_out, bf16, "residual_out"), _ptr(x, bf16, "x"),
        _ptr(residual, bf16, "residual"), _ptr(weight, bf16, "weight"),
        _ptr(global_scale, f32, "global_scale"), num_tokens, hidden, ctypes.c_float(eps),
        _stream(stream)))


def vg_silu_mul_nvfp4(q4, block_scale, gate_up, global_scale, stream=None,
                      num_tokens: int | None = None, inter: int | None = None):
    """SiLU(gate) * up -> NVFP4 through the C ABI: q4 [T,I/2] uint8,
    block_scale [T,I/16] E4M3 codes, gate_up [T,2I] bf16, global_scale fp32
    [1] on the device."""
    import torch
    bf16, fp8, f32 = _dtypes()
    if num_tokens is None or inter is None:
        num_tokens, two_i = _rows(gate_up, "gate_up")
        if two_i % 2:
            raise ValueError("gate_up must have an even number of columns")
        inter = two_i // 2
    _check(load().vg_silu_mul_nvfp4(
        _ptr(q4, (torch.uint8,), "q4"), _ptr(block_scale, fp8, "block_scale"),
        _ptr(gate_up, bf16, "gate_up"), _ptr(global_scale, f32, "global_scale"), num_tokens,
        inter, _stream(stream)))


# The calls below check all their tensors in one expression and look for the
# reason only when it fails (_arg, _shape): on a decode step the host's time
# for a call is longer than the kernel's.

def _arg(t, dtypes, name, dev, contiguous=True):
    """Refuses a tensor that is not of these dtypes, on the device ``dev`` and contiguous."""
    if not contiguous:
        t = t[:0]
    _ptr(t, dtypes, name)
    if t is not None and t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{dev}: call under "
                         "torch.cuda.device(tensor.device)")


def _shape(t, shape, name):
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")


@functools.cache
def _kinds():
    """(bf16, fp8, fp32, int64 dtypes, torch)"""
    import torch
    return *_dtypes(), (torch.int64,), torch


def _here(t, stream):
    """(current device, raw stream) of a call whose tensors should be where ``t`` is; for a CPU
    tensor a device that no tensor is on."""
    if t.get_device() < 0:
        return -2, 0
    torch = _kinds()[4]
    dev = torch.cuda.current_device()
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    return dev, _stream(stream)


def _sections(sections, positions):
    """(ctypes array or None, number of axes, tokens) of a rotary position tensor."""
    if sections is None:
        if positions.dim() != 1:
            raise ValueError("positions: expected a 1-D [T] tensor (or give sections)")
        return None, 1, positions.shape[0]
    n = len(sections)
    if positions.dim() != 2 or positions.shape[0] != n:
        raise ValueError(f"positions: expected a 2-D [{n}, T] tensor, one row per axis")
    return (ctypes.c_int32 * n)(*sections), n, positions.shape[1]


def _rope_args(qkv, q_weight, k_weight, cos_sin_cache, positions, sections, num_q_heads,
               num_kv_heads, head_dim, dev):
    """Checked pointers and sizes that the multi-axis and cache forms share."""
    bf16, _, f32, i64, _ = _kinds()
    sec, axes, T = _sections(sections, positions)
    row = (num_q_heads + 2 * num_kv_heads) * head_dim
    max_pos = cos_sin_cache.shape[0]
    if (qkv.shape != (T, row) or cos_sin_cache.shape != (max_pos, head_dim)
            or qkv.dtype not in bf16 or qkv.get_device() != dev or not qkv.is_contiguous()
            or cos_sin_cache.dtype not in f32 or cos_sin_cache.get_device() != dev
            or not cos_sin_cache.is_contiguous() or positions.dtype not in i64
            or positions.get_device() != dev or not positions.is_contiguous()):
        if _rows(qkv, "qkv")[1] != row:
            raise ValueError("qkv: expected (num_q_heads + 2 num_kv_heads) * head_dim columns")
        if qkv.shape[0] != T:
            raise ValueError("positions and qkv must have the same number of tokens")
        if _rows(cos_sin_cache, "cos_sin_cache")[1] != head_dim:
            raise ValueError("cos_sin_cache: expected head_dim columns")
        _arg(qkv, bf16, "qkv", dev)
        _arg(cos_sin_cache, f32, "cos_sin_cache", dev)
        _arg(positions, i64, "positions", dev)
    qw = kw = None
    if q_weight is not None:
        _shape(q_weight, (head_dim,), "q_weight")
        if q_weight.dtype not in bf16 or q_weight.get_device() != dev or not q_weight.is_contiguous():
            _arg(q_weight, bf16, "q_weight", dev)
        qw = q_weight.data_ptr()
    if k_weight is not None:
        _shape(k_weight, (head_dim,), "k_weight")
        if k_weight.dtype not in bf16 or k_weight.get_device() != dev or not k_weight.is_contiguous():
            _arg(k_weight, bf16, "k_weight", dev)
        kw = k_weight.data_ptr()
    return (qkv.data_ptr(), qw, kw, cos_sin_cache.data_ptr(), positions.data_ptr(), sec, axes, T,
            max_pos)


def vg_fused_qk_norm_mrope(qkv, q_weight, k_weight, cos_sin_cache, positions, sections,
                           num_q_heads: int, num_kv_heads: int, head_dim: int, eps: float,
                           is_neox: bool = True, interleaved: bool = False, stream=None):
    """Per-head QK RMSNorm + rotation with several position axes, in place on
    qkv [T, (Hq + 2 Hkv) * D] bf16.

    positions int64 [axes, T]; sections: how many of the D/2 pairs each axis
    turns (their sum is D/2), in runs or, ``interleaved``, taking turns.
    q_weight and k_weight [D] bf16, or both None: the rotation only."""
    dev, raw = _here(qkv, stream)
    q, qw, kw, table, pos, sec, axes, T, max_pos = _rope_args(
        qkv, q_weight, k_weight, cos_sin_cache, positions, sections, num_q_heads, num_kv_heads,
        head_dim, dev)
    st = (_lib or load()).vg_fused_qk_norm_mrope(
        q, qw, kw, table, pos, sec, axes, T, num_q_heads, num_kv_heads, head_dim, max_pos, eps,
        is_neox, interleaved, raw)
    if st:
        _check(st)


def vg_fused_qk_norm_rope_append(qkv, k_cache, v_cache, q_weight, k_weight, cos_sin_cache,
                                 positions, slots, num_q_heads: int, num_kv_heads: int,
                                 head_dim: int, eps: float, is_neox: bool = True, sections=None,
                                 interleaved: bool = False, k_scale=None, v_scale=None,
                                 stream=None):
    """QK RMSNorm (or none) + rotation, Q in place, K and V into a paged cache.

    k_cache, v_cache [pages, page_size, Hkv, D], bf16, or FP8 with k_scale and
    v_scale fp32 [1] on the device; any strides in multiples of 8 elements
    (the same for both) with contiguous head rows, so a [pages, Hkv,
    page_size, D] cache is passed as its transposed view.  slots int64 [T]:
    page * page_size + place in the page, distinct; a negative slot appends
    nothing.  positions int64 [T], or [axes, T] with ``sections`` as for
    vg_fused_qk_norm_mrope."""
    bf16, fp8, f32, i64, _ = _kinds()
    dev, raw = _here(qkv, stream)
    q, qw, kw, table, pos, sec, axes, T, max_pos = _rope_args(
        qkv, q_weight, k_weight, cos_sin_cache, positions, sections, num_q_heads, num_kv_heads,
        head_dim, dev)
    kinds, ks, vs = bf16, None, None
    if k_scale is not None or v_scale is not None:
        kinds = fp8
        for x, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if x is not None and x.numel() != 1:
                raise ValueError(f"{name}: expected one fp32 value on the device")
            _arg(x, f32, name, dev)
        ks = None if k_scale is None else k_scale.data_ptr()
        vs = None if v_scale is None else v_scale.data_ptr()
    shape, strides = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or shape[2] != num_kv_heads or shape[3] != head_dim or strides[3] != 1:
        raise ValueError("k_cache: expected [pages, page_size, num_kv_heads, head_dim] with "
                         "contiguous head rows")
    if shape != v_cache.shape or strides != v_cache.stride():
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    if (k_cache.dtype not in kinds or k_cache.get_device() != dev or v_cache.dtype not in kinds
            or v_cache.get_device() != dev or slots.shape != (T,) or slots.dtype not in i64
            or slots.get_device() != dev or not slots.is_contiguous()):
        _arg(k_cache, kinds, "k_cache", dev, False)
        _arg(v_cache, kinds, "v_cache", dev, False)
        _shape(slots, (T,), "slots")
        _arg(slots, i64, "slots", dev)
    st = (_lib or load()).vg_fused_qk_norm_rope_append(
        q, k_cache.data_ptr(), v_cache.data_ptr(), qw, kw, table, pos, slots.data_ptr(), ks, vs, sec,
        axes, T, num_q_heads, num_kv_heads, head_dim, max_pos, shape[0], shape[1], strides[0],
        strides[1], strides[2], eps, is_neox, interleaved, raw)
    if st:
        _check(st)


def _block_gemm_sizes(a, a_scale, w, w_scale, a_options, dev):
    """T, N and K of an FP8 product's checked operands."""
    _, fp8, f32, _, _ = _kinds()
    N, K = _rows(w, "w")
    T, kb = a.shape[0], K // BLOCK
    scales = (kb, (T + 3) // 4 * 4) if a_options & COLUMN_MAJOR else (T, kb)
    if (a.shape != (T, K) or a_scale.shape != scales or w_scale.shape != ((N + BLOCK - 1) // BLOCK, kb)
            or a.dtype not in fp8 or a.get_device() != dev or not a.is_contiguous()
            or w.dtype not in fp8 or w.get_device() != dev or not w.is_contiguous()
            or a_scale.dtype not in f32 or a_scale.get_device() != dev or not a_scale.is_contiguous()
            or w_scale.dtype not in f32 or w_scale.get_device() != dev or not w_scale.is_contiguous()):
        if _rows(a, "a")[1] != K:
            raise ValueError("a and w must have the same number of columns")
        _shape(a_scale, scales, "a_scale")
        _shape(w_scale, ((N + BLOCK - 1) // BLOCK, kb), "w_scale")
        for t, kinds, name in ((a, fp8, "a"), (a_scale, f32, "a_scale"), (w, fp8, "w"),
                               (w_scale, f32, "w_scale")):
            _arg(t, kinds, name, dev)
    return T, N, K


def vg_fp8_block_gemm(out, a, a_scale, w, w_scale, a_options: int = 0, stream=None):
    """FP8 product with a scale per block of 128 through the C ABI:
    out [T,N] bf16 = (a * a_scale) (w * w_scale)^T.

    a [T,K] fp8 with a_scale fp32 [T,K/128] (or, with COLUMN_MAJOR in
    a_options, [K/128,T4] as the per-group ops write it); w [N,K] fp8 with
    w_scale fp32 [ceil(N/128),K/128].  UE8M0 scales need no option.
    ``out`` None allocates it; returns out."""
    bf16, _, _, _, torch = _kinds()
    dev, raw = _here(a, stream)
    T, N, K = _block_gemm_sizes(a, a_scale, w, w_scale, a_options, dev)
    if out is None:
        out = _allocator(stream)((T, N), dtype=bf16[0], device=a.device)
    elif (out.shape != (T, N) or out.dtype not in bf16 or out.get_device() != dev
          or not out.is_contiguous()):
        _shape(out, (T, N), "out")
        _arg(out, bf16, "out", dev)
    st = (_lib or load()).vg_fp8_block_gemm(out.data_ptr(), a.data_ptr(), a_scale.data_ptr(),
                                            w.data_ptr(), w_scale.data_ptr(), T, N, K, a_options, raw)
    if st:
        _check(st)
    return out


def vg_fp8_block_gemm_silu_mul_fp8(q, scale, a, a_scale, w, w_scale, a_options: int = 0,
                                   out_options: int = 0, stream=None):
    """Gated feed-forward projection through the C ABI: the gate and up
    products, SiLU(gate) * up and its per-group-128 FP8 codes in one kernel.

    a and a_scale as for vg_fp8_block_gemm; w [2I,K] fp8 (gate rows [0,I), up
    rows [I,2I)) with w_scale [2I/128,K/128]; q [T,I] fp8, scale fp32
    [T,I/128], or with COLUMN_MAJOR in out_options [I/128,T4]; UE8M0 in
    out_options: power-of-two scales.  ``q`` and ``scale`` both None
    allocate them; returns (q, scale)."""
    _, fp8, f32, _, torch = _kinds()
    dev, raw = _here(a, stream)
    T, N, K = _block_gemm_sizes(a, a_scale, w, w_scale, a_options, dev)
    if N % 2:
        raise ValueError("w must have an even number of rows (gate, then up)")
    inter = N // 2
    shape = (inter // BLOCK, (T + 3) // 4 * 4) if out_options & COLUMN_MAJOR else (T, inter // BLOCK)
    if q is None and scale is None:
        empty = _allocator(stream)
        q = empty((T, inter), dtype=fp8[0], device=a.device)
        scale = empty(shape, dtype=f32[0], device=a.device)
    elif (q is None or scale is None or q.shape != (T, inter) or q.dtype not in fp8
          or q.get_device() != dev or not q.is_contiguous() or scale.shape != shape
          or scale.dtype not in f32 or scale.get_device() != dev or not scale.is_contiguous()):
        if q is None or scale is None:
            raise ValueError("q and scale: give both or neither")
        _shape(q, (T, inter), "q")
        _arg(q, fp8, "q", dev)
        _shape(scale, shape, "scale")
        _arg(scale, f32, "scale", dev)
    st = (_lib or load()).vg_fp8_block_gemm_silu_mul_fp8(
        q.data_ptr(), scale.data_ptr(), a.data_ptr(), a_scale.data_ptr(), w.data_ptr(),
        w_scale.data_ptr(), T, inter, K, a_options, out_options, raw)
    if st:
        _check(st)
    return q, scale


def vg_device_status(reset: bool = False) -> int:
    """Flags the library's kernels left on the current device
    (DEVICE_WAIT_TIMEOUT: a bounded wait gave up; that call's outputs are
    not valid).  Synchronous."""
    flags = ctypes.c_uint32(0)
    _check(load().vg_device_status(ctypes.byref(flags), 1 if reset else 0))
    return flags.value


# ------------------------------------------------- allocating wrappers

def _scale_out(empty, mode, T, n, group_size, scale, device):
    import torch
    if mode & COLUMN_MAJOR:
        return empty((n // group_size, (T + 3) // 4 * 4), dtype=torch.float32, device=device)
    mode &= 0xFF
    if mode == STATIC:
        if scale is None:
            raise ValueError("static mode needs a scale tensor")
        return scale
    if mode == PER_TOKEN:
        return empty((T,), dtype=torch.float32, device=device)
    return empty((T, n // group_size), dtype=torch.float32, device=device)


def fused_add_rms_norm_fp8(x, residual, weight, eps: float, mode: int, group_size: int = 128,
                           scale=None, inplace: bool = True, stream=None):
    """Returns (q float8_e4m3fn [T,H], scale, residual_out).  With
    ``inplace`` the residual is updated in place, as the fused op does."""
    import torch
    T, H = x.shape
    empty = _allocator(stream)
    q = empty((T, H), dtype=torch.float8_e4m3fn, device=x.device)
    s = _scale_out(empty, mode, T, H, group_size, scale, x.device)
    r_out = None
    if residual is not None:
        r_out = residual if inplace else empty(residual.shape, dtype=residual.dtype, device=residual.device)
    vg_fused_add_rms_norm_fp8(q, r_out, s, x, residual, weight, eps, mode, group_size, stream)
    return q, s, r_out


def silu_mul_fp8(gate_up, mode: int, group_size: int = 128, scale=None, stream=None):
    """Returns (q float8_e4m3fn [T,I], scale)."""
    import torch
    T, two_i = gate_up.shape
    empty = _allocator(stream)
    q = empty((T, two_i // 2), dtype=torch.float8_e4m3fn, device=gate_up.device)
    s = _scale_out(empty, mode, T, two_i // 2, group_size, scale, gate_up.device)
    vg_silu_mul_fp8(q, s, gate_up, mode, group_size, stream)
    return q, s


def mla_dual_rms_norm(q_c, q_weight, kv_c, kv_weight, eps_q: float, eps_kv: float,
                      q_fp8: bool = False, stream=None):
    """Returns (q_normed bf16 [T,q_dim], kv_normed bf16 [T,kv_dim]), or with
    ``q_fp8`` (q float8_e4m3fn [T,q_dim], q_scale fp32 [T], kv_normed)."""
    import torch
    T, q_dim = q_c.shape
    empty = _allocator(stream)
    kv = empty((T, kv_c.shape[1]), dtype=kv_c.dtype, device=kv_c.device)
    q = empty((T, q_dim), dtype=torch.float8_e4m3fn if q_fp8 else q_c.dtype, device=q_c.device)
    s = empty((T,), dtype=torch.float32, device=q_c.device) if q_fp8 else None
    if q_fp8:
        vg_fused_mla_dual_rms_norm_per_token_quant(q, s, kv, q_c, q_weight, kv_c, kv_weight,
                                                   eps_q, eps_kv, stream)
        return q, s, kv
    vg_fused_mla_dual_rms_norm(q, kv, q_c, q_weight, kv_c, kv_weight, eps_q, eps_kv, stream)
    return q, kv


def fused_add_rms_norm_pad(x, residual, weight, eps: float, padded_hidden: int,
                           inplace: bool = True, stream=None):
    """Returns (out bf16 [T, padded_hidden], residual_out)."""
    import torch
    T, H = x.shape
    empty = _allocator(stream)
    out = empty((T, padded_hidden), dtype=x.dtype, device=x.device)
    r_out = None
    if residual is not None:
        r_out = residual if inplace else empty(residual.shape, dtype=residual.dtype, device=residual.device)
    vg_fused_add_rms_norm_pad(out, r_out, x, residual, weight, eps, stream)
    return out, r_out


def fused_add_rms_norm_nvfp4(x, residual, weight, eps: float, global_scale, inplace: bool = True,
                             stream=None):
    """Returns (q4 uint8 [T,H/2], block_scale float8_e4m3fn [T,H/16],
    residual_out); global_scale is an fp32 [1] device tensor."""
    import torch
    T, H = x.shape
    empty = _allocator(stream)
    q4 = empty((T, H // 2), dtype=torch.uint8, device=x.device)
    sf = empty((T, H // 16), dtype=torch.float8_e4m3fn, device=x.device)
    r_out = None
    if residual is not None:
        r_out = residual if inplace else empty(residual.shape, dtype=residual.dtype, device=residual.device)
    vg_fused_add_rms_norm_nvfp4(q4, sf, r_out, x, residual, weight, global_scale, eps, stream)
    return q4, sf, r_out


def silu_mul_nvfp4(gate_up, global_scale, stream=None):
    """Returns (q4 uint8 [T,I/2], block_scale float8_e4m3fn [T,I/16])."""
    import torch
    T, two_i = gate_up.shape
    empty = _allocator(stream)
    q4 = empty((T, two_i // 4), dtype=torch.uint8, device=gate_up.device)
    sf = empty((T, two_i // 32), dtype=torch.float8_e4m3fn, device=gate_up.device)
    vg_silu_mul_nvfp4(q4, sf, gate_up, global_scale, stream)
    return q4, sf


def fp8_block_gemm(a, a_scale, w, w_scale, a_options: int = 0, stream=None):
    """Returns out bf16 [T,N]."""
    return vg_fp8_block_gemm(None, a, a_scale, w, w_scale, a_options, stream)


def fp8_block_gemm_silu_mul_fp8(a, a_scale, w, w_scale, a_options: int = 0, out_options: int = 0,
                                stream=None):
    """Returns (q float8_e4m3fn [T,I], scale)."""
    return vg_fp8_block_gemm_silu_mul_fp8(None, None, a, a_scale, w, w_scale, a_options, out_options,
                                          stream)
