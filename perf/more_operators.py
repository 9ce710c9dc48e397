"""Cases of the NVFP4 operators: quantisation and reading back, the product, the
gated feed-forward projection.

NVFP4: E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two a byte
with column 2i in the low nibble; one E4M3 scale per 16 columns of a row,
sf = e4m3(gs amax / 6); one fp32 scale gs for the tensor.  A code c stands for
c sf / gs, and is e2m1(x gs / sf).

  roundtrip  rows of bf16 to NVFP4, and read back to bf16
  gemm       out = bf16(alpha a w^T), a [T, K] and w [N, K] in NVFP4, alpha
             what the two tensors' own scales come to
  gated      g and u as gemm's (not rounded), SiLU(g) u, and NVFP4 again
  linear     rows of bf16 to NVFP4, and a product
  ffn        gated, and a product on what it wrote: a feed-forward block

``own`` selects the plain torch form (False) or this package's calls (True).
Sizes are the ones this repository's tests and benchmark use (hidden 4096 /
8192, intermediate 14336 / 28672, 32 or 64 query heads and 8 key/value heads
of 128 columns), with odd token counts beside them.
"""
import torch

own = False

FP8 = torch.float8_e4m3fn
BLOCK = 16
E2M1_MAX, E4M3_MAX = 6.0, 448.0


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the attention's output of one decoded token on its way into the next product
        dict(name="roundtrip_1x8192", op="roundtrip", T=1, n=8192, pitch=8192),
        # the same of prompts of odd total length, heads of a wider projected row
        dict(name="roundtrip_8191x4096", op="roundtrip", T=8191, n=4096, pitch=6144),
        # a down projection's weight, checked against its original
        dict(name="roundtrip_8192x28672", op="roundtrip", T=8192, n=28672, pitch=28672),
        # the qkv projection of one decoded token (hidden 4096, 32 + 2 * 8 heads of 128)
        dict(name="gemm_1x6144x4096", op="gemm", T=1, N=6144, K=4096),
        # the down projection of a decode batch
        dict(name="gemm_256x4096x14336", op="gemm", T=256, N=4096, K=14336),
        # the down projection of a long prompt of odd length
        dict(name="gemm_4093x8192x28672", op="gemm", T=4093, N=8192, K=28672),
        # the feed-forward block's first half for one decoded token
        dict(name="gated_1x14336x4096", op="gated", T=1, I=14336, K=4096),
        # the same for a decode batch of odd size at hidden 8192
        dict(name="gated_57x28672x8192", op="gated", T=57, I=28672, K=8192),
        # and for a chunk of a prompt
        dict(name="gated_1024x14336x4096", op="gated", T=1024, I=14336, K=4096),
        # the attention's output projection: a decode batch, and a long prompt
        dict(name="linear_33x8192x8192", op="linear", T=33, N=8192, K=8192),
        dict(name="linear_16384x4096x4096", op="linear", T=16384, N=4096, K=4096),
        # the feed-forward block of a prompt
        dict(name="ffn_4096x28672x8192", op="ffn", T=4096, I=28672, K=8192),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["roundtrip", "gemm", "gated", "linear", "ffn"])
    if op == "roundtrip":
        n = BLOCK * _log_int(rng, 4, 1792)
        T = _log_int(rng, 1, max(1, min(32768, 8192 * 28672 // n)))
        return dict(op=op, T=T, n=n, pitch=n + 8 * rng.choice([0, 0, 1, 50, 256]))
    K = 64 * _log_int(rng, 4, 448)
    T = _log_int(rng, 1, 8192)
    if op in ("gemm", "linear"):
        most = 4096 * 2 * 28672 * 8192 // (T * K)  # no more than the largest listed products
        return dict(op=op, T=T, N=8 * _log_int(rng, 16, max(16, min(3584, most // 8))), K=K)
    if op == "ffn":
        K = min(K, 8192)
    most = 4096 * 2 * 28672 * 8192 // (T * K)
    return dict(op=op, T=T, I=64 * _log_int(rng, 1, max(1, min(448, most // 128))), K=K)


# ------------------------------------------------------------------ the format, elementwise

def _e2m1(x):
    """Nearest E2M1 value, ties to the even code, saturating (x in any float type)."""
    a = x.abs().clamp_max(E2M1_MAX)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(x.dtype)
    return torch.copysign((a / step).round() * step, x)


def _e4m3(x):
    """Nearest E4M3 value of a non-negative x, ties to the even code, saturating."""
    a = x.clamp_max(E4M3_MAX)
    e = (torch.frexp(a).exponent - 1).clamp_min(-6) - 3
    step = ((e.long() + 1023) << 52).view(torch.float64).to(x.dtype)  # 2^e
    return (a / step).round() * step


def _quantised(x, gs):
    """(E2M1 values [T, n], E4M3 scale values [T, n / 16]) of x, in x's type."""
    T, n = x.shape
    b = x.reshape(T, n // BLOCK, BLOCK)
    sf = _e4m3(b.abs().amax(-1) * gs / E2M1_MAX)
    c = _e2m1(torch.where(sf[..., None] > 0, b * gs / sf[..., None], torch.zeros_like(b)))
    return c.view(T, n), sf


_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _packed(c):
    """Codes of E2M1 values, two a byte."""
    a = c.abs()
    code = torch.where(a <= 2, 2 * a, torch.where(a <= 4, a + 2, torch.full_like(a, 7)))
    code = (code + 8 * torch.signbit(c)).to(torch.uint8).view(c.shape[0], -1, 2)
    return code[..., 0] | (code[..., 1] << 4)


def _pairs():
    """The two E2M1 values of each byte, [256, 2]."""
    level = torch.tensor(_LEVELS + tuple(-v for v in _LEVELS), device="cuda")
    byte = torch.arange(256, device="cuda")
    return torch.stack([level[byte % 16], level[byte // 16]], 1)


def _values(q4, pairs):
    """E2M1 values [T, n] of packed codes [T, n / 2]."""
    return pairs[q4.int()].flatten(1)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)


def _rows(T, K, gen):
    """Activations: channels of different strength, as behind a norm's weight, and a few outliers."""
    x = torch.randn((T, K), generator=gen, device="cuda")
    x *= 1 + 0.5 * torch.randn((K,), generator=gen, device="cuda")
    x *= 1 + 20 * (torch.rand((T, K), generator=gen, device="cuda") < 0.001)
    return x


def _tensor_scale(x):
    """The tensor's scale: its largest value gets the largest block scale."""
    return (E4M3_MAX * E2M1_MAX / x.abs().max()).float().view(1)


def _activations(T, K, gen):
    x = _rows(T, K, gen)
    gs = _tensor_scale(x)
    c, sf = _quantised(x, gs)
    return _packed(c), sf.to(FP8), gs


def _weight(N, K, gen):
    """An [N, K] weight, quantised some rows at a time."""
    q = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda")
    sf = torch.empty((N, K // BLOCK), dtype=FP8, device="cuda")
    gs = torch.full((1,), E4M3_MAX * E2M1_MAX / 6 * K ** 0.5, device="cuda")  # six standard deviations
    for n0 in range(0, N, 4096):
        w = torch.randn((min(4096, N - n0), K), generator=gen, device="cuda") * K ** -0.5
        c, s = _quantised(w, gs)
        q[n0:n0 + 4096], sf[n0:n0 + 4096] = _packed(c), s.to(FP8)
    return q, sf, gs


def prepare(case, seed):
    gen = _gen(seed)
    s = dict(case)
    op = case["op"]
    s["pairs"] = _pairs()
    if op == "gated":  # a byte's two values in 8 bits each, as one number of 16
        s["pairs8"] = s["pairs"].to(FP8).view(torch.int16).view(256)
    if op == "roundtrip":
        T, n = case["T"], case["n"]
        s["x"] = torch.zeros((T, case["pitch"]), dtype=torch.bfloat16, device="cuda")[:, :n]
        s["x"].copy_(_rows(T, n, gen))
        s["gs"] = _tensor_scale(s["x"].float())
        return s
    T, K = case["T"], case["K"]
    if op == "linear":
        s["x"] = _rows(T, K, gen).to(torch.bfloat16)
        s["gs"] = _tensor_scale(s["x"].float())
    else:
        s["a"], s["a_scale"], s["gs"] = _activations(T, K, gen)
    s["w"], s["w_scale"], w_gs = _weight(case["N"] if op in ("gemm", "linear") else 2 * case["I"], K, gen)
    s["alpha"] = 1 / (s["gs"] * w_gs)
    if op in ("gated", "ffn"):
        # what is expected of the activation's largest values
        s["out_gs"] = torch.full((1,), E4M3_MAX * E2M1_MAX / 64, device="cuda")
    if op == "ffn":
        s["down"], s["down_scale"], down_gs = _weight(K, case["I"], gen)
        s["down_alpha"] = 1 / (s["out_gs"] * down_gs)
    return s


# ------------------------------------------------------------------ the plain forms

def _scaled(q4, sf, pairs):
    """Codes times their block scales, in 32 bits (exact: six significant bits)."""
    v = _values(q4, pairs)
    return (v.view(v.shape[0], -1, BLOCK) * sf.float()[..., None]).view(v.shape)


def _plain_product(s):
    pairs = s["pairs"]
    return s["alpha"] * (_scaled(s["a"], s["a_scale"], pairs) @ _scaled(s["w"], s["w_scale"], pairs).t())


def _plain_quantised(x, gs):
    """In 64 bits: next to a border 32 do not say on which side a value lies."""
    c, sf = _quantised(x.double(), gs.double())
    return c.float(), sf.float()


def _plain_gated(s):
    gu = _plain_product(s)
    g, u = gu[:, :s["I"]], gu[:, s["I"]:]
    return _quantised(g / (1 + torch.exp(-g)) * u, s["out_gs"])


def _plain(s):
    op = s["op"]
    if op == "roundtrip":
        c, sf = _plain_quantised(s["x"], s["gs"])
        v = c.view(s["T"], -1, BLOCK) * (sf / s["gs"])[..., None]
        return v.view(s["T"], s["n"]).to(torch.bfloat16), sf.to(FP8)
    if op == "gemm":
        return _plain_product(s).to(torch.bfloat16)
    if op == "linear":
        c, sf = _plain_quantised(s["x"], s["gs"])
        a = (c.view(s["T"], -1, BLOCK) * sf[..., None]).view(s["T"], s["K"])
        return (s["alpha"] * (a @ _scaled(s["w"], s["w_scale"], s["pairs"]).t())).to(torch.bfloat16)
    c, sf = _plain_gated(s)
    if op == "gated":
        return c.to(FP8), sf.to(FP8)
    y = (c.view(s["T"], -1, BLOCK) * sf[..., None]).view(s["T"], s["I"])
    return (s["down_alpha"] * (y @ _scaled(s["down"], s["down_scale"], s["pairs"]).t())).to(torch.bfloat16)


# ------------------------------------------------------------------ a pass

def run(state):
    s = state
    if not own:
        return _plain(s)
    import norm_activation_fp8_gb300 as vg
    op = s["op"]
    if op == "roundtrip":
        q4, sf = vg.nvfp4_quantize(s["x"], s["gs"])
        return vg.nvfp4_dequantize(q4, sf, s["gs"]), sf
    if op == "gemm":
        return vg.nvfp4_gemm(s["a"], s["a_scale"], s["w"], s["w_scale"], s["alpha"])
    if op == "linear":
        q4, sf = vg.nvfp4_quantize(s["x"], s["gs"])
        return vg.nvfp4_gemm(q4, sf, s["w"], s["w_scale"], s["alpha"])
    q4, sf = vg.nvfp4_gemm_silu_mul_nvfp4(s["a"], s["a_scale"], s["w"], s["w_scale"], s["alpha"],
                                          s["out_gs"])
    if op == "gated":
        return s["pairs8"][q4.int()].view(torch.uint8).view(FP8), sf
    return vg.nvfp4_gemm(q4, sf, s["down"], s["down_scale"], s["down_alpha"])


# ------------------------------------------------------------------ what a pass cannot do without

def _held(rows, n):
    """Bytes of an NVFP4 tensor."""
    return rows * n // 2 + rows * n // BLOCK


def work(case):
    T, op = case["T"], case["op"]
    if op == "roundtrip":
        n = case["n"]  # read, written in NVFP4, and that read and written in bf16
        return {"bytes": 4 * T * n + 2 * _held(T, n) + 4, "flops": 6 * T * n}
    K = case["K"]
    if op in ("gemm", "linear"):
        N = case["N"]
        read = _held(N, K) + (_held(T, K) if op == "gemm" else 2 * T * K + 2 * _held(T, K))
        return {"bytes": read + 2 * T * N + 4, "flops": 2 * T * N * K}
    I = case["I"]
    total = {"bytes": _held(T, K) + _held(2 * I, K) + _held(T, I) + 8, "flops": 4 * T * I * K}
    if op == "ffn":
        total["bytes"] += _held(T, I) + _held(K, I) + 2 * T * K
        total["flops"] += 2 * T * I * K
    return total


# ------------------------------------------------------------------ 64 bits, written apart

def _nearest(x, levels):
    """The nearest of ascending levels to a non-negative x, ties to the even place."""
    t = torch.tensor(levels, dtype=torch.float64, device=x.device)
    mid = (t[1:] + t[:-1]) / 2
    at = torch.searchsorted(mid, x.contiguous())  # how many midpoints lie below x
    here = at.clamp_max(len(levels) - 2)
    tie = (x == mid[here]) & (here % 2 == 1)
    return t[at + tie.long()]


def _e4m3_levels():
    sub = [m * 2.0 ** -9 for m in range(8)]
    return sub + [(8 + m) / 8 * 2.0 ** e for e in range(-6, 9) for m in range(8) if (e, m) != (8, 7)]


def _exact_quantised(y, gs):
    """Some rows at a time, y in 64 bits: (values, scales)."""
    T, n = y.shape
    values, scales = torch.empty_like(y), y.new_empty((T, n // BLOCK))
    rows = max(1, (1 << 25) // n)
    for t in range(0, T, rows):
        b = y[t:t + rows].reshape(-1, n // BLOCK, BLOCK)
        sf = _nearest(b.abs().max(-1).values.mul(gs).div(6.0), _e4m3_levels())
        scaled = b.mul(gs).div(sf.unsqueeze(-1))
        scaled[sf == 0] = 0
        values[t:t + rows] = (_nearest(scaled.abs(), _LEVELS) * scaled.sign()).view(-1, n)
        scales[t:t + rows] = sf
    return values, scales


def _exact_values(q4):
    q = q4.long()
    both = torch.stack([q & 15, q >> 4], -1).flatten(1)
    level = torch.tensor(_LEVELS, dtype=torch.float64, device=q4.device)[both & 7]
    return torch.where(both >= 8, -level, level)


def _exact_product(a, a_scale, w, w_scale, alpha):
    """a: 64-bit values and scales; w: codes, some rows at a time."""
    a = a * a_scale.double().repeat_interleave(BLOCK, 1)
    out = torch.empty((a.shape[0], w.shape[0]), dtype=torch.float64, device=a.device)
    for n in range(0, w.shape[0], 2048):
        b = _exact_values(w[n:n + 2048]) * w_scale[n:n + 2048].double().repeat_interleave(BLOCK, 1)
        out[:, n:n + 2048] = torch.mm(a, b.t())
    return out.mul_(alpha.double())


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "roundtrip":
        c, sf = _exact_quantised(s["x"].double(), s["gs"].double())
        return c * sf.repeat_interleave(BLOCK, 1) / s["gs"].double(), sf
    if op == "linear":
        a, a_scale = _exact_quantised(s["x"].double(), s["gs"].double())
    else:
        a, a_scale = _exact_values(s["a"]), s["a_scale"]
    p = _exact_product(a, a_scale, s["w"], s["w_scale"], s["alpha"])
    if op in ("gemm", "linear"):
        return p
    g, u = p[:, :case["I"]], p[:, case["I"]:]
    c, sf = _exact_quantised(torch.sigmoid(g) * g * u, s["out_gs"].double())
    if op == "gated":
        return c, sf
    return _exact_product(c, sf, s["down"], s["down_scale"], s["down_alpha"])
