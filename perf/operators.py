"""Cases of the FP8 block-scaled products and the rotary / paged-cache operators.

Four operators around the fused norms and activations of a decoder layer:

  gemm    out = bf16(a w^T), a [T, K] and w [N, K] in FP8 e4m3 with one fp32
          scale per 128 columns of a row of a and per 128 x 128 block of w
  gated   the gated feed-forward projection: gate and up products as above,
          SiLU(gate) * up, and FP8 with one scale per 128 columns, in one call
  append  per-head RMSNorm of Q and K (or none), rotation, Q in place, K and V
          into a paged cache (bf16, or FP8 with static scales) at each token's slot
  mrope   per-head RMSNorm of Q and K and a rotation whose position depends on
          the pair (time, height, width), in place

``own`` selects the plain torch form (False) or this package's calls (True).
Sizes are the ones this repository's tests and benchmark use (hidden 4096 /
8192, intermediate 14336 / 28672, 32 or 64 query heads and 8 key/value heads
of 128 columns), with odd token counts beside them.
"""
import torch

own = False

FP8 = torch.float8_e4m3fn
BLOCK = 128
FP8_MAX = 448.0
EPS = 1e-6
MAX_POS = 32768


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the qkv projection of one decoded token (hidden 4096, 32 + 2 * 8 heads of 128)
        dict(name="gemm_1x6144x4096", op="gemm", T=1, N=6144, K=4096, colmajor=False),
        # the down projection of a decode batch, scales in the column-major layout
        dict(name="gemm_256x4096x14336", op="gemm", T=256, N=4096, K=14336, colmajor=True),
        # the down projection of a long prompt of odd length
        dict(name="gemm_4093x8192x28672", op="gemm", T=4093, N=8192, K=28672, colmajor=False),
        # the feed-forward block's first half for one decoded token
        dict(name="gated_1x14336x4096", op="gated", T=1, I=14336, K=4096, colmajor=False),
        # the same for a decode batch of odd size at hidden 8192
        dict(name="gated_57x28672x8192", op="gated", T=57, I=28672, K=8192, colmajor=False),
        # and for a chunk of a prompt, in both layouts' sizes
        dict(name="gated_2048x14336x4096", op="gated", T=2048, I=14336, K=4096, colmajor=True),
        dict(name="gated_4096x28672x8192", op="gated", T=4096, I=28672, K=8192, colmajor=False),
        # one decoded token: latency
        dict(name="append_1_bf16", op="append", T=1, Hq=32, Hkv=8, D=128, norm=True, neox=True,
             fp8=False, page=16, axes=1, interleaved=False),
        # a prompt with QK norm into a bf16 cache
        dict(name="append_32768_bf16", op="append", T=32768, Hq=32, Hkv=8, D=128, norm=True,
             neox=True, fp8=False, page=16, axes=1, interleaved=False),
        # a batch of prompts of odd total length into an FP8 cache, rotation only
        dict(name="append_8191_fp8", op="append", T=8191, Hq=64, Hkv=8, D=128, norm=False,
             neox=True, fp8=True, page=64, axes=1, interleaved=False),
        # a decode batch of a model that reads images: three position axes
        dict(name="mrope_64", op="mrope", T=64, Hq=32, Hkv=8, D=128, norm=True, neox=True,
             axes=3, interleaved=True),
        # a video prompt
        dict(name="mrope_16411", op="mrope", T=16411, Hq=32, Hkv=8, D=128, norm=True, neox=True,
             axes=3, interleaved=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["gemm", "gated", "append", "mrope"])
    if op in ("gemm", "gated"):
        T = _log_int(rng, 1, 8192)
        K = BLOCK * _log_int(rng, 4, 224)
        c = dict(op=op, T=T, K=K, colmajor=rng.random() < 0.5)
        # no more than the largest listed case's products
        most = 4096 * 2 * 28672 * 8192 // (T * K)
        if op == "gemm":
            c["N"] = 8 * _log_int(rng, 16, max(16, min(3584, most // 8)))
        else:
            c["I"] = BLOCK * _log_int(rng, 1, max(1, min(224, most // 256)))
        return c
    D = rng.choice([64, 128, 128, 256])
    T = _log_int(rng, 1, 32768 if D < 256 else 8192)
    c = dict(op=op, T=T, Hq=rng.choice([4, 8, 16, 28, 32]), Hkv=rng.choice([1, 2, 4, 8]), D=D,
             norm=rng.random() < 0.6, neox=rng.random() < 0.7, interleaved=rng.random() < 0.5)
    if op == "mrope":
        c["norm"], c["axes"] = True, rng.choice([2, 3, 3, 4])
        return c
    c.update(fp8=rng.random() < 0.5, page=rng.choice([1, 16, 64, 96, 128]), axes=rng.choice([1, 1, 3]))
    return c


def _sections(case):
    """How many of the D/2 pairs each axis turns: the first axis takes what the others leave."""
    half, axes = case["D"] // 2, case["axes"]
    if axes == 1:
        return None
    part = 3 * half // (4 * axes) if axes > 2 else half // 3
    return (half - part * (axes - 1),) + (part,) * (axes - 1)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)


def _quantised_rows(x, colmajor):
    """FP8 codes of x [T, K] with a scale per 128 columns, as the fused norm writes them."""
    T, K = x.shape
    g = x.view(T, K // BLOCK, BLOCK)
    s = g.abs().amax(-1).clamp_min(1e-10) / FP8_MAX
    q = (g / s[..., None]).clamp(-FP8_MAX, FP8_MAX).to(FP8).view(T, K)
    if not colmajor:
        return q, s.contiguous()
    out = torch.zeros((K // BLOCK, (T + 3) // 4 * 4), dtype=torch.float32, device=x.device)
    out[:, :T] = s.t()
    return q, out


def _quantised_weight(N, K, gen):
    """FP8 codes of an [N, K] weight and a scale per 128 x 128 block (the last block of rows may be short)."""
    nb, kb = (N + BLOCK - 1) // BLOCK, K // BLOCK
    q = torch.empty((N, K), dtype=FP8, device="cuda")
    s = torch.empty((nb, kb), dtype=torch.float32, device="cuda")
    step = 32 * BLOCK
    for n0 in range(0, N, step):
        rows = min(step, N - n0)
        full = (rows + BLOCK - 1) // BLOCK * BLOCK
        w = torch.randn((full, K), generator=gen, device="cuda") * K ** -0.5
        w[rows:] = 0
        b = w.view(full // BLOCK, BLOCK, kb, BLOCK)
        sb = b.abs().amax((1, 3)) / FP8_MAX
        s[n0 // BLOCK:n0 // BLOCK + full // BLOCK] = sb
        q[n0:n0 + rows] = (b / sb[:, None, :, None]).view(full, K)[:rows].clamp(-FP8_MAX, FP8_MAX).to(FP8)
    return q, s


def _rope_table(D):
    f = 1e6 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    a = torch.arange(MAX_POS, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    gen = _gen(seed)
    c = dict(case)
    if case["op"] in ("gemm", "gated"):
        T, K = case["T"], case["K"]
        x = torch.randn((T, K), generator=gen, device="cuda")
        # channels of different strength, as behind a norm's weight, and a few outliers
        x *= 1 + 0.5 * torch.randn((K,), generator=gen, device="cuda")
        x *= 1 + 20 * (torch.rand((T, K), generator=gen, device="cuda") < 0.001)
        c["a"], c["a_scale"] = _quantised_rows(x, case["colmajor"])
        c["w"], c["w_scale"] = _quantised_weight(case["N"] if case["op"] == "gemm" else 2 * case["I"], K, gen)
        return c
    T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
    bf = torch.bfloat16
    c["qkv"] = torch.randn((T, (Hq + 2 * Hkv) * D), generator=gen, device="cuda").to(bf)
    for name in ("q_weight", "k_weight"):
        w = (1 + 0.1 * torch.randn((D,), generator=gen, device="cuda")).to(bf)
        c[name] = w if case["norm"] else None
    c["table"] = _rope_table(D)
    c["sections"] = _sections(case)
    shape = (T,) if case["axes"] == 1 else (case["axes"], T)
    c["positions"] = torch.randint(0, MAX_POS, shape, generator=gen, device="cuda")
    if case["op"] == "append":
        page = case["page"]
        need = (T + page - 1) // page
        pages = need + need // 4 + 1
        # each run of `page` tokens fills a page of its own; pages lie anywhere in the cache
        where = torch.randperm(pages, generator=gen, device="cuda")[:need]
        t = torch.arange(T, device="cuda")
        c["slots"] = where[t // page] * page + t % page
        if T > 8:  # a padded batch: a few tokens that belong to no sequence
            c["slots"][torch.randint(0, T, (T // 64 + 1,), generator=gen, device="cuda")] = -1
        kind = FP8 if case["fp8"] else bf
        for name in ("k_cache", "v_cache"):
            old = torch.randn((pages, page, Hkv, D), generator=gen, device="cuda")
            c[name] = old.to(kind)
        c["k_scale"] = c["v_scale"] = None
        if case["fp8"]:
            c["k_scale"] = torch.tensor([0.03], device="cuda")
            c["v_scale"] = torch.tensor([0.02], device="cuda")
    return c


# ------------------------------------------------------------------ the plain forms

def _dequantised(s):
    T, K = s["a"].shape
    sa = s["a_scale"][:, :T].t() if s["colmajor"] else s["a_scale"]
    a = (s["a"].float().view(T, K // BLOCK, BLOCK) * sa[..., None]).view(T, K)
    N = s["w"].shape[0]
    sw = s["w_scale"].repeat_interleave(BLOCK, 0)[:N]
    w = (s["w"].float().view(N, K // BLOCK, BLOCK) * sw[..., None]).view(N, K)
    return a, w


def _plain_gemm(s):
    a, w = _dequantised(s)
    return (a @ w.t()).to(torch.bfloat16)


def _plain_gated(s):
    a, w = _dequantised(s)
    T, I = s["T"], s["I"]
    gu = a @ w.t()
    g, u = gu[:, :I], gu[:, I:]
    y = (g / (1 + torch.exp(-g)) * u).view(T, I // BLOCK, BLOCK)
    scale = y.abs().amax(-1).clamp_min(1e-10) / FP8_MAX
    q = (y / scale[..., None]).clamp(-FP8_MAX, FP8_MAX).to(FP8).view(T, I)
    return q, scale


def _axis_of_pair(s, device):
    """The axis that each of the D/2 pairs turns by."""
    half, axes, sec = s["D"] // 2, s["axes"], s["sections"]
    if sec is None:
        return torch.zeros(half, dtype=torch.long, device=device)
    i = torch.arange(half, device=device)
    counts = torch.tensor(sec, device=device)
    if s["interleaved"]:  # axes take turns; an axis that has had its share leaves its turns to the first
        return torch.where(i // axes < counts[i % axes], i % axes, 0)
    return torch.searchsorted(torch.cumsum(counts, 0), i, right=True)


def _turned(s, x, weight):
    """Norm (with a weight) and rotation of heads x [T, H, D], in 32 bits."""
    D = s["D"]
    x = x.float()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    pos = s["positions"].view(s["axes"], -1)
    p = pos[_axis_of_pair(s, x.device)].t()  # [T, D/2]
    i = torch.arange(D // 2, device=x.device)
    cos, sin = s["table"][p, i][:, None], s["table"][p, i + D // 2][:, None]
    if s["neox"]:
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _heads(s):
    T, Hq, Hkv, D = s["T"], s["Hq"], s["Hkv"], s["D"]
    h = s["qkv"].view(T, Hq + 2 * Hkv, D)
    return h[:, :Hq], h[:, Hq:Hq + Hkv], h[:, Hq + Hkv:]


def _plain_mrope(s):
    q, k, _ = _heads(s)
    q.copy_(_turned(s, q, s["q_weight"]).to(torch.bfloat16))
    k.copy_(_turned(s, k, s["k_weight"]).to(torch.bfloat16))
    return s["qkv"]


def _put(cache, at, x, scale):
    """Rows x into the cache's slots; the bytes are moved, whatever the cache's type."""
    if scale is not None:
        x = (x / scale).clamp(-FP8_MAX, FP8_MAX)
    cache.view(-1, *cache.shape[2:]).view(torch.uint8)[at] = x.to(cache.dtype).view(torch.uint8)


def _plain_append(s):
    q, k, v = _heads(s)
    live = (s["slots"] >= 0).nonzero().view(-1)
    at = s["slots"][live]
    _put(s["k_cache"], at, _turned(s, k, s["k_weight"])[live], s["k_scale"])
    _put(s["v_cache"], at, v[live].float(), s["v_scale"])
    q.copy_(_turned(s, q, s["q_weight"]).to(torch.bfloat16))
    return s["qkv"], s["k_cache"], s["v_cache"]


# ------------------------------------------------------------------ a pass

def run(state):
    s = state
    if not own:
        return {"gemm": _plain_gemm, "gated": _plain_gated, "mrope": _plain_mrope,
                "append": _plain_append}[s["op"]](s)
    import norm_activation_fp8_gb300 as vg
    layout = vg.COLUMN_MAJOR if s.get("colmajor") else 0
    if s["op"] == "gemm":
        return vg.fp8_block_gemm(s["a"], s["a_scale"], s["w"], s["w_scale"], layout)
    if s["op"] == "gated":
        return vg.fp8_block_gemm_silu_mul_fp8(s["a"], s["a_scale"], s["w"], s["w_scale"], layout)
    if s["op"] == "mrope":
        vg.vg_fused_qk_norm_mrope(s["qkv"], s["q_weight"], s["k_weight"], s["table"],
                                  s["positions"], s["sections"], s["Hq"], s["Hkv"], s["D"], EPS,
                                  s["neox"], s["interleaved"])
        return s["qkv"]
    vg.vg_fused_qk_norm_rope_append(s["qkv"], s["k_cache"], s["v_cache"], s["q_weight"],
                                    s["k_weight"], s["table"], s["positions"], s["slots"],
                                    s["Hq"], s["Hkv"], s["D"], EPS, s["neox"], s["sections"],
                                    s["interleaved"], s["k_scale"], s["v_scale"])
    return s["qkv"], s["k_cache"], s["v_cache"]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    T = case["T"]
    if case["op"] in ("gemm", "gated"):
        K = case["K"]
        N = case["N"] if case["op"] == "gemm" else 2 * case["I"]
        read = T * K + 4 * T * (K // BLOCK) + N * K + 4 * ((N + BLOCK - 1) // BLOCK) * (K // BLOCK)
        wrote = 2 * T * N if case["op"] == "gemm" else T * case["I"] + 4 * T * (case["I"] // BLOCK)
        return {"bytes": read + wrote, "flops": 2 * T * N * K}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    turned = (Hq + Hkv) * D
    meta = 8 * case["axes"] + 4 * D  # positions and the cos/sin values of a token
    if case["op"] == "mrope":
        return {"bytes": T * (4 * turned + meta) + 4 * D, "flops": 10 * T * turned}
    cache = 1 if case["fp8"] else 2
    per = 2 * (Hq + 2 * Hkv) * D + 2 * Hq * D + 2 * cache * Hkv * D + meta + 8
    return {"bytes": T * per + (4 * D if case["norm"] else 0), "flops": 10 * T * turned}


# ------------------------------------------------------------------ 64 bits, written apart

def _exact_product(s, n0, n1):
    """Rows n0..n1 of the weight: each 128-column block's sum of products, scaled, in 64 bits."""
    out = None
    T, K = s["a"].shape
    block_row = torch.arange(n0, n1, device="cuda") // BLOCK
    for b in range(K // BLOCK):
        cols = slice(b * BLOCK, (b + 1) * BLOCK)
        part = torch.mm(s["a"][:, cols].double(), s["w"][n0:n1, cols].double().t())
        sa = s["a_scale"][b, :T] if s["colmajor"] else s["a_scale"][:, b]
        part *= sa.double()[:, None]
        part *= s["w_scale"][block_row, b].double()[None, :]
        out = part if out is None else out.add_(part)
    return out


def _exact_turned(s, heads, weight):
    """One pair at a time: norm, then the complex product with cos + i sin of the pair's position."""
    x = heads.double()
    if weight is not None:
        x = x * (x.pow(2).sum(-1, keepdim=True) / s["D"] + EPS).rsqrt() * weight.double()
    half = s["D"] // 2
    out = torch.empty_like(x)
    pos = s["positions"].view(s["axes"], -1)
    sec = list(s["sections"] or (half,))
    for i in range(half):
        if not s["interleaved"] or len(sec) == 1:
            axis = next(j for j in range(len(sec)) if i < sum(sec[:j + 1]))
        else:
            axis = i % len(sec) if i // len(sec) < sec[i % len(sec)] else 0
        c = s["table"][pos[axis], i].double()[:, None]
        n = s["table"][pos[axis], half + i].double()[:, None]
        lo, hi = (i, half + i) if s["neox"] else (2 * i, 2 * i + 1)
        out[..., lo] = x[..., lo] * c - x[..., hi] * n
        out[..., hi] = x[..., hi] * c + x[..., lo] * n
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemm":
        return _exact_product(s, 0, case["N"])
    if case["op"] == "gated":
        I = case["I"]
        g, u = _exact_product(s, 0, I), _exact_product(s, I, 2 * I)
        y = (torch.sigmoid(g) * g * u).view(case["T"], I // BLOCK, BLOCK)
        scale = torch.clamp(y.abs().amax(-1), min=1e-10) / FP8_MAX
        return (y / scale.unsqueeze(-1)).view(case["T"], I), scale
    T, Hq, Hkv, D = (case[k] for k in ("T", "Hq", "Hkv", "D"))
    qkv = s["qkv"].double().view(T, Hq + 2 * Hkv, D)
    q, k = _exact_turned(s, qkv[:, :Hq], s["q_weight"]), _exact_turned(s, qkv[:, Hq:Hq + Hkv], s["k_weight"])
    v = qkv[:, Hq + Hkv:]
    if case["op"] == "mrope":
        return torch.cat([q, k, v], 1).view(T, -1)
    caches = []
    keep = s["slots"] >= 0
    for cache, x, scale in ((s["k_cache"], k, s["k_scale"]), (s["v_cache"], v, s["v_scale"])):
        full = cache.double().view(-1, Hkv, D)
        if scale is not None:
            x = torch.clamp(x / scale.double(), -FP8_MAX, FP8_MAX)
        full[s["slots"][keep]] = x[keep]
        caches.append(full.view(cache.shape))
    return torch.cat([q, qkv[:, Hq:]], 1).view(T, -1), caches[0], caches[1]
