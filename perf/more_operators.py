"""What stands around the absorbed attention in a layer: the operators' cases, plain forms and calls.

Four operators, in the order a layer runs them:

  quant   kv8_quant_blocks     rows to e4m3 with one f32 scale for each block of 128 columns, a root-mean-square
                               norm before it where asked for
  mm      kv8_matmul8          product of such rows with an fmt=8 weight (e4m3 with one f32 scale for each block
                               of 128 x 128); cache rows, with one scale a row, are multiplied as they lie
  rope    kv8_rope             rotary positions of a part of each head, interleaved or half layout, any frequencies;
                               the rotated part and the rest come apart, as the attention calls take them
  rows    kv8_norm_rope_rows   a projection's fresh rows to cache rows: norm of the latent part, rotation of the
                               key part, quantization, and the write to the rows' places in the cache

`own` False computes each in elementary torch operations (32 bits, 64 for the angles), True makes the library's
calls.
"""
import math

import torch

own = False

KL, KR, D = 512, 64, 576
BLK = 128
EPS = 1e-6
INTERLEAVED, HALF = 0, 1


def listed():
    return [
        # one sequence's next token
        {"name": "rows_1", "op": "rows", "n": 1, "pad": 0, "f32": False, "layout": INTERLEAVED, "factor": 1.0},
        # a batch's drafted tokens, cut out of a wider projection's f32 output
        {"name": "rows_1000_f32", "op": "rows", "n": 1000, "pad": 1472, "f32": True, "layout": HALF, "factor": 40.0},
        # a long prompt at once
        {"name": "rows_65536", "op": "rows", "n": 65536, "pad": 0, "f32": False, "layout": INTERLEAVED, "factor": 40.0},
        # the query heads of one token, and of a prompt's chunk
        {"name": "rope_1x128", "op": "rope", "n": 1, "H": 128, "width": 192, "at": 128, "dim": 64, "f32": False, "out32": False, "layout": INTERLEAVED, "factor": 1.0},
        {"name": "rope_8192x128", "op": "rope", "n": 8192, "H": 128, "width": 192, "at": 128, "dim": 64, "f32": False, "out32": False, "layout": HALF, "factor": 40.0},
        # a token's hidden state, normed, before its projections
        {"name": "quant_1x4096", "op": "quant", "n": 1, "width": 4096, "f32": False, "norm": True},
        # a chunk's head outputs (128 heads of 128, in f32), before the output projection
        {"name": "quant_8192x16384", "op": "quant", "n": 8192, "width": 16384, "f32": True, "norm": False},
        # the output projection of one token
        {"name": "mm_1", "op": "mm", "M": 1, "N": 4096, "K": 16384, "f32": False, "row_scale": False},
        # the query projection (128 heads of 192) of a batch's drafted tokens
        {"name": "mm_37", "op": "mm", "M": 37, "N": 24576, "K": 2048, "f32": False, "row_scale": False},
        # the latent rows' projection of a short prompt: ragged in every direction, f32 for the norm that follows
        {"name": "mm_1000_f32", "op": "mm", "M": 1000, "N": 576, "K": 4112, "f32": True, "row_scale": False},
        # cached rows expanded to 128 heads' keys and values, straight from the cache
        {"name": "mm_expand", "op": "mm", "M": 4096, "N": 32768, "K": 512, "f32": False, "row_scale": True},
        # the output projection of a prompt's chunk: the largest call
        {"name": "mm_8192", "op": "mm", "M": 8192, "N": 4096, "K": 16384, "f32": False, "row_scale": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rows", "rope", "quant", "mm", "mm", "mm"])
    if op == "rows":
        f32 = rng.random() < 0.4
        return {"op": op, "n": _log(rng, 1, 32768 if f32 else 65536), "pad": rng.choice([0, 0, 64, 1472]), "f32": f32,
                "layout": rng.choice([INTERLEAVED, HALF]), "factor": rng.choice([1.0, 4.0, 40.0])}
    if op == "rope":
        width, at, dim = rng.choice([(192, 128, 64), (192, 128, 64), (128, 0, 64), (64, 0, 64), (128, 64, 32), (96, 0, 96)])
        H = rng.choice([1, 8, 16, 20, 64, 100, 128])
        return {"op": op, "n": _log(rng, 1, max(1, min(65536, 8192 * 128 * 192 // (2 * H * width)))), "H": H, "width": width, "at": at, "dim": dim,
                "f32": rng.random() < 0.3, "out32": rng.random() < 0.3, "layout": rng.choice([INTERLEAVED, HALF]),
                "factor": rng.choice([1.0, 4.0, 40.0])}
    if op == "quant":
        return {"op": op, "n": _log(rng, 1, 8192), "width": 16 * _log(rng, 8, 1024), "f32": rng.random() < 0.5,
                "norm": rng.random() < 0.5}
    if rng.random() < 0.2:
        return {"op": op, "M": _log(rng, 1, 4096), "N": 256 * rng.choice([8, 16, 20, 64, 128]), "K": KL, "f32": False, "row_scale": True}
    while True:
        c = {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 32768), "K": 16 * _log(rng, 8, 1024),
             "f32": rng.random() < 0.3, "row_scale": False}
        if c["M"] * c["N"] * c["K"] <= 8192 * 4096 * 16384 and c["M"] * c["N"] <= 4096 * 32768 and c["N"] * c["K"] <= 32768 * 8192:
            return c


def work(case):
    op = case["op"]
    if op == "rows":
        return {"bytes": case["n"] * (D * (4 if case["f32"] else 2) + 4 + 8 + 580) + KL * 4 + KR * 2, "flops": case["n"] * 10 * D}
    if op == "rope":
        n = case["n"] * case["H"]
        return {"bytes": n * case["width"] * ((4 if case["f32"] else 2) + (4 if case["out32"] else 2)) + case["n"] * 4 + case["dim"] * 2,
                "flops": 3 * n * case["dim"]}
    if op == "quant":
        n, w = case["n"], case["width"]
        return {"bytes": n * w * (5 if case["f32"] else 3) + n * -(-w // BLK) * 4 + (w * 4 if case["norm"] else 0), "flops": 6 * n * w}
    M, N, K = case["M"], case["N"], case["K"]
    kb = -(-K // BLK)
    return {"bytes": M * K + N * K + 4 * (M if case["row_scale"] else M * kb) + 4 * -(-N // BLK) * kb + M * N * (4 if case["f32"] else 2),
            "flops": 2.0 * M * N * K}


# ------------------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------------------
def _randn(shape, g):
    return torch.randn(shape, device="cuda", generator=g)


def _freqs(dim, factor):
    """A rotation's frequencies (radians a position), slowed down by `factor` where a turn is longer than the context."""
    f = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    return torch.where(2 * math.pi / f > 4096, f / factor, f).float()


def _bytes_of(x, amax):
    return (x * (448.0 / amax)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _blocks_of_rows(x):
    """(e4m3 bytes [n][w], scales [blocks][n]) of f32 rows, one scale for each block of 128 columns."""
    n, w = x.shape
    kb = -(-w // BLK)
    y = torch.zeros((n, kb * BLK), device="cuda")
    y[:, :w] = x
    y = y.view(n, kb, BLK)
    amax = y.abs().amax(2, keepdim=True).clamp(min=1e-20)
    q = _bytes_of(y, amax).view(n, kb * BLK)[:, :w].contiguous()
    return q, (amax[..., 0] / 448.0).t().contiguous()


def _weight(N, K, g):
    """An fmt=8 weight: e4m3 bytes [N][K], scales [ceil(N/128)][ceil(K/128)]."""
    nb, kb = -(-N // BLK), -(-K // BLK)
    w8 = torch.empty((nb * BLK, kb * BLK), dtype=torch.uint8, device="cuda")
    scale = torch.empty((nb, kb), device="cuda")
    for a in range(0, nb, 32):
        m = min(32, nb - a)
        w = _randn((m, BLK, kb, BLK), g) * (0.02 * torch.exp2(_randn((m, 1, kb, 1), g)))
        amax = w.abs().amax((1, 3), keepdim=True)
        w8[a * BLK:(a + m) * BLK] = _bytes_of(w, amax).view(m * BLK, kb * BLK)
        scale[a:a + m] = amax[:, 0, :, 0] / 448.0
    return w8[:N, :K].contiguous(), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"op": op}
    if op in ("rows", "rope"):
        n, kind = case["n"], torch.float32 if case["f32"] else torch.bfloat16
        s["layout"], s["scale"] = case["layout"], 1.0 + 0.1 * math.log(case["factor"])
        s["position"] = torch.randint(0, 1 << 20, (n,), dtype=torch.int32, device="cuda", generator=g)
        s["inv_freq"] = _freqs(KR if op == "rows" else case["dim"], case["factor"])
    if op == "rows":
        wide = (_randn((n, D + case["pad"]), g) * torch.exp2(2 * _randn((n, 1), g))).to(kind)
        s["x"] = wide[:, case["pad"]:]  # the latent rows stand behind the other columns of the projection
        s["w"] = 1.0 + 0.2 * _randn((KL,), g)
        rows = n + n // 8 + 16
        s["dst"] = torch.randperm(rows, device="cuda", generator=g)[:n].contiguous()
        old = torch.randint(0, 127, (rows, D), dtype=torch.uint8, device="cuda", generator=g)
        s["kv8"], s["kv_scale"] = old, torch.rand(rows, device="cuda", generator=g)
        return s
    if op == "rope":
        H, width = case["H"], case["width"]
        s["at"], s["dim"], s["out"] = case["at"], case["dim"], torch.float32 if case["out32"] else torch.bfloat16
        s["x"] = _randn((n, H, width), g).to(kind)
        s["rot"] = torch.empty((n, H, case["dim"]), dtype=s["out"], device="cuda")
        s["rest"] = torch.empty((n, H, width - case["dim"]), dtype=s["out"], device="cuda")
        return s
    if op == "quant":
        n, w = case["n"], case["width"]
        s["x"] = _randn((n, w), g)
        s["x"] *= torch.exp2(_randn((1, w), g))  # channels of unlike size, as hidden states have them
        s["x"] = s["x"] if case["f32"] else s["x"].to(torch.bfloat16)
        s["w"] = 1.0 + 0.2 * _randn((w,), g) if case["norm"] else None
        s["q"] = torch.empty((n, w), dtype=torch.uint8, device="cuda")
        s["scale"] = torch.empty((-(-w // BLK), n), device="cuda")
        return s
    M, N, K = case["M"], case["N"], case["K"]
    if case["row_scale"]:  # rows of a cache: 512 of its 576 bytes, one scale a row
        x = _randn((M, D), g) * torch.exp2(_randn((M, 1), g))
        amax = x.abs().amax(1, keepdim=True)
        s["a8"], s["a_scale"] = _bytes_of(x, amax)[:, :K], (amax[:, 0] / 448.0).contiguous()
    else:
        s["a8"], s["a_scale"] = _blocks_of_rows(_randn((M, K), g) * torch.exp2(_randn((1, K), g)))
    s["w8"], s["w_scale"] = _weight(N, K, g)
    s["out"] = torch.empty((M, N), dtype=torch.float32 if case["f32"] else torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------------------
def run(state):
    return {"rows": _rows, "rope": _rope, "quant": _quant, "mm": _mm}[state["op"]](state)


def _rotated(x, position, inv_freq, scale, layout):
    """x [n][heads][dim] in f32, its pairs turned by position * inv_freq; the angles in 64 bits."""
    a = position.double()[:, None] * inv_freq.double()
    c, s = (torch.cos(a) * scale).float()[:, None], (torch.sin(a) * scale).float()[:, None]
    if layout == INTERLEAVED:
        u, v = x[..., 0::2], x[..., 1::2]
        return torch.stack([u * c - v * s, u * s + v * c], -1).flatten(-2)
    u, v = x.chunk(2, -1)
    return torch.cat([u * c - v * s, u * s + v * c], -1)


def _normed(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _rows(s):
    if own:
        import fp8_latent_kv_gb300 as kv
        kv.kv8_norm_rope_rows(s["x"], s["w"], EPS, s["position"], s["inv_freq"], s["dst"], s["kv8"], s["kv_scale"],
                              rope_scale=s["scale"], layout=s["layout"])
    else:
        x = s["x"].float()
        y = torch.cat([_normed(x[:, :KL], s["w"]), _rotated(x[:, None, KL:], s["position"], s["inv_freq"], s["scale"], s["layout"])[:, 0]], 1)
        amax = y.abs().amax(1, keepdim=True)
        s["kv8"][s["dst"]] = _bytes_of(y, amax)
        s["kv_scale"][s["dst"]] = amax[:, 0] / 448.0
    return s["kv8"].view(torch.float8_e4m3fn), s["kv_scale"]


def _rope(s):
    if own:
        import fp8_latent_kv_gb300 as kv
        kv.kv8_rope(s["x"], s["position"], s["inv_freq"], s["at"], s["rot"], s["rest"], rope_scale=s["scale"], layout=s["layout"])
    else:
        x, at, dim = s["x"], s["at"], s["dim"]
        s["rot"].copy_(_rotated(x[..., at:at + dim].float(), s["position"], s["inv_freq"], s["scale"], s["layout"]))
        s["rest"].copy_(torch.cat([x[..., :at], x[..., at + dim:]], -1))
    return s["rot"], s["rest"]


def _quant(s):
    if own:
        import fp8_latent_kv_gb300 as kv
        kv.kv8_quant_blocks(s["x"], s["q"], s["scale"], norm_w=s["w"], eps=EPS)
    else:
        x = s["x"].float()
        x = x if s["w"] is None else _normed(x, s["w"])
        n, w = x.shape
        kb = -(-w // BLK)
        y = torch.nn.functional.pad(x, (0, kb * BLK - w)).view(n, kb, BLK)
        amax = y.abs().amax(2, keepdim=True)
        s["q"].copy_(_bytes_of(y, torch.where(amax == 0, torch.full_like(amax, 448.0), amax)).view(n, kb * BLK)[:, :w])
        s["scale"].copy_((amax[..., 0] / 448.0).t())
    return s["q"].view(torch.float8_e4m3fn), s["scale"]


def _mm(s):
    if own:
        import fp8_latent_kv_gb300 as kv
        kv.kv8_matmul8(s["a8"], s["a_scale"], s["w8"], s["w_scale"], s["out"])
        return s["out"]
    a = s["a8"].view(torch.float8_e4m3fn).float()
    w = s["w8"].view(torch.float8_e4m3fn).float()
    (M, K), N = a.shape, w.shape[0]
    if s["a_scale"].dim() == 1:
        a *= s["a_scale"][:, None]
    else:
        a *= s["a_scale"].t().repeat_interleave(BLK, 1)[:, :K]
    w *= s["w_scale"].repeat_interleave(BLK, 0)[:N].repeat_interleave(BLK, 1)[:, :K]
    s["out"].copy_(a @ w.t())
    return s["out"]


# ------------------------------------------------------------------------------------------------------------
# the definition, in 64 bits
# ------------------------------------------------------------------------------------------------------------
def _nearest_e4m3(y):
    """The e4m3 value next to y, ties to even: steps of 2^-9 up to 2^-6, of an eighth of the power of two below |y| from there."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def _turned(x, case, position, inv_freq):
    """Each pair as a complex number, times e^(i position inv_freq) and the scale."""
    d = x.shape[-1]
    i, j = (slice(0, None, 2), slice(1, None, 2)) if case["layout"] == INTERLEAVED else (slice(0, d // 2), slice(d // 2, d))
    angle = (position.double()[:, None] * inv_freq.double())[:, None, :]
    z = torch.complex(x[..., i], x[..., j]) * torch.polar(torch.full_like(angle, 1.0 + 0.1 * math.log(case["factor"])), angle)
    out = torch.empty_like(x)
    out[..., i], out[..., j] = z.real, z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        x, at, dim = s["x"].double(), case["at"], case["dim"]
        keep = [k for k in range(case["width"]) if not at <= k < at + dim]
        return _turned(x[:, :, at:at + dim], case, s["position"], s["inv_freq"]), x[:, :, keep]
    if op == "rows":
        x = s["x"].double()
        kv8, scale = s["kv8"].view(torch.float8_e4m3fn).double(), s["kv_scale"].double()
        x[:, :KL] /= torch.sqrt(torch.square(x[:, :KL]).sum(1, keepdim=True) / KL + EPS)
        x[:, :KL] *= s["w"].double()
        x[:, KL:] = _turned(x[:, None, KL:], case, s["position"], s["inv_freq"])[:, 0]
        top = x.abs().max(1).values
        kv8[s["dst"]] = _nearest_e4m3(x * 448.0 / top[:, None])
        scale[s["dst"]] = top / 448.0
        return kv8, scale
    if op == "quant":
        x = s["x"].double()
        if case["norm"]:
            x /= torch.sqrt(torch.square(x).sum(1, keepdim=True) / case["width"] + EPS)
            x *= s["w"].double()
        scale = torch.empty_like(s["scale"], dtype=torch.float64)
        for k in range(scale.shape[0]):
            part = x[:, k * BLK:(k + 1) * BLK]
            top = part.abs().max(1).values
            scale[k] = top / 448.0
            part.copy_(_nearest_e4m3(part * (448.0 / top)[:, None]))
        return x, scale
    a, w = s["a8"].view(torch.float8_e4m3fn), s["w8"].view(torch.float8_e4m3fn)
    out = torch.zeros((case["M"], case["N"]), dtype=torch.float64, device="cuda")
    by_row = s["w_scale"].double().repeat_interleave(BLK, 0)[:case["N"]]
    for k in range(by_row.shape[1]):
        cols = slice(k * BLK, (k + 1) * BLK)
        sa = s["a_scale"] if case["row_scale"] else s["a_scale"][k]
        out.addmm_(a[:, cols].double() * sa.double()[:, None], (w[:, cols].double() * by_row[:, k:k + 1]).t())
    return out
