"""The operators of a layer in low precision, as cases to time and compare:

  rmsnorm       h = x + residual; y = h / sqrt(mean(h^2) + eps) * gamma
  rmsnorm_mx8   the same, y as MXFP8 (E4M3 codes, one E8M0 scale per 32 columns)
  mx4_quantize  bf16 rows to MXFP4 (E2M1 codes, two a byte, one E8M0 scale per
                32 columns) and back to the values they stand for
  linear_mx4    y = epilogue(A W^T + bias) of two MXFP4 matrices
  rope3d        rotary positions over (time, row, column) on the heads of a
                token, rows of a wider tensor

With ``own`` false ``run`` computes them from elementary torch operations, with
``own`` true through this package.  ``exact`` computes them in 64 bits.
"""
import functools
import math

import torch

own = False

EPS = 1e-6
THETA = 10000.0
GROUP = 32        # elements that share a scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # the magnitudes of codes 0..7; bit 3 is the sign


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token of a 1152-wide layer: latency
        {"name": "rmsnorm 1 row", "op": "rmsnorm", "rows": 1, "cols": 1152, "dtype": "bf16", "residual": True},
        # a small fp32 layer without a residual
        {"name": "rmsnorm fp32", "op": "rmsnorm", "rows": 256, "cols": 256, "dtype": "f32", "residual": False},
        # five images packed into one batch
        {"name": "rmsnorm packed", "op": "rmsnorm", "rows": 10936, "cols": 1152, "dtype": "bf16", "residual": True},
        # the norm in front of an 8-bit projection, one image of 3900 patches
        {"name": "rmsnorm_mx8 image", "op": "rmsnorm_mx8", "rows": 3900, "cols": 1152},
        # the wide rows of 2x2-merged tokens
        {"name": "rmsnorm_mx8 merged", "op": "rmsnorm_mx8", "rows": 975, "cols": 4608},
        # a small image's activations
        {"name": "mx4_quantize small", "op": "mx4_quantize", "rows": 960, "cols": 1152},
        # the MLP's hidden activations of the packed batch
        {"name": "mx4_quantize packed", "op": "mx4_quantize", "rows": 10936, "cols": 4304},
        # one token through the QKV projection: the weight is what is read
        {"name": "linear_mx4 1 row", "op": "linear_mx4", "M": 1, "N": 3456, "K": 1152, "epi": "bias"},
        # fc1 of the 3900-patch image
        {"name": "linear_mx4 fc1", "op": "linear_mx4", "M": 3900, "N": 4304, "K": 1152, "epi": "gelu"},
        # fc2 of the packed batch, a ragged K
        {"name": "linear_mx4 fc2 packed", "op": "linear_mx4", "M": 10936, "N": 1152, "K": 4304, "epi": "residual"},
        # four frames of 24 x 37 patches, heads of 72 in three blocks
        {"name": "rope3d clip", "op": "rope3d", "frames": 4, "rows": 24, "cols": 37, "heads": 32, "head_dim": 72,
         "sections": "12,12,12", "layout": "blocks", "dtype": "bf16"},
        # a longer clip, heads of 128, frequencies shared out by sections
        {"name": "rope3d video", "op": "rope3d", "frames": 16, "rows": 32, "cols": 32, "heads": 32, "head_dim": 128,
         "sections": "16,24,24", "layout": "sections", "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rmsnorm", "rmsnorm_mx8", "mx4_quantize", "linear_mx4", "linear_mx4", "rope3d"])
    if op == "rmsnorm":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        cols = 8 * _log(rng, 8, 1024)
        rows = _log(rng, 1, min(16000, 24_000_000 // cols))
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "residual": rng.random() < 0.6}
    if op == "rmsnorm_mx8":
        cols = 8 * _log(rng, 8, 1024)
        return {"op": op, "rows": _log(rng, 1, min(16000, 24_000_000 // cols)), "cols": cols}
    if op == "mx4_quantize":
        cols = _log(rng, 33, 6000)
        return {"op": op, "rows": _log(rng, 1, min(16000, 40_000_000 // cols)), "cols": cols}
    if op == "linear_mx4":
        N, K = 8 * _log(rng, 8, 640), _log(rng, 33, 5000)
        return {"op": op, "M": _log(rng, 1, min(10936, 50_000_000_000 // (N * K))), "N": N, "K": K,
                "epi": rng.choice(["bias", "gelu", "residual"])}
    frames, rows, cols = _log(rng, 1, 24), rng.randint(1, 32), rng.randint(1, 32)
    head_dim, sections = rng.choice([(64, "8,12,12"), (72, "12,12,12"), (72, "10,13,13"), (128, "16,24,24"), (128, "24,20,20")])
    heads = _log(rng, 1, max(1, min(32, 40_000_000 // (frames * rows * cols * head_dim))))
    return {"op": op, "frames": frames, "rows": rows, "cols": cols, "heads": heads,
            "head_dim": head_dim, "sections": sections, "layout": rng.choice(["blocks", "sections", "turns"]),
            "dtype": "f32" if head_dim == 64 else rng.choice(["bf16", "bf16", "f32"])}


def work(case):
    op = case["op"]
    if op in ("rmsnorm", "rmsnorm_mx8"):
        rows, cols = case["rows"], case["cols"]
        n = rows * cols
        if op == "rmsnorm":
            es = 2 if case["dtype"] == "bf16" else 4
            return {"bytes": n * es * (4 if case["residual"] else 2) + cols * es, "flops": 4 * n}
        return {"bytes": n * 7 + rows * -(-cols // GROUP) + cols * 2, "flops": 6 * n}  # x, residual, h: 2 each; a code: 1
    if op == "mx4_quantize":
        n = case["rows"] * case["cols"]
        # x and the values in bf16, the codes written and read
        return {"bytes": n * 4 + 2 * (n / 2 + case["rows"] * -(-case["cols"] // GROUP)), "flops": 4 * n}
    if op == "linear_mx4":
        M, N, K = case["M"], case["N"], case["K"]
        b = (M + N) * (K / 2 + -(-K // GROUP)) + 2 * N + 2 * M * N * (2 if case["epi"] == "residual" else 1)
        return {"bytes": b, "flops": 2 * M * N * K}
    T = case["frames"] * case["rows"] * case["cols"]
    n = T * case["heads"] * case["head_dim"]
    return {"bytes": 2 * n * (2 if case["dtype"] == "bf16" else 4) + 12 * T, "flops": 3 * n}


# ---------------------------------------------------------------- inputs
def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _scale_bytes(rows, K):
    return -(-rows // 128) * -(-K // 128) * 512


def _activations(gen, rows, cols, dtype):
    """Rows of a residual stream: normal values, every row of its own size, and some columns that stand out."""
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    x *= torch.exp2(torch.rand(rows, 1, device="cuda", generator=gen) * 4 - 2)
    x *= 1 + 7 * (torch.rand(cols, device="cuda", generator=gen) < 0.01)
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op in ("rmsnorm", "rmsnorm_mx8"):
        rows, cols = case["rows"], case["cols"]
        dtype = _dtype(case.get("dtype"))
        s["x"] = _activations(gen, rows, cols, dtype)
        s["gamma"] = (1 + 0.1 * torch.randn(cols, device="cuda", generator=gen)).to(dtype)
        s["res"] = _activations(gen, rows, cols, dtype) if case.get("residual", True) else None
        s["h"] = torch.empty_like(s["x"]) if s["res"] is not None else None
        if op == "rmsnorm":
            s["y"] = torch.empty_like(s["x"])
        else:
            s["codes"] = torch.empty(rows, -(-cols // 16) * 16, dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty(_scale_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    elif op == "mx4_quantize":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _activations(gen, rows, cols, torch.bfloat16)
        s["codes"] = torch.empty(rows, -(-cols // 32) * 16, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(_scale_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        s["y"] = torch.empty_like(s["x"])
    elif op == "linear_mx4":
        M, N, K = case["M"], case["N"], case["K"]
        s["a"] = _packed(*_codes(_activations(gen, M, K, torch.bfloat16)))
        s["w"] = _packed(*_codes((0.02 * torch.randn(N, K, device="cuda", generator=gen)).to(torch.bfloat16)))
        s["bias"] = (0.01 * torch.randn(N, device="cuda", generator=gen)).to(torch.bfloat16)
        s["res"] = torch.randn(M, N, device="cuda", generator=gen).to(torch.bfloat16) if case["epi"] == "residual" else None
        s["y"] = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    else:
        T, H, d = case["frames"] * case["rows"] * case["cols"], case["heads"], case["head_dim"]
        # heads that are rotated (queries and keys), and half as many behind them that are not (values)
        wide = torch.randn(T, H + -(-H // 2), d, device="cuda", generator=gen).to(_dtype(case["dtype"]))
        s["x"] = wide[:, :H]
        s["y"] = torch.empty(T, H, d, dtype=wide.dtype, device="cuda")
        t, r, c = (torch.arange(n, dtype=torch.int32, device="cuda") for n in (case["frames"], case["rows"], case["cols"]))
        s["pos"] = torch.cartesian_prod(t + seed % 1000, r, c).reshape(T, 3).contiguous()  # a clip from the middle of a film
    return s


# ---------------------------------------------------------------- plain forms
def _place(rows, groups, device):
    """Where the scale of (row, group) stands: blocks of 128 rows x 4 groups, 512 bytes each."""
    r = torch.arange(rows, device=device)[:, None]
    g = torch.arange(groups, device=device)[None, :]
    blocks = -(-groups // 4)
    return ((r // 128) * blocks + g // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + g % 4


def _grouped(x):
    rows, K = x.shape
    return torch.nn.functional.pad(x, (0, -K % GROUP)).reshape(rows, -1, GROUP)


def _power(e):
    """2^e in 32 bits for whole -127 < e < 128 (0 for -127: only an all-zero group has it)."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _exponent(g, top):
    """The shared exponent of each group: floor(log2(largest magnitude)) - top, -127 for an all-zero group."""
    amax = g.abs().amax(-1, keepdim=True).to(torch.float32)
    e = (amax.view(torch.int32) >> 23) - 127 - top
    return torch.where(amax > 0, e.clamp(-127, 127), -127)


def _e2m1(a):
    """Magnitudes rounded to the nearest E2M1 value, ties to even, at most 6."""
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(a / step) * step).clamp_max(6)


def _codes(x):
    """bf16 rows as E2M1 codes (one a byte) and the exponents of their groups."""
    g = _grouped(x.to(torch.float32))
    e = _exponent(g, 2)
    v = _e2m1(g.abs() * _power(-e))
    code = torch.bucketize(v, torch.tensor(E2M1, device=x.device)) | (torch.signbit(g).to(torch.int64) << 3)
    return code.reshape(x.shape[0], -1)[:, : x.shape[1]], e[..., 0]


def _packed(code, e):
    """Codes two a byte (the lower nibble first, rows of a multiple of 16 bytes) and scale bytes at their places."""
    rows, K = code.shape
    c = torch.nn.functional.pad(code, (0, -K % 32)).to(torch.uint8)
    scales = torch.full((_scale_bytes(rows, K),), 127, dtype=torch.uint8, device=code.device)
    scales[_place(rows, e.shape[1], code.device)] = (e + 127).to(torch.uint8)
    return c[:, 0::2] | (c[:, 1::2] << 4), scales


def _unpacked(packed, K):
    """The values that packed codes and scales stand for, in 32 bits."""
    codes, scales = packed
    rows = codes.shape[0]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = table[torch.stack((codes & 15, codes >> 4), -1).reshape(rows, -1).to(torch.int32)]
    e = scales[_place(rows, -(-K // GROUP), codes.device)].to(torch.int32) - 127
    return (v.reshape(rows, -1, GROUP) * _power(e)[..., None]).reshape(rows, -1)[:, :K]


def _norm(x, res, gamma, wide):
    """The sum as it is stored, and its normalised rows in the wide type."""
    h = x if res is None else (x.to(torch.float32) + res.to(torch.float32)).to(x.dtype)
    v = h.to(wide)
    return h, v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS) * gamma.to(wide)


def _to_mx8(y):
    """bf16 rows as E4M3 values and E8M0 scales at their places."""
    rows, K = y.shape
    g = _grouped(y.to(torch.float32))
    e = _exponent(g, 8)
    q = (g * _power(-e)).clamp(-448, 448).reshape(rows, -1)[:, :K].to(torch.float8_e4m3fn)
    scales = torch.full((_scale_bytes(rows, K),), 127, dtype=torch.uint8, device=y.device)
    scales[_place(rows, e.shape[1], y.device)] = (e[..., 0] + 127).to(torch.uint8)
    return q, scales.view(torch.float8_e8m0fnu)


def _pairs(head_dim, sections, layout):
    """For each rotated pair of a head: its first dim, its second, its axis and its frequency."""
    sec = [int(v) for v in sections.split(",")]
    pairs, at = [], 0
    if layout == "blocks":
        for axis, n in enumerate(sec):
            pairs += [(at + j, at + n + j, axis, THETA ** (-j / n)) for j in range(n)]
            at += 2 * n
        return pairs
    half = head_dim // 2
    if layout == "sections":
        axes = [a for a, n in enumerate(sec) for _ in range(n)]
    else:  # the axes take turns while they have frequencies left
        left, axes = list(sec), []
        while len(axes) < half:
            for a in range(3):
                if left[a]:
                    axes.append(a)
                    left[a] -= 1
    return [(j, j + half, axes[j], THETA ** (-2 * j / head_dim)) for j in range(half)]


@functools.lru_cache(maxsize=None)
def _tables(head_dim, sections, layout):
    """_pairs() as tensors on the GPU."""
    lo, hi, axis, freq = zip(*_pairs(head_dim, sections, layout))
    return (torch.tensor(lo, device="cuda"), torch.tensor(hi, device="cuda"), torch.tensor(axis, device="cuda"),
            torch.tensor(freq, dtype=torch.float64, device="cuda"))


def _plain(s):
    op = s["op"]
    if op == "rmsnorm":
        h, y = _norm(s["x"], s["res"], s["gamma"], torch.float32)
        return {"y": y.to(h.dtype)} if s["res"] is None else {"h": h, "y": y.to(h.dtype)}
    if op == "rmsnorm_mx8":
        h, y = _norm(s["x"], s["res"], s["gamma"], torch.float64)  # codes next to a border
        codes, scales = _to_mx8(_to_bf16(y))
        return {"h": h, "codes": codes, "scales": scales}
    if op == "mx4_quantize":
        g = _grouped(s["x"].to(torch.float32))
        e = _exponent(g, 2)
        v = _e2m1(g.abs() * _power(-e)) * _power(e)
        return {"values": torch.copysign(v, g).reshape(g.shape[0], -1)[:, : s["cols"]].to(torch.bfloat16)}
    if op == "linear_mx4":
        y = _unpacked(s["a"], s["K"]) @ _unpacked(s["w"], s["K"]).T + s["bias"].to(torch.float32)
        if s["epi"] == "gelu":
            y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
        elif s["epi"] == "residual":
            y = y + s["res"].to(torch.float32)
        return {"y": y.to(torch.bfloat16)}
    lo, hi, axis, freq = _tables(s["head_dim"], s["sections"], s["layout"])
    angle = s["pos"].to(torch.float64)[:, axis] * freq  # far positions: 64 bits
    c, n = torch.cos(angle).to(torch.float32)[:, None], torch.sin(angle).to(torch.float32)[:, None]
    x = s["x"].to(torch.float32)
    a, b = x[..., lo], x[..., hi]
    y = torch.empty_like(x)
    y[..., lo] = a * c - b * n
    y[..., hi] = b * c + a * n
    return {"y": y.to(s["x"].dtype)}


def _to_bf16(v):
    """64-bit values rounded once to bf16: by way of 32 bits a value next to a border would be rounded twice."""
    f = v.to(torch.float32)
    bits = f.view(torch.int32)
    back = f.to(torch.float64).abs()
    tie = (bits & 0xFFFF) == 0x8000
    bits = bits + torch.where(tie & (v.abs() > back), 1, 0) - torch.where(tie & (v.abs() < back), 1, 0)
    return bits.to(torch.int32).view(torch.float32).to(torch.bfloat16)


# ---------------------------------------------------------------- this package
@functools.lru_cache(maxsize=None)
def _context(head_dim, dtype):
    import vision_transformer_encoder_layernorm_b200 as vit
    heads = 16
    return vit, vit.Context(heads * head_dim, heads, head_dim, 4304, vit.F32 if dtype == "f32" else vit.BF16, ln_eps=EPS, rope_theta=THETA)


def _own(s):
    op = s["op"]
    vit, ctx = _context(s.get("head_dim", 72), s.get("dtype", "bf16"))
    if op == "rmsnorm":
        ctx.rmsnorm(s["x"], s["gamma"], s["y"], residual=s["res"], h=s["h"])
        return {"y": s["y"]} if s["res"] is None else {"h": s["h"], "y": s["y"]}
    if op == "rmsnorm_mx8":
        ctx.rmsnorm_mx8(s["x"], s["gamma"], s["codes"], s["scales"], residual=s["res"], h=s["h"])
        return {"h": s["h"], "codes": s["codes"].view(torch.float8_e4m3fn)[:, : s["cols"]], "scales": s["scales"].view(torch.float8_e8m0fnu)}
    if op == "mx4_quantize":
        ctx.mx4_quantize(s["x"], s["codes"], s["scales"])
        ctx.mx4_dequantize(s["codes"], s["scales"], s["y"])
        return {"values": s["y"]}
    if op == "linear_mx4":
        epi = {"bias": vit.EPI_BIAS, "gelu": vit.EPI_BIAS_GELU, "residual": vit.EPI_BIAS_RESIDUAL}[s["epi"]]
        ctx.linear_mx4(s["a"], s["w"], s["bias"], s["y"], s["K"], epi=epi, residual=s["res"])
        return {"y": s["y"]}
    layout = {"blocks": vit.ROPE_BLOCKS, "sections": vit.ROPE_SECTIONS, "turns": vit.ROPE_TURNS}[s["layout"]]
    ctx.rope3d(s["x"], s["pos"], tuple(int(v) for v in s["sections"].split(",")), layout, out=s["y"])
    return {"y": s["y"]}


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---------------------------------------------------------------- 64 bits
def _nearest(v, grid):
    """The nearest value of a sorted grid, ties to the entry with an even index."""
    g = torch.tensor(grid, dtype=torch.float64, device=v.device)
    mid = (g[1:] + g[:-1]) / 2
    below, upto = torch.searchsorted(mid, v.contiguous(), right=False), torch.searchsorted(mid, v.contiguous(), right=True)
    return g[torch.where(below % 2 == 0, below, upto)]


def _group_power(v, top):
    m = v.abs().amax(-1, keepdim=True)
    e = torch.frexp(m).exponent - 1 - top  # a logarithm may be off where m is a power of two
    return torch.ldexp(torch.ones_like(m), torch.where(m > 0, e.clamp(-127, 127), -127))


def _groups64(v):
    rows, K = v.shape
    full = torch.zeros(rows, -(-K // GROUP) * GROUP, dtype=torch.float64, device=v.device)
    full[:, :K] = v
    return full.view(rows, -1, GROUP)


def _e4m3_grid():
    return [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rmsnorm", "rmsnorm_mx8"):
        x = s["x"].double()
        total = x if s["res"] is None else x + s["res"].double()
        # the norm is that of the sum as the type holds it
        h = total if s["x"].dtype == torch.float32 else total.to(torch.float32).to(torch.bfloat16).double()
        if s["x"].dtype == torch.float32 and s["res"] is not None:
            h = total.to(torch.float32).double()
        y = h * s["gamma"].double() * torch.rsqrt(h.square().sum(-1, keepdim=True) / case["cols"] + EPS)
        if op == "rmsnorm":
            return {"y": y} if s["res"] is None else {"h": total, "y": y}
        # bf16 in between: 8 significant bits, ties to even
        unit = torch.ldexp(torch.ones_like(y), torch.frexp(y).exponent - 8)
        g = _groups64(torch.round(y / unit) * unit)
        p = _group_power(g, 8)
        q = _nearest((g / p).abs(), _e4m3_grid()) * torch.sign(g)
        rows, groups = p.shape[:2]
        laid = torch.ones(-(-rows // 128), 32, 4, -(-groups // 4), 4, dtype=torch.float64, device=p.device)  # block row, r0, r1, block, group
        at = torch.arange(rows, device=p.device)
        for j in range(groups):
            laid[at // 128, at % 32, at // 32 % 4, j // 4, j % 4] = p[:, j, 0]
        return {"h": total, "codes": q.reshape(rows, -1)[:, : case["cols"]], "scales": laid.permute(0, 3, 1, 2, 4).reshape(-1)}
    if op == "mx4_quantize":
        g = _groups64(s["x"].double())
        p = _group_power(g, 2)
        v = _nearest((g / p).abs(), E2M1) * torch.sign(g) * p
        return {"values": v.reshape(case["rows"], -1)[:, : case["cols"]]}
    if op == "linear_mx4":
        M, N, K = case["M"], case["N"], case["K"]
        a, w = _decode64(s["a"], M, K), _decode64(s["w"], N, K)
        y = torch.addmm(s["bias"].double(), a, w.t())
        if case["epi"] == "gelu":
            y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))  # (1 + tanh u) / 2
        elif case["epi"] == "residual":
            y += s["res"].double()
        return {"y": y}
    d = case["head_dim"]
    z = s["x"].double()
    y = torch.empty_like(z)
    pos = s["pos"].double()
    for lo, hi, axis, freq in _pairs(d, case["sections"], case["layout"]):
        turn = torch.polar(torch.ones_like(pos[:, axis]), pos[:, axis] * freq)[:, None]
        r = torch.complex(z[..., lo], z[..., hi]) * turn
        y[..., lo], y[..., hi] = r.real, r.imag
    return {"y": y}


def _decode64(packed, rows, K):
    codes, scales = (t.long() for t in packed)
    out = torch.empty(rows, 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    for half, c in ((0, codes % 16), (1, codes // 16)):
        m, e = c % 2, c // 2 % 4
        v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * (1 << e) / 2)
        out[:, half::2] = torch.where(c >= 8, -v, v)
    blocks = -(-K // 128)
    p = scales.view(-1, blocks, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, 4 * blocks)[:rows]  # rows r1, r0; groups block, j
    p = torch.ldexp(torch.ones_like(out[:, :1]), p - 127).repeat_interleave(GROUP, dim=1)
    return out[:, :K] * p[:, :K]
