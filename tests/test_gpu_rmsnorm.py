"""vit_rmsnorm and vit_rmsnorm_mx8 against the fp64 definition.

bf16: h is the fp32 sum rounded once and y the correctly rounded value of the
formula for that h, so both are compared bit for bit (the fp64 reference is
within 2^-50 of the formula; a bf16 border that close does not occur here).
MXFP8 codes and scales are those of that y: bit for bit.  fp32: y is three
roundings from the formula (1/rms, and two products), each at most 2^-24
relative."""
import numpy as np
import pytest
import torch

import synth
from oracle import mxfp8_ref as MX
from oracle import norm_rope_ref as NR
from tests.gpu_util import from_dev, to_dev
from tests.test_gpu_mx8 import _scale_index
from tests.test_zzz_guard_bands import Band

pytestmark = pytest.mark.gpu

vit = pytest.importorskip("vision_transformer_encoder_layernorm_b200")
EPS = 1e-6


@pytest.fixture(scope="module", params=["bf16", "f32"])
def any_ctx(request):
    c = vit.Context(1152, 16, 72, 4304, vit.BF16 if request.param == "bf16" else vit.F32)
    c.name = request.param
    yield c
    c.close()


@pytest.fixture(scope="module")
def ctx():
    c = vit.Context(1152, 16, 72, 4304, vit.BF16)
    yield c
    c.close()


def rows_of(rows, cols, seed, dtype):
    """Rows of very different sizes, one of zeros, one with a single large value."""
    g = np.random.Generator(np.random.PCG64(seed))
    a = g.standard_normal((rows, cols)) * np.exp2(g.integers(-20, 20, (rows, 1)))
    if rows > 2:
        a[1] = 0
        a[2, cols // 2] = 2.0 ** 60
    return store(a, dtype)


def store(a, dtype):
    return to_dev(synth.round_bf16_bits(a) if dtype == "bf16" else a.astype(np.float32), dtype)


bf16_of = NR.to_bf16


def summed(x, r):
    """The stored sum: fp32, then the type."""
    return (x.float() + r.float()).to(x.dtype)


SHAPES = [(1, 8), (1, 1152), (5, 200), (129, 512), (257, 1152), (300, 1280), (33, 1288), (70, 3080),
          (12, 4608), (9, 5128), (3, 16384), (2, 8192),
          (3000, 1152), (3000, 64), (700, 4616), (600, 16384)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_rmsnorm(any_ctx, rows, cols, residual):
    dt = any_ctx.name
    x, r = rows_of(rows, cols, rows + cols, dt), rows_of(rows, cols, rows + cols + 1, dt)
    gamma = store(1 + 0.1 * np.random.Generator(np.random.PCG64(7)).standard_normal(cols), dt)
    tt = torch.bfloat16 if dt == "bf16" else torch.float32
    y, h = Band((rows, cols), tt), Band((rows, cols), tt)
    any_ctx.rmsnorm(x, gamma, y.t, residual=r if residual else None, h=h.t, eps=EPS)
    y.check("y"), h.check("h")
    want_h = summed(x, r) if residual else x
    assert torch.equal(h.t, want_h)
    ref = NR.rmsnorm(from_dev(want_h), from_dev(gamma), float(np.float32(EPS)))
    got = from_dev(y.t)
    if dt == "bf16":
        assert np.array_equal(got, bf16_of(ref))
    else:
        assert np.all(np.abs(got - ref) <= 3.01 * 2.0 ** -24 * np.abs(ref) + 2.0 ** -148)
    # without h, the same y
    y2 = torch.empty_like(x)
    any_ctx.rmsnorm(x, gamma, y2, residual=r if residual else None, eps=EPS)
    assert torch.equal(y2, y.t)
    assert any_ctx.device_status() == 0


def test_rmsnorm_in_place(any_ctx):
    dt = any_ctx.name
    x, r = rows_of(37, 1152, 1, dt), rows_of(37, 1152, 2, dt)
    g = store(np.ones(1152), dt)
    y, h = torch.empty_like(x), torch.empty_like(x)
    any_ctx.rmsnorm(x, g, y, residual=r, h=h, eps=EPS)
    for hx, yx in (("r", None), ("x", None), ("x", "r"), ("r", "x"), (None, "x"), (None, "r")):
        b = {"x": x.clone(), "r": r.clone()}
        out = b[yx] if yx else torch.empty_like(x)
        any_ctx.rmsnorm(b["x"], g, out, residual=b["r"], h=b[hx] if hx else None, eps=EPS)
        assert torch.equal(out, y) and (hx is None or torch.equal(b[hx], h)), (hx, yx)
    xx = x.clone()  # x added to itself
    any_ctx.rmsnorm(xx, g, y, residual=xx, h=xx, eps=EPS)
    assert torch.equal(xx, summed(x, x))


def test_rmsnorm_sum_of_any_bf16_values(ctx):
    """h is the fp32 sum rounded to bf16 for every kind of pair: equal and far
    exponents, subnormals, sums that overflow (random bit patterns, NaN left out)."""
    g = np.random.Generator(np.random.PCG64(11))
    bits = g.integers(0, 1 << 16, (2, 512, 4096)).astype(np.uint16)
    near = bits[0] ^ g.integers(0, 1 << 9, bits[0].shape).astype(np.uint16)  # close in size
    bits[1, :256] = near[:256] ^ (g.integers(0, 2, near[:256].shape).astype(np.uint16) << 15)
    x, r = (to_dev(b, "bf16") for b in bits)
    x[~torch.isfinite(x)], r[~torch.isfinite(r)] = 1.0, -2.0
    h, y = torch.empty_like(x), torch.empty_like(x)
    ctx.rmsnorm(x, torch.ones(4096, dtype=torch.bfloat16, device="cuda"), y, residual=r, h=h)
    assert torch.equal(h.view(torch.int16), summed(x, r).view(torch.int16))


def test_rmsnorm_rounds_correctly_next_to_borders(ctx):
    """Many outputs within fp32 rounding of a bf16 midpoint: of twenty gammas each
    column takes the one that brings the most of its rows there."""
    g = np.random.Generator(np.random.PCG64(12))
    rows, cols = 400, 1152
    a = bf16_of(g.standard_normal((rows, cols)))
    x = to_dev(synth.round_bf16_bits(a), "bf16")
    best = None
    for _ in range(20):
        gm = bf16_of(1 + g.standard_normal(cols) * 0.3)
        ref = NR.rmsnorm(a, gm, float(np.float32(EPS)))
        m, _ = np.frexp(ref)
        t = np.abs(np.abs(m) * 256 % 1 - 0.5)  # distance from a bf16 midpoint, in steps
        score = (t < 2.0 ** -12).sum(0)
        best = (score, gm) if best is None else (np.maximum(score, best[0]), np.where(score > best[0], gm, best[1]))
    assert best[0].sum() > 200
    gamma = to_dev(synth.round_bf16_bits(best[1]), "bf16")
    ref = bf16_of(NR.rmsnorm(a, best[1], float(np.float32(EPS))))
    for n in (3, rows):  # few rows and many rows take different thread layouts
        y = torch.empty_like(x[:n])
        ctx.rmsnorm(x[:n].contiguous(), gamma, y, eps=EPS)
        assert np.array_equal(from_dev(y), ref[:n])


def test_rmsnorm_values_at_the_ends(ctx):
    cols = 1152
    a = np.ones((6, cols))
    a[0] *= 3e38          # the squares leave fp32
    a[1] *= 2.0 ** -130   # subnormal
    a[2, 3] = np.inf
    a[3, 4] = np.nan
    a[4] = 0
    x = to_dev(synth.round_bf16_bits(a), "bf16")
    gamma = store(np.full(cols, 1.5), "bf16")
    y = torch.empty_like(x)
    for eps in (EPS, 0.0):
        ctx.rmsnorm(x, gamma, y, eps=eps)
        with np.errstate(all="ignore"):
            ref = bf16_of(NR.rmsnorm(from_dev(x), from_dev(gamma), float(np.float32(eps))))
        assert np.array_equal(from_dev(y), ref, equal_nan=True), eps


MX_SHAPES = [(3900, 1152), (5000, 72), (1000, 4608), (1, 8), (1, 1152), (130, 40), (257, 200), (300, 1152), (129, 1536), (20, 4608),
             (140, 5000), (3, 16384)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", MX_SHAPES)
def test_rmsnorm_mx8(ctx, rows, cols, residual):
    x, r = rows_of(rows, cols, rows + cols, "bf16"), rows_of(rows, cols, rows + cols + 1, "bf16")
    gamma = store(1 + 0.1 * np.random.Generator(np.random.PCG64(8)).standard_normal(cols), "bf16")
    res = r if residual else None
    h, codes = Band((rows, cols), torch.bfloat16), Band((rows, vit.mx8_row_bytes(cols)), torch.uint8)
    scales = Band((vit.mx8_scale_bytes(rows, cols),), torch.uint8)
    ctx.rmsnorm_mx8(x, gamma, codes.t, scales.t, residual=res, h=h.t, eps=EPS)
    codes.check("codes"), scales.check("scales"), h.check("h")
    y = torch.empty_like(x)
    ctx.rmsnorm(x, gamma, y, residual=res, eps=EPS)
    c2, s2 = torch.empty_like(codes.t), torch.empty_like(scales.t)
    ctx.mx8_quantize(y, c2, s2)
    assert torch.equal(codes.t[:, :cols], c2[:, :cols]) and torch.equal(scales.t, s2)
    assert torch.equal(h.t, summed(x, r) if residual else x)
    ref = NR.rmsnorm(from_dev(h.t), from_dev(gamma), float(np.float32(EPS)))
    q, s = MX.mx_quantize(bf16_of(ref))
    assert np.array_equal(codes.t.cpu().numpy()[:, :cols], q)
    assert np.array_equal(scales.t.cpu().numpy()[_scale_index(rows, cols)], s)
    assert ctx.device_status() == 0


def test_rmsnorm_large_offsets(ctx):
    # rows whose element offsets pass 2^31
    rows, cols = 140_000, 16384
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = rows_of(64, cols, 9, "bf16")
    x[-64:] = tail
    g = store(np.ones(cols), "bf16")
    y = torch.empty_like(tail)
    ctx.rmsnorm(tail, g, y, eps=EPS)
    ctx.rmsnorm(x, g, x, eps=EPS)
    assert torch.equal(x[-64:], y)
