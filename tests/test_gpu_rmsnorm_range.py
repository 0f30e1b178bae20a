"""RMSNorm where h * gamma leaves the fp32 range although the result does not,
and where the result lies exactly between two bf16 values.

bf16: y is the formula's value for the stored h rounded once to nearest, ties to
even.  The fp64 reference is within 2^-50 of the formula, and a random value is
closer than that to a bf16 midpoint with probability 2^-41, so y is compared bit
for bit; exact ties are computed by hand.  MXFP8 codes are those of that y.
fp32: three roundings from the formula, 2^-24 relative each, and one fp32
subnormal step for results below the normal range."""
import numpy as np
import pytest
import torch

import synth
from oracle import norm_rope_ref as NR
from tests.gpu_util import from_dev, to_dev

pytestmark = pytest.mark.gpu

vit = pytest.importorskip("vision_transformer_encoder_layernorm_b200")
MANY = 3000  # rows enough for several vectors a thread


@pytest.fixture(scope="module")
def ctx():
    c = vit.Context(1152, 16, 72, 4304, vit.BF16)
    yield c
    c.close()


def bf16(a):
    with np.errstate(all="ignore"):
        return to_dev(synth.round_bf16_bits(NR.to_bf16(a)), "bf16")


def check(ctx, h, gamma, eps, want=None):
    """y and the codes of y, for the rows alone and among many."""
    x, g = bf16(h), bf16(gamma)
    if want is None:
        with np.errstate(all="ignore"):
            want = NR.to_bf16(NR.rmsnorm(from_dev(x), from_dev(g), float(np.float32(eps))))
    rows, cols = x.shape
    times = -(-MANY // rows)
    for xs, w in ((x, want), (x.repeat(times, 1), np.tile(want, (times, 1)))):
        y = torch.empty_like(xs)
        ctx.rmsnorm(xs, g, y, eps=eps)
        got = from_dev(y)
        bad = ~((got == w) | (np.isnan(got) & np.isnan(w)))
        assert not bad.any(), (bad.mean(), np.argwhere(bad)[:4].tolist(), got[bad][:4], w[bad][:4])
        q = [(torch.empty((len(xs), vit.mx8_row_bytes(cols)), dtype=torch.uint8, device="cuda"),
              torch.empty(vit.mx8_scale_bytes(len(xs), cols), dtype=torch.uint8, device="cuda"))
             for _ in range(2)]
        ctx.rmsnorm_mx8(xs, g, *q[0], eps=eps)
        ctx.mx8_quantize(bf16(w), *q[1])
        assert torch.equal(q[0][0][:, :cols], q[1][0][:, :cols]) and torch.equal(q[0][1], q[1][1])
    assert ctx.device_status() == 0


def test_zeros_keep_their_sign(ctx):
    """Also in vectors of 8 columns that hold a value next to a bf16 border: among
    3000 rows some do, at about 1 vector in 2000."""
    g = np.random.Generator(np.random.PCG64(6))
    h = g.standard_normal((500, 1152))
    h[:, 1::2] = 0
    gamma = -(1 + 0.3 * g.random(1152))
    check(ctx, h, gamma, 1e-6)
    x, w = bf16(h).repeat(6, 1), bf16(gamma)
    y = torch.empty_like(x)
    ctx.rmsnorm(x, w, y, eps=1e-6)
    assert torch.all(torch.signbit(y[:, 1::2]))
    ctx.rmsnorm(-x, w, y, eps=1e-6)  # -0 times a negative gamma
    assert not torch.any(torch.signbit(y[:, 1::2]))


@pytest.mark.parametrize("cols", [64, 1152, 4616])
@pytest.mark.parametrize("row,gam,eps", [
    (80, 60, 1e-6),     # the product overflows, the result is 2^60
    (100, 27, 1e-6), (126, 100, 0.0),
    (-90, -70, 0.0),    # the product underflows, the result is 2^-70
    (-95, -48, 0.0),    # the product is subnormal and has lost bits
    (-60, -70, 0.0), (-99, 126, 0.0), (-130, 20, 0.0), (0, -126, 1e-6), (0, 120, 1e-6),
    (-20, -120, 0.0), (3, -130, 1e-6)])
def test_products_out_of_range(ctx, cols, row, gam, eps):
    g = np.random.Generator(np.random.PCG64(abs(row) + abs(gam)))
    h = g.standard_normal((9, cols)) * 2.0 ** row
    h[:, ::7] = 0
    gamma = (1 + 0.3 * g.standard_normal(cols)) * 2.0 ** gam
    check(ctx, np.clip(h, -3e38, 3e38), gamma, eps)
    gamma[::3] = 1 + 0.3 * g.standard_normal(len(gamma[::3]))  # neighbours of ordinary size
    check(ctx, np.clip(h, -3e38, 3e38), gamma, eps)


@pytest.mark.parametrize("cols", [256, 1160])
def test_values_of_every_size(ctx, cols):
    """Rows of any size, elements far below their row's, gammas of any size."""
    g = np.random.Generator(np.random.PCG64(cols))
    rows = 200
    h = g.standard_normal((rows, cols)) * np.exp2(g.integers(-126, 120, (rows, 1)) - g.integers(0, 60, (rows, cols)) * (g.random((rows, cols)) < 0.8))
    gamma = g.standard_normal(cols) * np.exp2(g.integers(-126, 126, cols).astype(float))
    check(ctx, h, gamma, 0.0)
    check(ctx, h, gamma, 1e-6)


def test_exact_ties_go_to_even(ctx):
    """One value a in 576 columns and no eps: y = 24 gamma sign(a) exactly, which for
    gamma = m / 64 (m odd, 87 .. 169) lies half-way between two bf16 values."""
    cols, m = 576, np.arange(87, 170, 2)
    g = np.random.Generator(np.random.PCG64(5))
    gamma = np.ones(cols)
    at = g.permutation(cols)[: len(m)]
    gamma[at] = m / 64
    a = NR.to_bf16((1 + g.random(len(m))) * np.exp2(g.integers(-30, 30, len(m)))) * np.where(g.random(len(m)) < 0.5, -1, 1)
    h, want = np.zeros((len(m), cols)), np.zeros((len(m), cols))
    h[np.arange(len(m)), at] = a
    # 3m/8 has 9 significant bits, the last one set: bf16 keeps 8
    want[np.arange(len(m)), at] = np.sign(a) * np.rint(3 * m / 2) / 4
    check(ctx, h, gamma, 0.0, want)


def test_exact_ties_out_of_range(ctx):
    """The same in rows whose size sends them through fp64 throughout."""
    cols, m = 576, np.arange(87, 170, 2)
    h, gamma, want = np.zeros((len(m), cols)), np.ones(cols), np.zeros((len(m), cols))
    gamma[: len(m)] = m / 64
    for r, e in enumerate(np.where(np.arange(len(m)) % 2, 126, -120)):
        h[r, r] = 1.5 * 2.0 ** e
        want[r, r] = np.rint(3 * m[r] / 2) / 4
    check(ctx, h, gamma, 0.0, want)


@pytest.mark.parametrize("rows", [5, 700])
def test_fp32_elements_far_below_their_row(rows):
    ctx = vit.Context(1152, 16, 72, 4304, vit.F32)
    g = np.random.Generator(np.random.PCG64(rows))
    cols = 512
    h = g.standard_normal((rows, cols))
    h[:, 1::2] *= np.exp2(-g.integers(60, 149, (rows, cols // 2)).astype(float))
    h = (h * np.exp2(g.integers(0, 20, (rows, 1)).astype(float))).astype(np.float32)
    gamma = (g.standard_normal(cols) * np.exp2(g.integers(-20, 100, cols).astype(float))).astype(np.float32)
    y = torch.empty(rows, cols, device="cuda")
    ctx.rmsnorm(to_dev(h, "f32"), to_dev(gamma, "f32"), y, eps=0.0)
    ref = NR.rmsnorm(h.astype(np.float64), gamma.astype(np.float64), 0.0)
    assert np.all(np.abs(from_dev(y) - ref) <= 3.01 * 2.0 ** -24 * np.abs(ref) + 2.0 ** -148)
    ctx.close()
