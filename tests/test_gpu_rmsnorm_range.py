"""RMSNorm at the edges of its arithmetic.

bf16: y is the formula's value for the stored h rounded once to nearest.  The fp64
reference is within 2^-50 of the formula, and a random value is closer than that to
a bf16 midpoint with probability 2^-41, so y is compared bit for bit.  MXFP8 codes
are those of that y."""
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
