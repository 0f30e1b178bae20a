"""vit_rope3d against the fp64 oracle.  A pair's results are fp32 sums of two
products with fp32 cos and sin: within (|a| + |b|) 2^-21 of the formula (three
roundings of 2^-24, the sine's own error and the angle's 1e-7), 1e-6 more where
positions are far (the frequency is an fp64 value), then one rounding to the
type."""
import numpy as np
import pytest
import torch

import synth
from oracle import norm_rope_ref as NR
from tests.gpu_util import from_dev, to_dev
from tests.test_zzz_guard_bands import Band

pytestmark = pytest.mark.gpu

vit = pytest.importorskip("vision_transformer_encoder_layernorm_b200")
LAYOUT = {"blocks": vit.ROPE_BLOCKS, "sections": vit.ROPE_SECTIONS, "turns": vit.ROPE_TURNS}
CTX = {}


def context(d, dt):
    if (d, dt) not in CTX:
        CTX[d, dt] = vit.Context(4 * d, 4, d, 64, vit.BF16 if dt == "bf16" else vit.F32)
    return CTX[d, dt]


def data(shape, seed, dt):
    return to_dev(synth.random_tensor(shape, seed, dt), dt)


def positions(T, seed, far=False):
    g = np.random.Generator(np.random.PCG64(seed))
    p = g.integers(-2 ** 31, 2 ** 31, (T, 3)) if far else g.integers(0, 5000, (T, 3))
    if far and T > 1:
        p[0], p[1] = -2 ** 31, 2 ** 31 - 1
    return torch.from_numpy(p.astype(np.int32)).cuda()


def check(got, x, pos, sec, layout, dt, far=False):
    xr, p = from_dev(x), pos.cpu().numpy()
    ref = NR.rope3d(xr, p, sec, layout)
    size = np.empty_like(xr)
    for lo, hi, _, _ in NR.rope3d_pairs(xr.shape[2], sec, layout):
        size[..., lo] = size[..., hi] = np.abs(xr[..., lo]) + np.abs(xr[..., hi])
    tol = size * (2.0 ** -21 + (1e-6 if far else 0))
    step = 2.0 ** -8 if dt == "bf16" else 2.0 ** -24
    assert np.all(np.abs(from_dev(got) - ref) <= tol + step * (np.abs(ref) + tol))


CASES = [(64, "f32", (8, 12, 12)), (64, "f32", (10, 11, 11)), (72, "bf16", (12, 12, 12)),
         (72, "bf16", (10, 13, 13)), (72, "f32", (0, 18, 18)), (128, "bf16", (16, 24, 24)),
         (128, "bf16", (64, 0, 0)), (128, "bf16", (1, 31, 32)), (128, "f32", (24, 20, 20))]


@pytest.mark.parametrize("layout", list(LAYOUT))
@pytest.mark.parametrize("d,dt,sec", CASES)
def test_rope3d(d, dt, sec, layout):
    c = context(d, dt)
    for T, H in ((1, 1), (7, 3), (130, 32), (33, 5), (3, 70)):
        x, pos = data((T, H, d), T + H, dt), positions(T, T)
        y = Band((T, H, d), x.dtype)
        c.rope3d(x, pos, sec, LAYOUT[layout], out=y.t)
        y.check(f"rope3d {T} {H}")
        check(y.t, x, pos, sec, layout, dt)
        z = x.clone()
        c.rope3d(z, pos, sec, LAYOUT[layout])  # in place
        assert torch.equal(z, y.t)
    assert c.device_status() == 0


@pytest.mark.parametrize("layout", list(LAYOUT))
def test_far_positions(layout):
    c = context(128, "f32")
    x, pos = data((64, 2, 128), 5, "f32"), positions(64, 6, far=True)
    y = torch.empty_like(x)
    c.rope3d(x, pos, (16, 24, 24), LAYOUT[layout], out=y)
    check(y, x, pos, (16, 24, 24), layout, "f32", far=True)


@pytest.mark.parametrize("off", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("d,dt", [(72, "bf16"), (128, "bf16"), (128, "f32")])
def test_rows_of_a_wider_tensor(d, dt, off):
    """Queries and keys in place in front of the values, at any alignment; what
    lies between the rows, and rows behind the last token, stay as they were."""
    c, T, H = context(d, dt), 50, 6
    sec = (12, 12, 12) if d == 72 else (16, 24, 24)
    width = 9 * d + off
    flat = data(((T + 2) * width + off,), 3, dt)
    wide = flat[off:off + (T + 2) * width].view(T + 2, width)
    before, pos = wide.clone(), positions(T, 9)
    x = wide[:T, :H * d].unflatten(1, (H, d))
    c.rope3d(x, pos, sec, vit.ROPE_TURNS)
    check(x, before[:T, :H * d].unflatten(1, (H, d)), pos, sec, "turns", dt)
    assert torch.equal(wide[:T, H * d:], before[:T, H * d:]) and torch.equal(wide[T:], before[T:])
    # from one part of the row to another: only the three heads there change
    now = wide.clone()
    dst = wide[:T, H * d:9 * d].unflatten(1, (3, d))
    c.rope3d(x[:, :3], pos, sec, vit.ROPE_SECTIONS, out=dst)
    check(dst, now[:T, :3 * d].unflatten(1, (3, d)), pos, sec, "sections", dt)
    assert torch.equal(wide[:T, :H * d], now[:T, :H * d]) and torch.equal(wide[T:], now[T:])
    assert torch.equal(wide[:T, 9 * d:], now[:T, 9 * d:])


def test_equals_rope2d_without_time():
    """(0, d/4, d/4) in blocks is vit_rope2d's convention.  Its fp32 angles (at
    most 80 radians) are off by up to 80 * 2^-23, which moves a result by that
    times |a| + |b| at most; bf16 results round on top, by half a step each."""
    for d, dt in ((72, "bf16"), (128, "bf16"), (64, "f32")):
        c, T = context(d, dt), 96
        qkv, pos = data((T, 12, d), 4, dt), positions(T, 5) % 80
        want = qkv.clone()
        c.rope2d(want.view(T, -1), pos[:, 1:].contiguous())
        c.rope3d(qkv[:, :8], pos, (0, d // 4, d // 4))
        step = 2.0 ** -7 if dt == "bf16" else 2.0 ** -23
        tol = 80 * 2.0 ** -23 * 2 * np.abs(from_dev(want)).max() * 1.5
        assert np.all(np.abs(from_dev(qkv) - from_dev(want)) <= step * np.abs(from_dev(want)) + tol)
        assert torch.equal(qkv[:, 8:], want[:, 8:])


def test_offsets_past_32_bits():
    c, d, H = context(128, "bf16"), 128, 1
    T, stride = 70_000, 1 << 15  # the last rows start past 2^31 elements
    wide = torch.zeros(T, stride, dtype=torch.bfloat16, device="cuda")
    x = data((64, H, d), 8, "bf16")
    wide[-64:, :d] = x[:, 0]
    pos = positions(T, 8)
    y = torch.empty_like(x)
    c.rope3d(x, pos[-64:].contiguous(), (16, 24, 24), out=y)
    c.rope3d(wide[:, :d].unflatten(1, (H, d)), pos, (16, 24, 24))
    assert torch.equal(wide[-64:, :d], y[:, 0])
