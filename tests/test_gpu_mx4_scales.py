"""vit_linear_mx4 on operands whose scales are far apart, against the fp64 oracle
from end to end: the oracle quantises the bf16 inputs and multiplies what its own
codes stand for.

Rows differ by up to 2^60 and groups of a row by up to 2^40, some groups are zero
(scale byte 0), some hold bf16 subnormals, and one pair of operands has scale
bytes near both ends.  The error is bounded as for ordinary operands: 2^-22 of S =
sum |a w| + |b| + |residual| per K = 64 step of the tensor core and 4 more, and one
rounding to bf16, 2^-8 relative; S bounds the terms of every step, however far
apart they are."""
import numpy as np
import pytest
import torch

import synth
from oracle import mxfp4_ref as M4
from tests.gpu_util import from_dev, to_dev
from tests.test_gpu_mx8 import _scale_index

pytestmark = pytest.mark.gpu

vit = pytest.importorskip("vision_transformer_encoder_layernorm_b200")


@pytest.fixture(scope="module")
def ctx():
    c = vit.Context(1152, 16, 72, 4304, vit.BF16)
    yield c
    c.close()


def bf16(a):
    bits = synth.round_bf16_bits(a)
    return to_dev(bits, "bf16"), synth.bf16_bits_to_f64(bits)


def spread(g, rows, K, row_exp, group_exp):
    """Normal values times a power of two for the row and one for the group; a tenth
    of the groups zero."""
    e = np.repeat(g.integers(-group_exp, group_exp + 1, (rows, -(-K // 32))), 32, 1)[:, :K]
    z = np.repeat(g.random((rows, -(-K // 32))) < 0.1, 32, 1)[:, :K]
    a = g.standard_normal((rows, K)) * np.exp2(e + g.integers(-row_exp, row_exp + 1, (rows, 1)))
    a[z] = 0
    if rows > 1:
        a[rows // 2] = 0
    return a


def quantize(ctx, x, xr):
    """The library's codes and scales, and the oracle's; they have to agree."""
    rows, K = x.shape
    codes = torch.empty((rows, vit.mx4_row_bytes(K)), dtype=torch.uint8, device="cuda")
    scales = torch.empty(vit.mx4_scale_bytes(rows, K), dtype=torch.uint8, device="cuda")
    ctx.mx4_quantize(x, codes, scales)
    q, s = M4.mx4_quantize(xr)
    assert np.array_equal(codes.cpu().numpy(), M4.pack(q))
    assert np.array_equal(scales.cpu().numpy()[_scale_index(rows, K)], s)
    return (codes, scales), (q, s)


def check(ctx, xr, wr, epi, seed, size=1.0):
    (x, xr), (w, wr) = bf16(xr), bf16(wr)
    (M, K), N = x.shape, w.shape[0]
    g = np.random.Generator(np.random.PCG64(seed))
    b, br = bf16(size * g.standard_normal(N))
    r, rr = bf16(size * g.standard_normal((M, N)))
    (a, ar), (wq, wqr) = quantize(ctx, x, xr), quantize(ctx, w, wr)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    ctx.linear_mx4(a, wq, b, y, K, epi=epi, residual=r if epi == 2 else None)
    assert ctx.device_status() == 0
    ref = M4.mx4_linear(ar, wqr, br, "residual" if epi == 2 else "none", rr)
    S = np.abs(M4.mx4_dequantize(*ar)) @ np.abs(M4.mx4_dequantize(*wqr)).T + np.abs(br)
    tol = (-(-K // 64) + 4) * 2.0 ** -22 * (S + (np.abs(rr) if epi == 2 else 0))
    got = from_dev(y)
    bad = ~(np.abs(got - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol))
    assert not bad.any(), (bad.mean(), np.argwhere(bad)[:5].tolist(), got[bad][:5], ref[bad][:5])


TILES = ["1x128", "2x128", "2x192", "2x256", "1x128x2", "1x128x4", "1x128x8"]


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("M,N,K,epi", [(130, 392, 2100, 0), (257, 520, 2081, 2), (1, 200, 2305, 2)])
def test_scales_far_apart(ctx, monkeypatch, tile, M, N, K, epi):
    """Tiles of 192 columns start inside a block of 128 scale rows."""
    monkeypatch.setenv("VIT_MX4_TILE", tile)
    g = np.random.Generator(np.random.PCG64(M + N + K))
    check(ctx, spread(g, M, K, 15, 20), spread(g, N, K, 15, 20), epi, M + K)


@pytest.mark.parametrize("tile", TILES)
def test_every_row_keeps_its_own_scale(ctx, monkeypatch, tile):
    """Rows of A and W that differ by powers of two alone: results do too, exactly."""
    monkeypatch.setenv("VIT_MX4_TILE", tile)
    M, N, K = 260, 584, 2177
    g = np.random.Generator(np.random.PCG64(3))
    ea, ew = g.integers(-30, 31, M), g.integers(-30, 31, N)
    x, _ = bf16(np.tile(g.standard_normal((1, K)), (M, 1)) * np.exp2(ea)[:, None].astype(float))
    w, _ = bf16(np.tile(g.standard_normal((1, K)), (N, 1)) * np.exp2(ew)[:, None].astype(float))
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")

    def q(t):
        codes = torch.empty((t.shape[0], vit.mx4_row_bytes(K)), dtype=torch.uint8, device="cuda")
        scales = torch.empty(vit.mx4_scale_bytes(t.shape[0], K), dtype=torch.uint8, device="cuda")
        ctx.mx4_quantize(t, codes, scales)
        return codes, scales
    ctx.linear_mx4(q(x), q(w), None, y, K)
    got = from_dev(y) * np.exp2(-(ea[:, None] + ew[None, :]).astype(float))
    assert got[0, 0] != 0 and np.all(got == got[0, 0])


@pytest.mark.parametrize("ax,aw", [(100, -100), (-100, 100), (120, -110), (-130, 118)])
def test_scale_bytes_near_the_ends(ctx, ax, aw):
    g = np.random.Generator(np.random.PCG64(abs(ax)))
    M, N, K = 70, 136, 333
    x = g.standard_normal((M, K)) * 2.0 ** ax
    w = g.standard_normal((N, K)) * 2.0 ** aw
    check(ctx, x, w, 0, 9, size=2.0 ** (ax + aw))
