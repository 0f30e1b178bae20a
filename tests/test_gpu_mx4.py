"""MXFP4 quantiser, dequantiser and linear layer against the fp64 oracle.

The quantiser decides from exact arithmetic and the dequantiser is exact: bit
for bit.  The linear layer works on the same codes as the oracle; products of
E2M1 values and power-of-two scales are exact, so its error is
  - fp32 accumulation: at most 2^-22 of S = sum |a w| (+ |b| + |residual|) per
    K = 64 step of the tensor core (an addition that may truncate, 2^-23, and
    the alignment of its terms), and 4 more for the epilogue;
  - GELU: its slope is at most 1.13 on that error, and the hardware tanh is
    within 2^-10.9 relative, half of u times that;
  - one rounding to bf16, 2^-8 relative."""
import numpy as np
import pytest
import torch

import synth
from oracle import mxfp4_ref as M4
from tests.gpu_util import from_dev, to_dev
from tests.test_gpu_mx8 import _scale_index
from tests.test_zzz_guard_bands import Band

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


def normal(shape, seed, scale=1.0):
    return bf16(scale * np.random.Generator(np.random.PCG64(seed)).standard_normal(shape))


def quantize(ctx, x):
    rows, K = x.shape
    codes = torch.empty((rows, vit.mx4_row_bytes(K)), dtype=torch.uint8, device="cuda")
    scales = torch.empty(vit.mx4_scale_bytes(rows, K), dtype=torch.uint8, device="cuda")
    ctx.mx4_quantize(x, codes, scales)
    return codes, scales


@pytest.mark.parametrize("rows,K", [(1, 1), (1, 31), (3, 33), (5, 48), (130, 130), (257, 200),
                                    (300, 1152), (129, 1151), (66, 4304), (7, 1025), (2, 9000),
                                    (17, 1154), (40, 1026), (9, 4301), (300, 35), (50, 4303)])
def test_quantize_and_dequantize(ctx, rows, K):
    g = np.random.Generator(np.random.PCG64(rows + K))
    a = g.standard_normal((rows, K)) * np.exp2(g.integers(-30, 30, (rows, 1)))
    a[rows // 2] = 0
    if rows > 2:
        a[0] = g.choice([0.25, 0.75, 2.5, 3.5, 5.0, 5.03125, 7.0, 7.9375, -5.0], K)  # ties and tops
        a[1] *= 2.0 ** -100
        a[2] = g.choice([2.0 ** -133, 2.0 ** -126, 3 * 2.0 ** -128, 0], K)  # subnormals
    x, xr = bf16(a)
    codes, scales = Band((rows, vit.mx4_row_bytes(K)), torch.uint8), Band((vit.mx4_scale_bytes(rows, K),), torch.uint8)
    ctx.mx4_quantize(x, codes.t, scales.t)
    codes.check("codes"), scales.check("scales")
    q, s = M4.mx4_quantize(xr)
    assert np.array_equal(codes.t.cpu().numpy(), M4.pack(q))  # zeros past K
    sc, idx = scales.t.cpu().numpy(), _scale_index(rows, K)
    assert np.array_equal(sc[idx], s)
    pad = np.ones(sc.size, bool)
    pad[idx.ravel()] = False
    assert np.all(sc[pad] == 127)
    y = Band((rows, K), torch.bfloat16)
    ctx.mx4_dequantize(codes.t, scales.t, y.t)
    y.check("values")
    assert np.array_equal(from_dev(y.t), M4.mx4_dequantize(q, s))
    assert ctx.device_status() == 0


def test_quantize_infinity_and_nan(ctx):
    a = np.random.Generator(np.random.PCG64(1)).standard_normal((4, 96))
    a[0, 5], a[1, 40], a[2, 70], a[2, 71] = np.inf, np.nan, np.nan, -np.inf
    a[3, :32] = 3.38e38
    x, _ = bf16(np.nan_to_num(a, nan=0.0, posinf=0.0, neginf=0.0))
    x[0, 5], x[1, 40], x[2, 70], x[2, 71] = float("inf"), float("nan"), float("nan"), float("-inf")
    codes, scales = quantize(ctx, x)
    with np.errstate(all="ignore"):
        q, s = M4.mx4_quantize(from_dev(x))
    assert np.array_equal(codes.cpu().numpy(), M4.pack(q))
    assert np.array_equal(scales.cpu().numpy()[_scale_index(4, 96)], s)
    y = torch.empty_like(x)
    ctx.mx4_dequantize(codes, scales, y)
    v = from_dev(y)
    assert np.isnan(v[1, 32:64]).all() and np.isfinite(v[1, :32]).all() and np.isposinf(v[0, 5])
    # a NaN in a row of A reaches that row of the product and no other
    out = torch.empty(4, 8, dtype=torch.bfloat16, device="cuda")
    w, _ = normal((8, 96), 3)
    ctx.linear_mx4((codes, scales), quantize(ctx, w), None, out, 96)
    assert torch.isnan(out[1]).all() and torch.isnan(out[2]).all() and not torch.isnan(out[3]).any()


def check_linear(ctx, M, N, K, epi, seed, bias=True, rows=None):
    x, _ = normal((M, K), seed)
    w, _ = normal((N, K), seed + 1, 0.05)
    b, br = normal((N,), seed + 2)
    r, rr = normal((M, N), seed + 3)
    a, wq = quantize(ctx, x), quantize(ctx, w)
    y = Band((M, N), torch.bfloat16)
    ctx.linear_mx4(a, wq, b if bias else None, y.t, K, epi=epi, residual=r if epi == 2 else None)
    y.check(f"linear {M}x{N}x{K} epi {epi}")
    assert ctx.device_status() == 0
    rows = np.arange(M) if rows is None else rows

    def value(pair, n):
        va = torch.empty(n, K, dtype=torch.bfloat16, device="cuda")
        ctx.mx4_dequantize(*pair, va)
        return va.double()
    va, vw = value(a, M)[torch.from_numpy(rows).cuda()], value(wq, N)
    u = (va @ vw.T).cpu().numpy() + (br if bias else 0)
    S = (va.abs() @ vw.abs().T).cpu().numpy() + np.abs(br)
    tol = (-(-K // 64) + 4) * 2.0 ** -22 * (S + (np.abs(rr[rows]) if epi == 2 else 0))
    ref = u
    if epi == 1:
        ref = 0.5 * u * (1 + np.tanh(np.sqrt(2 / np.pi) * (u + 0.044715 * u ** 3)))
        tol = 1.13 * tol + 0.5 * np.abs(u) * 2.0 ** -10.9
    elif epi == 2:
        ref = u + rr[rows]
    got = from_dev(y.t)[rows]
    bad = np.abs(got - ref) > tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert not bad.any(), (np.argwhere(bad)[:5].tolist(), got[bad][:5], ref[bad][:5], bad.mean())
    return a, wq, b, r, y.t


@pytest.mark.parametrize("M,N,K,epi", [
    (1, 8, 1, 0), (1, 8, 64, 1), (1, 136, 65, 2), (2, 128, 128, 0), (127, 256, 129, 0),
    (128, 264, 255, 1), (129, 128, 256, 2), (130, 1152, 257, 0), (255, 384, 320, 2),
    (256, 256, 385, 0), (257, 392, 1151, 1), (300, 520, 1152, 2), (513, 1152, 4304, 0),
    (1, 3456, 1152, 0), (7, 1152, 4304, 2), (33, 4304, 1152, 1), (64, 1152, 9001, 0)])
def test_linear(ctx, M, N, K, epi):
    check_linear(ctx, M, N, K, epi, M + N + K, bias=(M + K) % 3 != 0)


@pytest.mark.parametrize("tile", ["1x128", "2x128", "2x192", "2x256"])
@pytest.mark.parametrize("M,N,K,epi", [
    (1, 8, 65, 2), (129, 392, 130, 1), (255, 200, 640, 2), (300, 1152, 1100, 0), (700, 1160, 2049, 2),
    (1300, 4304, 300, 1), (5000, 2056, 257, 2)])
def test_linear_every_tile(ctx, monkeypatch, tile, M, N, K, epi):
    """Every tile shape on sizes that the choice by size gives to another: odd
    rows and columns, one to several tiles a worker."""
    monkeypatch.setenv("VIT_MX4_TILE", tile)
    check_linear(ctx, M, N, K, epi, M + N + K)


@pytest.mark.parametrize("tile", ["1x128x2", "1x128x4", "1x128x8"])
@pytest.mark.parametrize("M,N,K,epi", [(1, 1152, 4304, 0), (1, 8, 2100, 1), (33, 136, 2049, 2),
                                       (128, 1152, 4400, 1), (260, 264, 2305, 2)])
def test_linear_split_tiles(ctx, monkeypatch, tile, M, N, K, epi):
    """A tile's k-blocks over 2, 4 or 8 CTAs, in runs of unequal length."""
    monkeypatch.setenv("VIT_MX4_TILE", tile)
    y = check_linear(ctx, M, N, K, epi, M + N + K)[4].clone()
    for _ in range(3):  # the sums' order does not depend on which CTA is done first
        assert torch.equal(check_linear(ctx, M, N, K, epi, M + N + K)[4], y)


@pytest.mark.parametrize("M,N,K,epi", [(3900, 4304, 1152, 1), (3900, 3456, 1152, 0),
                                       (10936, 1152, 4304, 2), (960, 1152, 1152, 2)])
def test_linear_layer_sizes(ctx, M, N, K, epi):
    g = np.random.Generator(np.random.PCG64(M))
    rows = np.unique(np.concatenate([g.choice(M, 300, replace=False), [0, 127, 128, 255, 256, M - 129, M - 1]]))
    check_linear(ctx, M, N, K, epi, 5, rows=rows)


def test_linear_residual_in_place_and_repeatable(ctx):
    for M, N, K in ((300, 392, 1152), (5, 1152, 4304)):
        a, w, b, r, y = check_linear(ctx, M, N, K, 2, 11)
        for _ in range(3):
            out = r.clone()
            ctx.linear_mx4(a, w, b, out, K, epi=2, residual=out)
            assert torch.equal(out, y)


def test_linear_ignores_what_lies_past_k(ctx):
    # code bytes past K's, and the scales of groups past K, are not the caller's to set
    M, N, K = 130, 136, 70
    x, _ = normal((M, K), 21)
    w, _ = normal((N, K), 22)
    a, wq = quantize(ctx, x), quantize(ctx, w)
    y, y2 = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ctx.linear_mx4(a, wq, None, y, K)
    for codes, _ in (a, wq):
        codes[:, 35:] = 0xFF
    ctx.linear_mx4(a, wq, None, y2, K)
    assert torch.equal(y, y2)


def test_linear_two_streams_and_two_graphs(ctx):
    """Calls in flight together (eager on two streams, two captured graphs) share
    nothing."""
    jobs = []
    for i, (M, N, K, epi) in enumerate([(700, 1152, 1152, 2), (9, 1152, 4304, 0)]):
        a, w, b, r, y = check_linear(ctx, M, N, K, epi, 31 + i)
        jobs.append((a, w, b, r if epi == 2 else None, y.clone(), torch.empty_like(y), K, epi))
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (a, w, b, r, _, out, K, epi) in zip(streams, jobs):
            ctx.linear_mx4(a, w, b, out, K, epi=epi, residual=r, stream=s)
    torch.cuda.synchronize()
    for j in jobs:
        assert torch.equal(j[5], j[4])
    graphs = []
    for a, w, b, r, _, out, K, epi in jobs:
        out.zero_()
        st = ctx.graph_begin()
        for _ in range(10):
            ctx.linear_mx4(a, w, b, out, K, epi=epi, residual=r, stream=st)
        graphs.append(ctx.graph_end())
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            g.launch(s)
    torch.cuda.synchronize()
    for j in jobs:
        assert torch.equal(j[5], j[4])
    for g in graphs:
        g.close()
    assert ctx.device_status() == 0
