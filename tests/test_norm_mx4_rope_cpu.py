"""Host-only checks of RMSNorm, MXFP4 and three-axis RoPE: pins of their
oracles, and the refusals of the C entry points and of the binding.  A refusal
reads nothing of a context but its configuration, so a zeroed block that starts
with one stands in for a context here; no call below gets past the checks."""
import ctypes

import numpy as np
import pytest
import torch

import vision_transformer_encoder_layernorm_b200 as vit
from oracle import mxfp4_ref as M4
from oracle import norm_rope_ref as NR
from oracle import vit_ref as R

BAD, SHAPE, UNSUP = 1, 2, 3


# ---------------------------------------------------------------- oracles
def test_e2m1_table_and_rounding():
    assert M4.e2m1_decode(np.arange(8)).tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert np.array_equal(M4.e2m1_encode(M4.e2m1_decode(np.arange(16))), np.arange(16))
    # ties go to the even code, everything above 6 to 6
    x = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 7.9, -0.25, -5.0]
    assert M4.e2m1_decode(M4.e2m1_encode(x)).tolist() == [0, 1, 1, 2, 2, 4, 4, 6, 6, 0, -4]


def test_mx4_quantize_blocks():
    x = np.zeros((1, 70))
    x[0, :4] = [6.0, -3.0, 0.5, 7.5]     # amax 7.5: X = 0, 7.5 clamps to 6
    x[0, 32:34] = [2.0 ** -130, 2.0 ** -133]  # X = -132 clamps to -127
    x[0, 66] = np.nan
    c, s = M4.mx4_quantize(x)
    assert s.tolist() == [[127, 0, 255]]
    assert M4.mx4_dequantize(c, s)[0, :4].tolist() == [6.0, -3.0, 0.5, 6.0]
    assert np.isnan(M4.mx4_dequantize(c, s)[0, 64:]).all() and not c[0, 64:].any()
    g = np.random.Generator(np.random.PCG64(1)).standard_normal((5, 77))
    c, s = M4.mx4_quantize(g)
    # a step of E2M1 is at most half the block's power of two times 4; half of it is the error
    lim = np.repeat(np.exp2(s - 127.0), 32, 1)[:, :77] * np.where(np.abs(g) >= 0, 1.0, 0)
    assert np.all(np.abs(M4.mx4_dequantize(c, s) - g) <= 2 * lim)  # 8 -> 6 at the very top
    assert np.array_equal(M4.unpack(M4.pack(c), 77), c)


def test_rope3d_blocks_without_time_is_rope2d():
    g = np.random.Generator(np.random.PCG64(2))
    x = g.standard_normal((6, 2, 72))
    pos = g.integers(0, 60, (6, 3))
    a = NR.rope3d(x, pos, (0, 18, 18), "blocks")
    b = R.rope2d(x, pos[:, 1:], 10000.0)
    np.testing.assert_allclose(a, b, atol=1e-12)


@pytest.mark.parametrize("layout,sec", [("blocks", (10, 13, 13)), ("sections", (12, 12, 12)),
                                        ("turns", (4, 16, 16)), ("turns", (36, 0, 0))])
def test_rope3d_pairs_cover_the_head(layout, sec):
    p = NR.rope3d_pairs(72, sec, layout)
    assert sorted([q[0] for q in p] + [q[1] for q in p]) == list(range(72))
    assert [sum(q[2] == a for q in p) for a in range(3)] == list(sec)
    # a rotation keeps every pair's length, and position 0 changes nothing
    x = np.random.Generator(np.random.PCG64(3)).standard_normal((3, 1, 72))
    y = NR.rope3d(x, np.array([[0, 0, 0], [5, 900, 7], [-3, 1, 2 ** 31 - 1]]), sec, layout)
    assert np.array_equal(y[0], x[0])
    for lo, hi, _, _ in p:
        np.testing.assert_allclose(np.hypot(y[..., lo], y[..., hi]), np.hypot(x[..., lo], x[..., hi]))


def test_to_bf16_rounds_once():
    # a value just above a midpoint that fp32 would first round to the midpoint
    v = 1 + 2.0 ** -8 + 2.0 ** -40
    assert NR.to_bf16([v, -v, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8]).tolist() == \
        [1 + 2.0 ** -7, -1 - 2.0 ** -7, 1, 1 + 2.0 ** -6]
    x = np.random.Generator(np.random.PCG64(5)).standard_normal(1000) * np.exp2(np.arange(1000) % 250 - 126.0)
    assert np.array_equal(NR.to_bf16(x), torch.from_numpy(x).bfloat16().double().numpy())
    assert NR.to_bf16([3.4e38, 1e300])[1] == np.inf


def test_rmsnorm_scale_invariance():
    g = np.random.Generator(np.random.PCG64(4))
    h, w = g.standard_normal((4, 40)), g.standard_normal(40)
    np.testing.assert_allclose(NR.rmsnorm(h * 8, w, 0), NR.rmsnorm(h, w, 0))
    np.testing.assert_allclose(np.mean(NR.rmsnorm(h, np.ones(40), 0) ** 2, 1), 1)


# ---------------------------------------------------------------- refusals of the C entry points
def fake(dtype=None, head_dim=72):
    buf = ctypes.create_string_buffer(1 << 16)
    cfg = vit.VitConfig(16 * head_dim, 16, head_dim, 64, 1e-6, 1e4,
                        vit.BF16 if dtype is None else dtype, 0)
    ctypes.memmove(buf, ctypes.byref(cfg), ctypes.sizeof(cfg))
    return buf


P = [(i + 1) << 32 for i in range(8)]  # addresses far apart, 16-byte aligned, never read
L = vit.lib


def test_sizes():
    for K, rb in [(0, 0), (1, 16), (32, 16), (33, 32), (1152, 576), (4304, 2160)]:
        assert vit.mx4_row_bytes(K) == rb
    for rows, K in [(1, 1), (129, 128), (3900, 4304), (0, 64)]:
        assert vit.mx4_scale_bytes(rows, K) == vit.mx8_scale_bytes(rows, K)
    assert L.vit_mx4_row_bytes(-1) == 0 and L.vit_mx4_scale_bytes(-1, 1) == 0
    assert L.vit_mx4_scale_bytes(1, -1) == 0


def test_rmsnorm_refusals():
    c, f = fake(), fake(vit.F32)
    nan = float("nan")

    def call(ctx=c, x=P[0], res=P[1], g=P[2], h=P[3], y=P[4], rows=4, cols=64, eps=1e-6):
        return L.vit_rmsnorm(ctx, x, res, g, h, y, rows, cols, eps, None)

    def mx8(ctx=c, x=P[0], res=P[1], g=P[2], h=P[3], rows=4, cols=64, eps=1e-6, q=P[5], s=P[6]):
        return L.vit_rmsnorm_mx8(ctx, x, res, g, h, rows, cols, eps, q, s, None)

    for kw in ({"ctx": None}, {"x": None}, {"g": None}, {"y": None}, {"rows": -1}, {"cols": -8},
               {"eps": -1e-6}, {"eps": nan}, {"x": P[0] + 8}, {"res": P[1] + 2}, {"h": P[3] + 4},
               {"h": P[4]}, {"y": P[4] + 8}, {"y": P[0] + 16}, {"h": P[1] + 128}, {"h": P[2]},
               {"y": P[2] - 16}):
        assert call(**kw) == BAD, kw
    for kw in ({"cols": 60}, {"cols": 16392}):
        assert call(**kw) == UNSUP, kw
    assert call(f, cols=62) == UNSUP
    for kw in ({"rows": 0}, {"cols": 0}):
        assert call(**kw) == 0 and mx8(**kw) == 0
    for kw in ({"ctx": None}, {"q": None}, {"s": None}, {"q": P[5] + 4}, {"q": P[0]}, {"s": P[3]},
               {"s": P[5] + 16}, {"q": P[2]}, {"h": P[0] + 64}, {"eps": nan}):
        assert mx8(**kw) == BAD, kw
    assert mx8(f) == UNSUP and mx8(cols=36) == UNSUP


def test_mx4_refusals():
    c, f = fake(), fake(vit.F32)
    for fn, order in ((L.vit_mx4_quantize, "x r k c s"), (L.vit_mx4_dequantize, "c s r k x")):
        def call(ctx=c, **kw):
            v = {"x": P[0], "r": 4, "k": 70, "c": P[1], "s": P[2], **kw}
            return fn(ctx, *[v[n] for n in order.split()], None)
        for kw in ({"x": None}, {"c": None}, {"s": None}, {"r": -1}, {"k": -1}, {"x": P[0] + 2},
                   {"c": P[1] + 8}, {"s": P[2] + 1}, {"c": P[0] + 16}, {"s": P[1] + 32}, {"s": P[0]}):
            assert call(**kw) == BAD, kw
        assert call(None) == BAD and call(f) == UNSUP and call(k=(1 << 30) + 1) == UNSUP
        assert call(r=0) == 0 and call(k=0) == 0

    def lin(ctx=c, a=P[0], sa=P[1], w=P[2], sw=P[3], b=P[4], res=None, y=P[5], M=4, N=16, K=70,
            epi=0):
        return L.vit_linear_mx4(ctx, a, sa, w, sw, b, res, y, M, N, K, epi, None)
    for kw in ({"ctx": None}, {"a": None}, {"sa": None}, {"w": None}, {"sw": None}, {"y": None},
               {"M": -1}, {"N": 0}, {"K": 0}, {"epi": 3}, {"epi": 2}, {"y": P[5] + 2},
               {"b": P[4] + 8}, {"y": P[0]}, {"y": P[3] + 16}, {"y": P[4]},
               {"epi": 2, "res": P[5] + 16}):
        assert lin(**kw) == BAD, kw
    big = (1 << 30) + 8
    assert lin(f) == UNSUP and lin(N=12) == UNSUP and lin(M=0) == 0
    assert lin(M=big) == UNSUP and lin(N=big) == UNSUP and lin(K=big) == UNSUP


def test_rope3d_refusals():
    c = fake()
    sec = (ctypes.c_int32 * 3)(12, 12, 12)

    def call(ctx=c, x=P[0], xs=2304, y=P[1], ys=2304, pos=P[2], T=5, H=32, s=sec, layout=0):
        return L.vit_rope3d(ctx, x, xs, y, ys, pos, T, H, s, layout, None)
    for kw in ({"ctx": None}, {"x": None}, {"y": None}, {"pos": None}, {"s": None}, {"T": -1},
               {"H": 0}, {"layout": 3}, {"layout": -1}, {"x": P[0] + 1}, {"pos": P[2] + 2},
               {"s": (ctypes.c_int32 * 3)(-1, 18, 19)},
               {"y": P[0] + 2}, {"y": P[0], "ys": 2305},        # meets x
               {"y": P[0] + 2304, "xs": 4000, "ys": 4000},      # half a row behind x
               {"pos": P[1] + 64}):
        assert call(**kw) == BAD, kw
    for kw in ({"s": (ctypes.c_int32 * 3)(12, 12, 11)}, {"xs": 2303}, {"ys": 2300}):
        assert call(**kw) == SHAPE, kw
    assert call(xs=(1 << 30) + 1) == UNSUP
    assert call(T=0) == 0


# ---------------------------------------------------------------- refusals of the binding
@pytest.fixture
def ctx():
    """A Context over a stand-in, on the CPU "device" -1."""
    c = vit.Context.__new__(vit.Context)
    c.cfg = vit.VitConfig(1152, 16, 72, 64, 1e-6, 1e4, vit.BF16, 0)
    c._buf, c._h, c._device = fake(), None, -1
    return c


def refused(code, f, *a, **kw):
    with pytest.raises(vit.VitError) as e:
        f(*a, stream=0, **kw)
    assert e.value.code == code


def test_binding_checks_types_shapes_and_strides(ctx):
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    u = lambda *s: torch.zeros(*s, dtype=torch.uint8)     # noqa: E731
    x, g = b(4, 64), b(64)
    refused(BAD, ctx.rmsnorm, x.float(), g, b(4, 64))
    refused(BAD, ctx.rmsnorm, b(64, 4).t(), g, b(4, 64))
    refused(SHAPE, ctx.rmsnorm, x, b(32), b(4, 64))
    refused(SHAPE, ctx.rmsnorm, x, g, b(4, 32))
    refused(SHAPE, ctx.rmsnorm, x, g, b(4, 64), residual=b(3, 64))
    refused(BAD, ctx.rmsnorm, x, g, b(4, 64), h=torch.zeros(4, 64))
    refused(SHAPE, ctx.rmsnorm_mx8, x, g, u(4 * 63), u(512))
    refused(SHAPE, ctx.rmsnorm_mx8, x, g, u(4, 64), u(511))
    refused(BAD, ctx.rmsnorm_mx8, x, g, b(4, 64), u(512))
    refused(SHAPE, ctx.mx4_quantize, b(4, 70), u(4, 47), u(512))
    refused(BAD, ctx.mx4_quantize, b(4, 140)[:, ::2], u(4, 48), u(512))
    refused(SHAPE, ctx.mx4_dequantize, u(4, 48), u(100), b(4, 70))
    a, w = (u(4, 48), u(512)), (u(16, 48), u(512))
    refused(SHAPE, ctx.linear_mx4, a, a, None, b(4, 16), 70)           # W too small
    refused(BAD, ctx.linear_mx4, a, w, torch.zeros(16), b(4, 16), 70)
    refused(SHAPE, ctx.linear_mx4, a, w, b(15), b(4, 16), 70)
    refused(SHAPE, ctx.linear_mx4, a, w, None, b(4, 16), 70, epi=2, residual=b(4, 8))
    q, pos = b(5, 3, 72), torch.zeros(5, 3, dtype=torch.int32)
    refused(BAD, ctx.rope3d, q, pos.long(), (12, 12, 12))
    refused(SHAPE, ctx.rope3d, q, pos[:4], (12, 12, 12))
    refused(SHAPE, ctx.rope3d, q, pos, (18, 18))
    refused(SHAPE, ctx.rope3d, b(5, 3, 64), pos, (12, 12, 12))
    refused(BAD, ctx.rope3d, b(5, 72, 3).transpose(1, 2), pos, (12, 12, 12))
    refused(BAD, ctx.rope3d, b(5, 6, 72)[:, ::2], pos, (12, 12, 12))
    refused(SHAPE, ctx.rope3d, q, pos, (12, 12, 12), out=b(5, 2, 72))


def test_binding_takes_empty_batches(ctx):
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    u = lambda *s: torch.zeros(*s, dtype=torch.uint8)     # noqa: E731
    ctx.rmsnorm(b(0, 64), b(64), b(0, 64), residual=b(0, 64), h=b(0, 64), stream=0)
    ctx.rmsnorm_mx8(b(0, 64), b(64), u(0, 64), u(0), stream=0)
    ctx.mx4_quantize(b(0, 70), u(0, 48), u(0), stream=0)
    ctx.mx4_dequantize(u(0, 48), u(0), b(0, 70), stream=0)
    ctx.linear_mx4((u(0, 48), u(0)), (u(16, 48), u(512)), b(16), b(0, 16), 70, stream=0)
    ctx.rope3d(b(0, 4, 72), torch.zeros(0, 3, dtype=torch.int32), (12, 12, 12), stream=0)
    refused(SHAPE, ctx.rmsnorm, b(0, 64), b(32), b(0, 64))  # checked all the same


def test_closed_context_and_wrong_kinds_of_arguments(ctx):
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    refused(BAD, ctx.rmsnorm, b(4, 64), b(64), b(4, 64))  # all is well but the handle
    for bad in (None, 3, "x"):
        with pytest.raises((AttributeError, TypeError)):
            ctx.rmsnorm(bad, b(64), b(4, 64), stream=0)
        with pytest.raises((AttributeError, TypeError)):
            ctx.rmsnorm(b(4, 64), b(64), bad, stream=0)
    with pytest.raises(TypeError):
        ctx.rope3d(b(5, 3, 72), torch.zeros(5, 3, dtype=torch.int32), (12, 12, 12.5), stream=0)
    refused(SHAPE, ctx.rmsnorm, b(64), b(64), b(64))      # one dimension
    refused(BAD, ctx.linear_mx4, (None, None), (None, None), None, b(4, 16), -1)


def test_choices_past_an_int_are_refused_not_cut_off(ctx):
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    u = lambda *s: torch.zeros(*s, dtype=torch.uint8)     # noqa: E731
    for v in (1 << 32, -(1 << 32), (1 << 32) + 1):        # 0 and 1 in their low 32 bits
        refused(BAD, ctx.linear_mx4, (u(0, 48), u(0)), (u(16, 48), u(512)), None, b(0, 16), 70,
                epi=v)
        refused(BAD, ctx.rope3d, b(0, 4, 72), torch.zeros(0, 3, dtype=torch.int32), (12, 12, 12),
                layout=v)
