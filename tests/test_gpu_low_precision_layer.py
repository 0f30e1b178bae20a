"""RMSNorm, MXFP8 and MXFP4 projections and three-axis RoPE together, as the
attention half of a layer over a short clip runs them, eagerly and as a captured
graph; every step is checked against the oracle on that step's own inputs."""
import numpy as np
import pytest
import torch

import synth
from oracle import mxfp8_ref as MX
from oracle import norm_rope_ref as NR
from oracle import vit_ref as R
from tests.gpu_util import assert_close, from_dev, to_dev

pytestmark = pytest.mark.gpu

vit = pytest.importorskip("vision_transformer_encoder_layernorm_b200")

H, D, SEC = 4, 72, (12, 12, 12)
C = H * D
FRAMES = [(3, 6, 7), (2, 5, 5)]  # two clips of different shape


def _dev(shape, seed, scale=1.0):
    return to_dev(synth.random_tensor(shape, seed, "bf16", scale), "bf16")


def _mx(rows, K, row_bytes, scale_bytes):
    return (torch.empty(rows, row_bytes(K), dtype=torch.uint8, device="cuda"),
            torch.empty(scale_bytes(rows, K), dtype=torch.uint8, device="cuda"))


def test_attention_half_layer_over_clips():
    ctx = vit.Context(C, H, D, 4 * C, vit.BF16)
    lens = [t * r * c for t, r, c in FRAMES]
    T = sum(lens)
    pos = torch.cat([torch.cartesian_prod(*(torch.arange(n, dtype=torch.int32) for n in f))
                     for f in FRAMES]).cuda()
    cu = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32, device="cuda")
    sq = vit.seqs(T, len(lens), max(lens), cu)
    w_qkv, b_qkv = _dev((3 * C, C), 1, 0.05), _dev((3 * C,), 2, 0.1)
    w_o, b_o = _dev((C, C), 3, 0.05), _dev((C,), 4, 0.1)
    g1, g2 = _dev((C,), 5, 0.3), _dev((C,), 6, 0.3)
    wq = _mx(3 * C, C, vit.mx8_row_bytes, vit.mx8_scale_bytes)
    wo = _mx(C, C, vit.mx4_row_bytes, vit.mx4_scale_bytes)
    ctx.mx8_quantize(w_qkv, *wq)
    ctx.mx4_quantize(w_o, *wo)
    x, r = _dev((T, C), 7), _dev((T, C), 8)
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    b = {"h": e(T, C), "qkv": e(T, 3 * H, D), "o": e(T, C), "h2": e(T, C), "y": e(T, C)}
    n8 = _mx(T, C, vit.mx8_row_bytes, vit.mx8_scale_bytes)
    n4 = _mx(T, C, vit.mx4_row_bytes, vit.mx4_scale_bytes)

    def half(stream=None):
        ctx.rmsnorm_mx8(x, g1, *n8, residual=r, h=b["h"], stream=stream)
        ctx.linear_mx8(n8, wq, b_qkv, b["qkv"].view(T, 3 * C), C, stream=stream)
        ctx.rope3d(b["qkv"][:, :2 * H], pos, SEC, vit.ROPE_TURNS, stream=stream)
        ctx.attention(b["qkv"], b["o"], sq, stream=stream)
        ctx.mx4_quantize(b["o"], *n4, stream=stream)
        ctx.linear_mx4(n4, wo, b_o, b["h2"], C, epi=vit.EPI_BIAS_RESIDUAL, residual=b["h"],
                       stream=stream)
        ctx.rmsnorm(b["h2"], g2, b["y"], stream=stream)

    half()
    torch.cuda.synchronize()
    assert ctx.device_status() == 0
    got = {k: v.clone() for k, v in b.items()}
    # each step from the bf16 values the GPU had before it; bars of the steps'
    # own tests (a product's rounding, 2^-8 relative of the largest, 1e-2)
    assert torch.equal(got["h"], (x.float() + r.float()).bfloat16())
    n = NR.rmsnorm(from_dev(got["h"]), from_dev(g1), float(np.float32(1e-6)))
    qkv = MX.mx_project(NR.to_bf16(n), from_dev(w_qkv), from_dev(b_qkv)).reshape(T, 3 * H, D)
    qkv[:, :2 * H] = NR.rope3d(qkv[:, :2 * H], pos.cpu().numpy(), SEC, "turns")
    assert_close(from_dev(got["qkv"]), qkv, 1e-2, 0.9999, "qkv")
    q, k, v = (from_dev(got["qkv"]).reshape(T, 3, H, D)[:, i] for i in range(3))
    cu_h = cu.cpu().numpy()
    o = R.attention(q, k, v, cu_h, None)
    assert_close(from_dev(got["o"]).reshape(T, H, D), o, 2e-2, 0.9999, "attention")
    a4, w4 = e(T, C), e(C, C)
    ctx.mx4_dequantize(*n4, a4)
    ctx.mx4_dequantize(*wo, w4)
    h2 = from_dev(got["h"]) + from_dev(a4) @ from_dev(w4).T + from_dev(b_o)
    assert_close(from_dev(got["h2"]), h2, 1e-2, 0.9999, "output projection")
    y = NR.rmsnorm(from_dev(got["h2"]), from_dev(g2), float(np.float32(1e-6)))
    assert np.array_equal(from_dev(got["y"]), NR.to_bf16(y))
    # the same work as a captured graph, on buffers that hold something else before
    st = ctx.graph_begin()
    half(st)
    graph = ctx.graph_end()
    assert graph.kernels == 7
    for t in b.values():
        t.fill_(float("nan"))
    graph.launch()
    torch.cuda.synchronize()
    for name, t in b.items():
        assert torch.equal(t, got[name]), name
    graph.close()
    ctx.close()
