"""Sizes of MXFP8 scale buffers up to the largest row counts an int holds, and the
overlap check of vit_rmsnorm_mx8 that goes by them (on a stand-in for a context: a
refusal reads its configuration alone)."""
import ctypes

import pytest

import vision_transformer_encoder_layernorm_b200 as vit

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("rows,K", [(TOP, 8), (TOP - 126, 128), (TOP - 127, 8), (TOP, 16384),
                                    (8, TOP), (TOP, TOP)])
def test_scale_bytes_of_large_matrices(rows, K):
    want = -(-rows // 128) * -(-K // 128) * 512
    assert vit.mx8_scale_bytes(rows, K) == want
    assert vit.mx4_scale_bytes(rows, K) == want


def test_overlap_check_of_many_rows():
    buf = ctypes.create_string_buffer(1 << 16)
    cfg = vit.VitConfig(1152, 16, 72, 64, 1e-6, 1e4, vit.BF16, 0)
    ctypes.memmove(buf, ctypes.byref(cfg), ctypes.sizeof(cfg))
    G = 1 << 40  # far apart: x, gamma and codes take 32 GB, scales 8 GB

    def call(scales):
        return vit.lib.vit_rmsnorm_mx8(buf, G, None, 5 * G, None, TOP, 8, 1e-6, 2 * G, scales, None)
    inside = 1 << 30
    assert call(2 * G - inside) == 1         # the codes begin inside the scales
    assert call(G - inside) == 1             # x does
    assert call(5 * G - 2 ** 33 + 512) == 1  # gamma begins in their last block
