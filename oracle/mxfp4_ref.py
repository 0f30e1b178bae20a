"""fp64 CPU oracle of MXFP4 quantisation and its linear layer.  TEST
INFRASTRUCTURE, as mxfp8_ref.py.

Format (OCP Microscaling v1.0, MXFP4): E2M1 elements -- sign, 2 exponent bits
(bias 1), 1 mantissa bit; exponent field 0 holds 0 and 0.5; no infinity, no
NaN; largest value 6 -- in blocks of 32 consecutive elements of K sharing an
E8M0 scale 2^X (byte X + 127; 255 is NaN).  X = floor(log2(amax)) - 2 clamped
to [-127, 127], -127 for an all-zero block; elements x / 2^X rounded to nearest,
ties to even, magnitudes above 6 clamped to 6.  A block that holds a NaN has
scale byte 255 and zero codes.
"""
from __future__ import annotations

import numpy as np

__all__ = ["BLOCK", "e2m1_decode", "e2m1_encode", "mx4_quantize", "mx4_dequantize", "mx4_linear",
           "pack", "unpack"]

BLOCK = 32


def e2m1_decode(codes):
    """E2M1 codes (0..15) -> fp64 values, from the bit fields."""
    c = np.asarray(codes, dtype=np.int64)
    e, m = (c >> 1) & 3, c & 1
    v = np.where(e == 0, 0.5 * m, (1 + 0.5 * m) * np.exp2(e - 1.0))
    return np.where(c & 8, -v, v)


def e2m1_encode(x):
    """fp64 values -> E2M1 codes: nearest value, ties to the even code, at most 6."""
    x = np.asarray(x, dtype=np.float64)
    grid = e2m1_decode(np.arange(8))
    mid = (grid[1:] + grid[:-1]) / 2
    a = np.abs(x)
    lo = np.searchsorted(mid, a, side="left")    # a tie stays below
    hi = np.searchsorted(mid, a, side="right")   # a tie goes up
    return (np.where(lo % 2 == 0, lo, hi) | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def _padded(x):
    x = np.asarray(x, dtype=np.float64)
    return np.pad(x, ((0, 0), (0, -x.shape[1] % BLOCK))).reshape(x.shape[0], -1, BLOCK)


def mx4_quantize(x):
    """[R, K] -> (E2M1 codes [R, K], E8M0 scale bytes [R, ceil(K/32)])."""
    g = _padded(x)
    nan = np.isnan(g).any(-1)
    amax = np.where(nan, 0.0, np.abs(g).max(-1))
    _, fe = np.frexp(np.where(np.isinf(amax), 1.0, amax))
    X = np.where(amax > 0, fe - 1 - 2, -127)
    X = np.clip(np.where(np.isinf(amax), 126, X), -127, 127)  # infinities: as magnitude 2^128
    codes = e2m1_encode(g / np.exp2(X.astype(np.float64))[..., None])
    codes = np.where(nan[..., None], 0, codes).astype(np.uint8)
    scales = np.where(nan, 255, X + 127).astype(np.uint8)
    return codes.reshape(g.shape[0], -1)[:, :np.asarray(x).shape[1]], scales


def mx4_dequantize(codes, scales):
    """(codes [R, K], scale bytes [R, nb]) -> fp64 [R, K]."""
    s = np.asarray(scales, dtype=np.int64)
    p = np.where(s == 255, np.nan, np.exp2(s - 127.0))
    return (_padded(e2m1_decode(codes)) * p[..., None]).reshape(p.shape[0], -1)[:, :codes.shape[1]]


def mx4_linear(a, w, bias=None, epilogue="none", residual=None):
    """y = deq(a) deq(w)^T + b and the epilogue; a and w are (codes, scales)."""
    y = mx4_dequantize(*a) @ mx4_dequantize(*w).T
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)
    if epilogue == "gelu":
        y = 0.5 * y * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (y + 0.044715 * y ** 3)))
    elif epilogue == "residual":
        y = y + np.asarray(residual, dtype=np.float64)
    elif epilogue != "none":
        raise ValueError(epilogue)
    return y


def pack(codes):
    """Codes [R, K] two a byte, the even column in the low nibble; rows of
    16 ceil(K/32) bytes, zeros past K."""
    c = np.pad(np.asarray(codes, dtype=np.uint8), ((0, 0), (0, -codes.shape[1] % BLOCK)))
    return c[:, 0::2] | (c[:, 1::2] << 4)


def unpack(packed, K):
    """The inverse of pack for K columns."""
    p = np.asarray(packed, dtype=np.uint8)
    return np.stack((p & 15, p >> 4), -1).reshape(p.shape[0], -1)[:, :K]
