"""fp64 CPU oracle of RMSNorm with the residual's addition and of RoPE over
three axes.  TEST INFRASTRUCTURE, as vit_ref.py.
"""
from __future__ import annotations

import numpy as np

__all__ = ["to_bf16", "rmsnorm", "rope3d_pairs", "rope3d"]


def to_bf16(a):
    """fp64 values rounded once to the nearest bf16 value (ties to even), as fp64."""
    a = np.asarray(a, dtype=np.float64)
    _, e = np.frexp(a)
    unit = np.ldexp(1.0, np.maximum(e - 8, -133))  # 8 significant bits, 2^-133 at the least
    r = np.rint(a / unit) * unit
    return np.where(np.abs(r) > 255 * 2.0 ** 120, np.copysign(np.inf, r), r)


def rmsnorm(h, gamma, eps):
    """h [R, C] -> h / sqrt(mean(h^2) + eps) * gamma."""
    h = np.asarray(h, dtype=np.float64)
    return h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * np.asarray(gamma, np.float64)


def rope3d_pairs(head_dim, sections, layout, theta=10000.0):
    """(lo, hi, axis, frequency) of each rotated pair; layout "blocks" (an axis
    has its own dims), "sections" or "turns" (pairs (j, j + d/2) shared out in
    one run per axis, or one at a time while an axis has any left)."""
    half = head_dim // 2
    assert sum(sections) == half
    theta = np.longdouble(theta)
    if layout == "blocks":
        out, at = [], 0
        for axis, n in enumerate(sections):
            out += [(at + j, at + n + j, axis, theta ** (-np.longdouble(j) / n)) for j in range(n)]
            at += 2 * n
        return out
    if layout == "sections":
        axes = np.repeat(np.arange(3), sections).tolist()
    else:
        axes, left = [], list(sections)
        while any(left):
            for a in range(3):
                if left[a]:
                    axes.append(a)
                    left[a] -= 1
    return [(j, j + half, axes[j], theta ** (-np.longdouble(2 * j) / head_dim)) for j in range(half)]


def rope3d(x, pos, sections, layout, theta=10000.0):
    """x [T, heads, d], pos [T, 3]: each pair (a, b) turned by pos[axis] * f
    (angles in extended precision: positions may be far)."""
    x = np.asarray(x, dtype=np.float64)
    y = np.empty_like(x)
    for lo, hi, axis, f in rope3d_pairs(x.shape[2], sections, layout, theta):
        angle = np.asarray(pos)[:, axis].astype(np.longdouble) * f
        c = np.cos(angle).astype(np.float64)[:, None]
        s = np.sin(angle).astype(np.float64)[:, None]
        y[..., lo] = x[..., lo] * c - x[..., hi] * s
        y[..., hi] = x[..., hi] * c + x[..., lo] * s
    return y
