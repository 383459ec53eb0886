"""Position rotation for the KV-cache oracle.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Pair i of a head's first rot_dim elements, (x_i, x_{i + rot_dim/2}) or
(x_{2i}, x_{2i+1}), is the complex number a + ib; the rotation multiplies it
by cos + i sin of the table row of the pair's position.  fp64 numpy.
"""
from __future__ import annotations

import numpy as np


def pair_columns(rot_dim: int, interleaved: bool):
    """Columns of the first and second elements of the pairs."""
    i = np.arange(rot_dim // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot_dim // 2)


def rotate(x, cos_sin, positions, interleaved: bool = False, pair_axis=None) -> np.ndarray:
    """x [T, H, D]; cos_sin [P, rot_dim]; positions [axes, T] -> fp64 [T, H, D]."""
    x = np.array(x, dtype=np.float64)
    cos_sin = np.asarray(cos_sin, dtype=np.float64)
    positions = np.atleast_2d(np.asarray(positions))
    half = cos_sin.shape[1] // 2
    first, second = pair_columns(2 * half, interleaved)
    out = x.copy()
    for i in range(half):
        p = positions[0 if pair_axis is None else pair_axis[i]]
        c, s = cos_sin[p, i][:, None], cos_sin[p, half + i][:, None]
        a, b = x[:, :, first[i]], x[:, :, second[i]]
        out[:, :, first[i]] = a * c - b * s
        out[:, :, second[i]] = b * c + a * s
    return out


def magnitude(x, rot_dim: int, interleaved: bool = False) -> np.ndarray:
    """|a| + |b| of each element's pair (|x| where nothing turns): what the
    fp32 rounding errors of a rotation are bounded by."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    first, second = pair_columns(rot_dim, interleaved)
    out = x.copy()
    out[..., first] = out[..., second] = x[..., first] + x[..., second]
    return out
