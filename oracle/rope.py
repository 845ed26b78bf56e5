"""Position rotation of heads, in fp64.

Pair i of a head at position p turns by the angle p f_i:
(x_a, x_b) -> (x_a cos - x_b sin, x_b cos + x_a sin), with pair i = (i, i + r/2)
of the first r = 2 len(f) values, or (2i, 2i + 1) when interleaved.  The
rotation is orthogonal, so its backward is the rotation by -p.
"""
from __future__ import annotations

import numpy as np


def rotate(x, positions, inv_freq, interleaved=False, back=False):
    """x [tokens][heads][d]; positions [tokens]; inv_freq [r / 2]."""
    x = np.array(x, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.float64)
    a = np.asarray(positions, dtype=np.float64)[:, None] * f
    cos, sin = np.cos(a)[:, None], (-1 if back else 1) * np.sin(a)[:, None]
    h = len(f)
    first = slice(0, 2 * h, 2) if interleaved else slice(0, h)
    second = slice(1, 2 * h, 2) if interleaved else slice(h, 2 * h)
    xa, xb = x[..., first].copy(), x[..., second].copy()
    x[..., first] = xa * cos - xb * sin
    x[..., second] = xb * cos + xa * sin
    return x
