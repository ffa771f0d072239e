"""Float64 reference of the norms and position rotation of queries and keys, row by row from the definition:

    y = w x / sqrt(mean_c x_c^2 + eps)   (y = x without w),
    (a, b) -> (a cos t - b sin t, a sin t + b cos t),   t = 2 pi frac(p F_i / 2^64),

for the pairs (i, i + R / 2) or (2 i, 2 i + 1) of the first R channels.  The angle's fraction of a turn is formed in whole
numbers.
"""
import numpy as np


def angles(positions, turns):
    """[T, n] in radians; turns: whole numbers modulo 2^64."""
    wrap = 1 << 64
    return np.array([[2 * np.pi * ((int(p) * (int(f) % wrap)) % wrap / wrap) for f in turns] for p in positions],
                    np.float64).reshape(len(positions), len(turns))


def norm_rope(x, weight, eps, positions, turns, interleaved):
    """x [T, heads, d].  Returns (y, spread): spread bounds the magnitudes that each result is a sum of."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    y, spread = x.copy(), np.abs(x)
    n = len(turns)
    t = angles(positions, turns)[:, None]
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y[..., a] = x[..., a] * np.cos(t) - x[..., b] * np.sin(t)
    y[..., b] = x[..., a] * np.sin(t) + x[..., b] * np.cos(t)
    spread[..., a] = spread[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, spread
