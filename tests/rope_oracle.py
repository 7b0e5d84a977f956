"""fp64 definition of oscar_norm_rope for the tests, and the error that its arithmetic allows."""

import numpy as np


def norm_rope(x, weight, eps, turns, interleaved, scale, positions):
    """(y, bound): x [n, H, d] float64; turns: Python ints (units of 2^-64 of a turn); positions [n] ints.

    bound, derived from the fp32 arithmetic: the sum of squares (8 products a lane, up to 4 rounds of shuffles), half of
    whose relative error enters the root, rsqrtf (2 ulp), eps and three products: below 16 * 2^-24 of y. Sine and cosine
    are off by 2 ulp, their argument by a rounding (2^-24 of at most pi), the products and the sum by one each: below
    12 * 2^-23 of scale (|a| + |b|). In all below 2^-19 (|a| + |b|), and the rounding to bf16."""
    x = np.asarray(x, np.float64)
    y = x if weight is None else np.asarray(weight, np.float64) * (x / np.sqrt((x * x).mean(-1, keepdims=True) + eps))
    rot = 2 * len(turns)
    got, mag = y.copy(), np.abs(y)
    for i in range(len(turns)):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, rot // 2 + i)
        frac = [((int(p) * int(turns[i])) % (1 << 64)) / 2.0 ** 64 for p in positions]
        t = 2 * np.pi * np.array(frac)[:, None]
        ya, yb = y[..., a], y[..., b]
        got[..., a], got[..., b] = scale * (ya * np.cos(t) - yb * np.sin(t)), scale * (yb * np.cos(t) + ya * np.sin(t))
        mag[..., a] = mag[..., b] = abs(scale) * (np.abs(ya) + np.abs(yb))
    err = 2.0 ** -19 * mag
    return got, err + 2.0 ** -8 * (np.abs(got) + err)
