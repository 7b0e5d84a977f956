"""Turn tables of ``oscar_norm_rope``: how far each pair of channels turns a position, on the host in 64 bits."""

import math

import numpy as np


def rope_turns(rot_dim, base=10000.0, scaling=None):
    """(turns, scale): int64 [rot_dim / 2] turns a position in units of 2^-64 (the bits of an unsigned fraction), and
    the factor on the rotated channels.

    Pair i turns base^(-2 i / rot_dim) radians a position. ``scaling`` stretches that for contexts longer than the
    trained one, as a dict with ``kind`` and ``factor`` (at least 1):
      "linear"  every pair slower by the factor;
      "ntk"     the base grows by factor^(rot_dim / (rot_dim - 2)): the fastest pair stays, the slowest gets the factor;
      "yarn"    pairs of at most ``slow`` (1) turns over the ``trained`` positions slower by the factor, of at least
                ``fast`` (32) as they are, a ramp over the pairs between them; scale = 0.1 ln(factor) + 1.
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim %s is not a positive even number" % (rot_dim,))
    if not (math.isfinite(base) and base > 1.0):
        raise ValueError("base %s is not a finite number above 1" % (base,))
    half, scale = rot_dim // 2, 1.0
    options = dict(scaling or {})
    kind, factor = options.pop("kind", None), float(options.pop("factor", 1.0))
    trained = options.pop("trained", None) if kind == "yarn" else None
    fast, slow = (float(options.pop(k, v)) if kind == "yarn" else v for k, v in (("fast", 32.0), ("slow", 1.0)))
    if options or (scaling is not None and kind not in ("linear", "ntk", "yarn")):
        raise ValueError("scaling %r: kind is linear, ntk or yarn, with factor (yarn: trained, fast and slow too)" % (scaling,))
    if not (math.isfinite(factor) and factor >= 1.0):
        raise ValueError("scaling factor %s is not a finite number of at least 1" % (factor,))
    if kind == "ntk" and rot_dim > 2:
        base *= factor ** (rot_dim / (rot_dim - 2))
    freq = [base ** (-2.0 * i / rot_dim) for i in range(half)]
    if kind == "linear":
        freq = [f / factor for f in freq]
    if kind == "yarn":
        if trained is None or not trained > 0 or not fast > slow > 0:
            raise ValueError("yarn needs trained > 0 and fast > slow > 0, got %r" % (scaling,))
        pair = lambda turns: rot_dim * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot_dim - 1)
        for i in range(half):
            ramp = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
            freq[i] = freq[i] / factor * ramp + freq[i] * (1.0 - ramp)
        scale = 0.1 * math.log(factor) + 1.0
    turns = [int(round(f / (2 * math.pi) * 2.0 ** 64)) for f in freq]
    return np.array(turns, np.uint64).view(np.int64), scale
