"""Turn tables of the rotation: the host arithmetic against its definition, and what it refuses."""

import math

import numpy as np
import pytest

from bit_kv_cache_write_gb300 import rope


def radians(turns):
    return np.asarray(turns).view(np.uint64).astype(np.float64) * 2 * np.pi / 2.0 ** 64


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (8, 500.0), (64, 10000.0), (128, 1e6)])
def test_unscaled_turns(rot, base):
    turns, scale = rope.rope_turns(rot, base)
    assert turns.dtype == np.int64 and turns.shape == (rot // 2,) and scale == 1.0
    np.testing.assert_allclose(radians(turns), [base ** (-2 * i / rot) for i in range(rot // 2)], rtol=1e-12)


def test_linear_and_ntk():
    plain, _ = rope.rope_turns(64, 1e4)
    lin, _ = rope.rope_turns(64, 1e4, dict(kind="linear", factor=4))
    np.testing.assert_allclose(radians(lin) * 4, radians(plain), rtol=1e-12)
    ntk, scale = rope.rope_turns(64, 1e4, dict(kind="ntk", factor=4))
    assert scale == 1.0
    np.testing.assert_allclose(radians(ntk)[0], radians(plain)[0], rtol=1e-12)
    np.testing.assert_allclose(radians(ntk)[-1] * 4, radians(plain)[-1], rtol=1e-12)


def test_yarn_keeps_fast_pairs_and_slows_slow_ones():
    plain, _ = rope.rope_turns(128, 1e6)
    got, scale = rope.rope_turns(128, 1e6, dict(kind="yarn", factor=8, trained=32768))
    ratio = radians(plain) / radians(got)
    made = radians(plain) * 32768 / (2 * np.pi)           # turns over the trained positions
    assert scale == pytest.approx(0.1 * math.log(8) + 1)
    np.testing.assert_allclose(ratio[made > 40], 1.0, rtol=1e-12)
    # turns are rounded to whole units: half a unit of the smallest, 2^64 1e-6^(126/128) / (2 pi) / 8 = 4.5e11 units, is
    # 1.1e-12 of it, an eighth of that of the unscaled one: 1.3e-12 in a ratio, 2 * 8 * 1.3e-12 between two of them
    np.testing.assert_allclose(ratio[made < 0.8], 8.0, rtol=2e-12)
    assert (np.diff(ratio) >= -2.5e-11).all() and ((ratio > 1.01) & (ratio < 7.9)).any()


def test_factor_of_one_changes_nothing():
    for kind, more in (("linear", {}), ("ntk", {}), ("yarn", dict(trained=4096))):
        turns, scale = rope.rope_turns(64, 1e4, dict(kind=kind, factor=1.0, **more))
        assert scale == 1.0
        np.testing.assert_allclose(radians(turns), radians(rope.rope_turns(64, 1e4)[0]), rtol=1e-12)


@pytest.mark.parametrize("args", [
    (0,), (7,), (-2,), (64, 1.0), (64, math.nan), (64, math.inf), (64, 1e4, dict(kind="other", factor=2)),
    (64, 1e4, dict(factor=2)), (64, 1e4, dict(kind="linear", factor=0.5)), (64, 1e4, dict(kind="linear", factor=math.nan)),
    (64, 1e4, dict(kind="linear", factor=2, trained=4)), (64, 1e4, dict(kind="yarn", factor=2)),
    (64, 1e4, dict(kind="yarn", factor=2, trained=0)), (64, 1e4, dict(kind="yarn", factor=2, trained=9, fast=1, slow=2)),
])
def test_refusals(args):
    with pytest.raises(ValueError):
        rope.rope_turns(*args)
