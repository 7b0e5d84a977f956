"""Steps of the key bounds from calibration keys that are not all numbers."""

import numpy as np
import pytest

from bit_kv_cache_write_gb300 import calibration


def test_nan_keys_are_refused():
    """A channel with a NaN has no largest magnitude, and no int8 stands for its step."""
    k = np.ones((3, 2, 64))
    k[1, 0, 5] = np.nan
    with pytest.raises(ValueError, match="NaN"):
        calibration.key_steps(k)


def test_no_keys_are_refused():
    with pytest.raises(ValueError):
        calibration.key_steps(np.ones((0, 2, 64)))


def test_infinite_keys_take_the_largest_step():
    k = np.ones((3, 2, 64))
    k[1, 0, 5] = -np.inf
    steps = calibration.key_steps(k)
    assert steps[0, 5] == 100 and (steps[1] == steps[0, 0]).all()
