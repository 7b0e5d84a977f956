"""Pins of the paged-cache oracle, and what the paged calls refuse before they touch a device."""

import ctypes

import numpy as np
import pytest
import torch

from bit_kv_cache_write_gb300 import calibration
from bit_kv_cache_write_gb300 import oscar as O
from oracle import paged

P = 16


def test_plan_by_hand():
    # request 0 continues page 7 and needs one more; 1 appends nothing; 2 starts empty
    tables = np.array([[5, 7, 0, 0], [9, 0, 0, 0], [0, 0, 0, 0]])
    t, slots, rows, total, state = paged.plan_append([30, 4, 0], [3, 0, 17], [1, 2, 3, 4, 6], 1, tables, 22)
    assert t.tolist() == [[5, 7, 2, 0], [9, 0, 0, 0], [3, 4, 0, 0]]
    assert slots.tolist() == [7 * 16 + 14, 7 * 16 + 15, 2 * 16] + [3 * 16 + i for i in range(16)] + [4 * 16, -1, -1]
    assert rows.tolist() == [0, 3, 3, 20] and total.tolist() == [33, 4, 17] and state.tolist() == [4, 20, 0, -1]


def test_plan_rejects_and_goes_on():
    # 0 needs two pages of one; 1 needs none; 2 has a negative length; 3 passes its row of the table
    t, slots, rows, total, state = paged.plan_append([0, 3, -1, 31], [17, 2, 4, 2], [8], 0, np.full((4, 2), 5), 25)
    assert state.tolist() == [0, 25, 3, 0] and total.tolist() == [0, 5, -1, 31]
    assert slots[:17].tolist() == [-1] * 17 and slots[17:19].tolist() == [5 * 16 + 3, 5 * 16 + 4]
    assert (slots[19:] == -1).all() and (t == 5).all()


def test_key_codes():
    assert paged.key_codes([0.5, 1.5, -2.5, 1e30, -np.inf, np.nan], [0] * 6).tolist() == [0, 2, -2, 127, -127, 0]
    assert paged.key_codes([1.0, 1.0], [-3, 3]).tolist() == [8, 0]


def test_query_codes_cover_the_range():
    codes, e = paged.query_codes([1.0, -0.5, 0.0, 1e-9], [0] * 4)
    assert e == -6 and codes.tolist() == [64, -32, 0, 0]
    codes, e = paged.query_codes([0.999999, 0.0], [0, 0])
    assert e == -7 and codes.tolist() == [127, 0]
    assert paged.query_codes([0.0, 2.0 ** -70], [0, 0])[0].tolist() == [0, 0]


def test_key_steps_are_the_least_that_cover_the_calibration():
    k = np.random.default_rng(3).standard_normal((50, 2, 64)) * np.exp2(np.arange(64) - 40.0)
    k[:, 1, 5] = 0
    steps = calibration.key_steps(k)
    assert steps.dtype == np.int8 and steps[1, 5] == -100
    top = 1.25 * np.abs(k).max(0)
    live = top > 0
    assert (top[live] <= 127 * np.exp2(steps[live].astype(float))).all()
    assert (top[live] > 127 * np.exp2(steps[live] - 1.0)).all()
    assert np.abs(paged.key_codes(k, steps)).max() < 127                     # the margin: nothing saturates


def test_score_bounds_the_logits():
    """2^e sum max(u lo, u hi) is within the roundings of the largest q.k of the page."""
    r = np.random.default_rng(1)
    d = 64
    steps = np.full(d, -4)
    for _ in range(20):
        k, q = r.standard_normal((16, d)), r.standard_normal(d)
        c = paged.key_codes(k, steps)
        u, e = paged.query_codes(q, steps)
        score = np.maximum(u * c.min(0), u * c.max(0)).sum() * 2.0 ** e
        # a code is off by half a step of 2^-4, a query code by half of 2^e in steps
        slack = np.abs(q).sum() * 2.0 ** -5 + np.abs(c).max(0).sum() * 2.0 ** (e - 1)
        assert score >= (k @ q).max() - slack


def test_selection_windows_and_ties():
    d = 64
    bounds = np.zeros((40, 2, d), np.int64)
    bounds[:, 1] = 3                                          # every page scores alike: the lowest win
    args = ([np.ones(d)], np.zeros(d), bounds, np.arange(40), 600)
    assert paged.select(*args, 4, 64, 256) == [0, 1, 2, 3, 4, 5, 6, 7] + list(range(21, 38))
    assert paged.select(*args, 0, 0, 1) == [37]
    assert paged.select(*args, 100, 64, 256) == list(range(38))
    assert paged.select([np.ones(d)], np.zeros(d), bounds, np.arange(40), 0, 4, 64, 256) == []
    bounds[30, 1] = 4
    assert paged.select([np.ones(d)], np.zeros(d), bounds, np.arange(40), 640, 1, 16, 16) == [0, 30, 39]


def test_decode_of_one_token_and_of_none():
    r = np.random.default_rng(2)
    pool = r.standard_normal((3, 2, 2, P, 64))
    q = r.standard_normal((2, 4, 64))
    out = paged.decode(q, pool, np.array([[2, 0], [1, 0]]), [1, 0], 0.125)
    assert np.allclose(out[0].reshape(2, 2, 64), pool[2, :, 1, 0][:, None]) and (out[1] == 0).all()


def test_append_starts_a_page_anew_and_widens_it():
    pool, bounds = np.zeros((2, 1, 2, P, 64)), np.full((2, 1, 2, 64), 99, np.int64)
    k = np.arange(3)[:, None, None] * np.ones((1, 1, 64))
    paged.append(pool, bounds, k, k, [16, 17, 5], np.zeros((1, 64)))
    assert bounds[1, 0, :, 0].tolist() == [0, 1]             # rows 0 and 1: a fresh page
    assert bounds[0, 0, :, 0].tolist() == [2, 99]            # row 5 widens what was there
    paged.append(pool, bounds, k[2:] * 4, k[2:], [18], np.zeros((1, 64)))
    assert bounds[1, 0, :, 0].tolist() == [0, 8] and pool[1, 0, 0, 2, 0] == 8


def test_null_context_is_refused(liboscar):
    n = None
    assert liboscar.oscar_plan_append(n, n, n, 0, n, 0, n, n, 0, n, 0, n, n, n, n) == -1
    assert liboscar.oscar_append_bf16(n, n, 0, n, 0, n, 0, n, 0, n, n, n) == -1
    assert liboscar.oscar_decode_bf16(n, n, 0, n, 0, n, 0, n, 0, n, 0, n, 0, 0, n) == -1
    assert liboscar.oscar_decode_bf16_sparse(n, n, 0, n, 0, n, n, n, 0, n, 0, 0, n, n, n, 0, n, 0, 0, n) == -1
    assert liboscar.oscar_decode_bf16_workspace_size(n, 1, 100) == 0
    assert liboscar.oscar_decode_bf16_sparse_workspace_size(n, 1, 100, 4) == 0
    assert liboscar.oscar_sparse_capacity(n, 4) == 0


def test_binding_refuses_host_tensors(liboscar, monkeypatch):
    monkeypatch.setitem(O._configs, 12345, (4, 2, 64, 0, 21))
    bf = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k must be a CUDA tensor"):
        O.oscar_append_bf16(12345, bf, bf, torch.zeros(2, dtype=torch.int64), torch.zeros(4096, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        O.oscar_decode_bf16(12345, bf, bf, bf, bf, 1, bf, None)
    with pytest.raises(ValueError, match="not created by oscar_create"):
        O.oscar_decode_bf16(54321, bf, bf, bf, bf, 1, bf, None)
