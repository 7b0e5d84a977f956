"""The bounds that the GPU tests of the paged decodes use see the mistakes that they are for, planted here in the
64-bit reference; and the vectorised selection is the oracle's."""

import numpy as np
import pytest
import torch

from oracle import paged
from paged_bounds import P, IntCache, attention, choose


def worst(got, want, bound):
    return float(((got - want).abs() / bound).max())


def rounded(x):
    return x.to(torch.bfloat16).double()


CASES = [([4099], 2, 64, 300, 2.0 ** -5), ([4099], 8, 128, 300, 2.0 ** -5), ([131070], 2, 128, 400, 2.0 ** -5),
         ([900], 4, 64, 300, 0.25)]


@pytest.mark.parametrize("lens,g,d,pages,scale", CASES, ids=str)
def test_the_bound_sees_the_mistakes_that_it_is_for(lens, g, d, pages, scale):
    c = IntCache(1, lens, g, 1, d, pages)
    want, bound = c.reference(scale)
    want, bound = want[0], bound[0]
    q = c.q[0].double()
    k, v = c.rows(0, 0)
    n = len(k)
    assert n == lens[0]
    seen = lambda keep, **how: worst(attention(q, k[keep], v[keep], scale, g, **how)[0], want, bound)
    every = torch.ones(n, dtype=torch.bool)
    without = lambda lo, hi: torch.cat([every[:lo], ~every[lo:hi], every[hi:]])
    assert seen(every) == 0
    assert seen(without(n - 1, n)) > 2                                    # the last token
    for page in (0, 7, 33, n // P - 2):
        assert seen(without(page * P, (page + 1) * P)) > 2                # one page
    assert seen(every, logits=rounded) > 2 and seen(every, weights=rounded) > 2
    one = torch.cat([torch.arange(n), torch.tensor([5])])                 # a token counted twice
    assert worst(attention(q, k[one], v[one], scale, g)[0], want, bound) > 1


def test_an_fp32_computation_is_within_the_bound():
    """The same sums in numpy's fp32, page by page with a running reference, as the bound's derivation has them."""
    c = IntCache(2, [2000], 4, 1, 64)
    want, bound = c.reference(0.25)
    q, (k, v) = c.q[0].float().numpy(), (x.float().numpy() for x in c.rows(0, 0))
    m, l, acc = np.full((4, 1), -3e38, np.float32), np.zeros((4, 1), np.float32), np.zeros((4, 64), np.float32)
    scale = np.float32(0.25 * 1.4426950408889634)
    for t in range(0, 2000, P):
        x = (q @ k[t:t + P].T) * scale
        top = x.max(1, keepdims=True)
        new = np.where(top > m + 8, top, m).astype(np.float32)
        f = np.exp2(np.maximum(m - new, np.float32(-1000)))
        p = np.exp2(x - new)
        m, l, acc = new, l * f + p.sum(1, keepdims=True), acc * f + p @ v[t:t + P]
    assert acc.dtype == np.float32 and worst(torch.from_numpy((acc / l).astype(np.float64)), want[0], bound[0]) < 1


@pytest.mark.parametrize("top", [0, 1, 9, 40, 500])
@pytest.mark.parametrize("length", [0, 5, 330, 700, 1600])
def test_choose_is_the_oracle_s_selection(length, top):
    c = IntCache(3, [1600], 4, 2, 64, 60)
    c.bounds[::3] = 5                                                     # ties
    c.tables[0, 30:33] = torch.tensor([-1, 10 ** 6, -7], dtype=torch.int32)
    q, steps, bounds, table = c.q[0].double().numpy(), c.steps.numpy(), c.bounds.numpy(), c.tables[0].numpy()
    got = choose(q, steps, bounds, table, length, top, 64, 256)
    assert got == [paged.select(q[h * 2:h * 2 + 2], steps[h], bounds[:, h], table, length, top, 64, 256) for h in range(2)]
