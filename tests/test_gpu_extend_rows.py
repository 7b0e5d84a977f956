"""oscar_extend_bf16: blocks that rows fill in part, rows that infinities and NaN reach."""

import pytest

from test_gpu_extend import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cached", [200, 20000])
@pytest.mark.parametrize("h_q", [1, 2])
def test_partly_filled_warps(cuda, d, cached, h_q):
    """Row counts around those of a warp and a block, in whole items and in parts: lanes with a row beside lanes without
    one."""
    new = [1, 2, 31, 32, 33, 63, 97, 127, 128, 129, 161, 255, 257]
    c = Case([(cached if m < 40 else cached % 301, m) for m in new], h_q, 1, d, seed=cached + h_q, spare=2)
    c.check(c.run(cuda))
