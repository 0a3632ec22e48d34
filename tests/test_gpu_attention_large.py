"""moe_paged_attention with values near the end of bf16's range."""

import pytest
import torch

from paged import Setup
from test_gpu_attention import _run, _wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,new,height", [(64, 1, 64), (128, 4, 64), (128, 20, 64), (128, 40, 128), (64, 70, 256)])
def test_weighted_sums_of_values_near_the_largest(D, new, height):
    """A maximum that rises by less than 2^8: sums of 2^118 at every position
    end below 2^128."""
    Hq = 8
    s = Setup([(new, 512 + new)], 1, D, page=16, max_pages=_wide(new, Hq, D, height))
    s.v.fill_(2.0 ** 118)
    s.k.zero_()
    for p in range(256, 512):
        s.k[s.place(0, p)][:, 0] = 5.1875
    q = torch.zeros((new, Hq, D), dtype=torch.bfloat16)
    q[..., 0] = 1.0
    _, out, _, _ = _run(s, Hq, q=q.view(new, -1), scale=1.0)
    # (all values are equal: the divisor is the sum of the same weights)
    assert bool(((out.double() - 2.0 ** 118).abs() <= 2.0 ** 110).all())
