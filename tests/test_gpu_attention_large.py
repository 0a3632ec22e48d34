"""moe_paged_attention with values near the ends of their range."""

import numpy as np
import pytest
import torch

from oracle import attention as ref
from paged import Setup
from test_gpu_attention import _off, _run, _wide

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


@pytest.mark.parametrize("cache,power", [("bf16", -122), ("f8", -118)])
@pytest.mark.parametrize("D,new,height", [(64, 1, 64), (128, 4, 64), (256, 1, 64), (128, 40, 64), (128, 40, 128), (64, 70, 256)])
def test_values_near_the_smallest(cache, power, D, new, height):
    """Values of 2^-122, or of 8-bit codes whose scale is 2^-118, which a weight
    is multiplied with before it is rounded to bf16: half a step of the smallest
    bf16 numbers, 2^-134, is 2^-16 of that scale and counts for every position."""
    Hq, length = 8, 200 + new
    s = Setup([(new, length)], 1, D, cache, max_pages=_wide(new, Hq, D, height))
    if cache == "f8":
        s.v_scale.fill_(1.0)
    k, v, seen = s.sequence(0)
    if cache == "f8":
        s.v_scale.fill_(2.0 ** power)
    else:
        s.v = (s.v.float() * 2.0 ** power).bfloat16()
    q, out, _, _ = _run(s, Hq)
    t = np.unique(np.linspace(0, new - 1, 6).astype(int))
    want, *scales = ref.attend(q[t].double().numpy().reshape(len(t), Hq, D), k, v, s.positions(0)[t], seen,
                               float(np.float32(D ** -0.5)))
    got = out[t].double().numpy().reshape(want.shape) * 2.0 ** -power
    off = _off(cache == "f8", D, want, *scales) + length * 2.0 ** -16 * np.abs(v).mean(axis=0)
    # (and values below 2^-126 themselves, of few bits)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + off + (2.0 ** -11 if cache == "bf16" else 0.0)).all()
