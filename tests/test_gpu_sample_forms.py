"""moe_sample and moe_verify_sample in both of their forms: one workgroup per
row (V <= 36,000, or many rows), and slices of a row per workgroup (few long
rows).  Each test runs with a vocabulary of either side; the tolerances are
those of test_gpu_sample.py."""

import numpy as np
import pytest
import torch

from test_gpu_sample import _check, _logits, _params

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [9001, 50257])
def test_logits_near_the_end_of_the_type(V):
    """A token forced with a huge finite logit, and rows whose bins cross the
    last values of fp32, at ordinary and at very large temperatures."""
    big = float(np.finfo(np.float32).max)
    rng = np.random.default_rng(V)
    x = _logits(12, V, 50)
    x[0, 17] = 3e38
    x[1, 17] = big
    x[2, [5, 17, 700]] = 3e38
    x[3] = big * rng.uniform(-1, 1, V)
    x[4] = x[3]
    x[4, 0] = big
    x[5] = 3e38 + 1e36 * rng.standard_normal(V)
    x[6] = np.minimum(big, 3.2e38 + 1e37 * rng.standard_normal(V))
    x[7] = rng.uniform(2.99e38, 3.01e38, V)
    x[8] = x[4]
    x[9] = -3e38 + 1e36 * rng.standard_normal(V)
    x[10, 5] = 3.0000001e38
    x[10, 6] = 2.9999999e38
    x[11] = np.where(rng.random(V) < 0.01, 3e38, x[11])
    p = _params(12, seed=11, min_p=0.0,
                temperature=[0.9, 0.9, 1.1, 1e38, 1e38, 1e36, 1e37, 1e36, 3e37, 1e36, 1e31, 0.7],
                top_k=[0, 50, 0, 0, 300, 0, 200, 0, 1000, 0, 0, 70],
                top_p=[1, 0.9, 1, 0.9, 0.8, 1, 0.95, 0.5, 1, 0.9, 1, 0.9])
    _check(x, p)
    _check(torch.as_tensor(np.clip(x, -3.3e38, 3.3e38)).to(torch.bfloat16), p)
