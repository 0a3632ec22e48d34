"""moe_sample and moe_verify_sample in both of their forms: one workgroup per
row (V <= 36,000, or many rows), and slices of a row per workgroup (few long
rows).  Each test runs with a vocabulary of either side; the tolerances are
those of test_gpu_sample.py."""

import numpy as np
import pytest
import torch

from oracle import around
from test_gpu_sample import _call, _check, _expect, _logits, _params

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


@pytest.mark.parametrize("V", [9001, 50257])
def test_the_last_kept_token(V):
    """u >= 1 takes the last kept token, however little it weighs: alone, in
    runs of equal logits (more than a wave searches, more than the list
    holds), behind top-k, top-p and min-p."""
    x = np.full((10, V), -np.inf, np.float32)
    x[:, 3] = 0.0
    x[0, 900] = -40.0
    x[1, [900, 77, 8000]] = [-38.0, -40.5, -41.9]
    x[2, 100:200] = -40.0
    x[3, 100:] = -39.0
    x[4, 100:] = -39.0
    x[5, 100:200] = -39.0
    x[6, 100:200] = -2.0
    x[7] = _logits(1, V, 60)[0]
    x[8, 100:110] = -41.5
    x[9, 100:300] = np.linspace(-41, -30, 200)
    p = _params(10, temperature=1.0, min_p=[0, 0, 0, 0, 0, 0, 0.1, 0, 0, 0],
                top_k=[0, 0, 0, 0, V // 2, 58, 30, 100, 5, 100],
                top_p=[1, 1, 1, 1, 1, 1, 0.9, 1, 1, 1], u=[1, 2, 1, 1, 1, np.inf, 1, 1, 1, 1])
    t = torch.as_tensor(x)
    tok, prob = _call(t.cuda(), p)
    order = [np.argsort(-r.astype(np.float64), kind="stable") for r in x]
    want = [900, 8000, 199, V - 1, 100 + V // 2 - 2, 156, None, order[7][99], 103, order[9][99]]
    want[6] = around.sample_row(x[6], 1.0, 1.0, 30, float(np.float32(0.9)), float(np.float32(0.1)))[0]
    np.testing.assert_array_equal(tok, want)
    probs = np.array([around.sample_row(x[t], 1.0, 1.0, int(p["top_k"][t]), float(p["top_p"][t]),
                                        float(p["min_p"][t]))[1] for t in range(10)])
    assert (np.abs(prob - probs) <= 2.0 ** -23 * probs + 1e-30).all()


@pytest.mark.parametrize("V,T", [(36001, 54), (36001, 55), (36000, 60), (50257, 76), (50257, 77)])
def test_either_side_of_the_rule_in_the_workspace_asked_for(V, T):
    """The last batch in slices and the first with a workgroup per row: equal
    to each row by itself, and nothing behind the workspace is written."""
    import routed_expert_ffn_gemv_amd as moe
    x = _logits(T, V, T)
    p = _params(T, seed=T)
    d = {k: torch.as_tensor(v, device="cuda") for k, v in p.items()}
    u = d.pop("u")
    xs = torch.as_tensor(x, device="cuda")
    size = moe.moe_sample_workspace_size(T, V)
    ws = torch.full((size + 65536,), 0x5A, dtype=torch.uint8, device="cuda")
    tok = torch.full((T,), -5, dtype=torch.int32, device="cuda")
    prob = torch.zeros(T, device="cuda")
    moe.moe_sample(xs, T, V, u, tok, ws[:size], prob=prob, **d)
    torch.cuda.synchronize()
    want, want_p = _expect(x.astype(np.float64), p)
    np.testing.assert_array_equal(tok.cpu().numpy(), want)
    assert (np.abs(prob.cpu().numpy() - want_p) <= 2.0 ** -23 * want_p + 1e-30).all()
    assert bool((ws[size:] == 0x5A).all())
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    one_p = torch.zeros(1, device="cuda")
    for t in (0, T // 2, T - 1):
        moe.moe_sample(xs[t:t + 1], 1, V, u[t:t + 1], one, ws[:size], prob=one_p,
                       **{k: v[t:t + 1] for k, v in d.items()})
        torch.cuda.synchronize()
        assert int(one) == int(tok[t]) and float(one_p) == float(prob[t])


@pytest.mark.parametrize("V", [9001, 50257])
def test_drafts_right_behind_the_tokens(V):
    """Drafts that touch the tokens' ends are drafts like others."""
    import routed_expert_ffn_gemv_amd as moe
    T = 4
    x = _logits(T, V, 70)
    p = _params(T, seed=70)
    want, _ = _expect(x.astype(np.float64), p)
    d = {k: torch.as_tensor(v, device="cuda") for k, v in p.items()}
    u = d.pop("u")
    ws = torch.empty(moe.moe_sample_workspace_size(T, V), dtype=torch.uint8, device="cuda")
    for drafts, tokens in ((slice(0, 3), slice(3, 7)), (slice(4, 7), slice(0, 4))):
        buf = torch.full((7,), -5, dtype=torch.int32, device="cuda")
        buf[drafts] = torch.as_tensor([want[0], want[1], (want[2] + 1) % V], dtype=torch.int32)
        n = torch.zeros(1, dtype=torch.int32, device="cuda")
        moe.moe_verify_sample(torch.as_tensor(x, device="cuda"), T, V, buf[drafts], u, buf[tokens], n, ws, **d)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(buf[tokens].cpu().numpy(), want)
        assert int(n) == 3
