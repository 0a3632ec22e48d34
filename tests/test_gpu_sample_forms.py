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


VS = (9001, 50257)


@pytest.mark.parametrize("V", VS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masks_infinities_and_nan(V, dtype):
    x = _logits(12, V, 80)
    low = float(torch.finfo(dtype).min)
    x[0, :] = -np.inf                        # nothing left
    x[1, :] = -np.inf
    x[1, 777] = -3.0                         # one left
    x[2, ::2] = -np.inf
    x[3, 5:] = low                           # the type's lowest value is a logit like another
    x[4, :] = low
    x[5, ::3] = np.nan
    x[6, :] = np.nan
    x[7, [8, 100, 4000]] = np.inf            # equal infinities share the draw
    x[8, :] = -np.inf
    x[8, V - 1] = low
    x[9, ::5] = np.inf
    x[10, [0, V - 1]] = np.inf
    x[10, 1:V - 1:2] = np.nan
    x[11, :V - 2] = -np.inf                  # the last two, of one value
    x[11, V - 2:] = -7.5
    p = _params(12, temperature=[0.9] * 9 + [np.inf, 1e-40, 0.3], top_k=[0] * 9 + [1000, 0, 0],
                top_p=[0.97] * 9 + [0.4567, 1, 1], min_p=0.0, seed=80)
    t = torch.as_tensor(x).to(dtype)
    _check(t, p)
    tok, prob = _call(t.cuda(), p)
    assert tok[0] == tok[6] == -1 and prob[0] == prob[6] == 0


@pytest.mark.parametrize("V", VS)
def test_every_extreme_parameter(V):
    T = 16
    p = _params(T, seed=81,
                temperature=[0, -1, np.nan, 1e-30, 1e-45, 1e30, np.inf, 1, 1, 1, 1, 1, 1, 1, 1, 100],
                top_k=[0, 0, 0, 0, 0, 0, 0, -4, 2 ** 31 - 1, V, V + 1, 1, 0, 0, 0, V - 1],
                top_p=[1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, np.nan, 1.5, -2, 0.9],
                min_p=[0, 0, 0, 0, 0, 0, 0, np.nan, -1, 0, 0, 0, 1, 2, 0, 0],
                u=[0.5, 0.5, 0.5, 0.5, 0.5, 0.31, 0.77, 0.2, 0.4, 0.6, 0.8, 0.9, 0.3, 0.9, 0.9, 0.77])
    _check(_logits(T, V, 81), p)


@pytest.mark.parametrize("V", VS)
def test_draws_outside_the_unit_interval(V):
    x = np.repeat(_logits(1, V, 82), 6, axis=0)
    u = np.array([0.0, 1.0, 5.0, -1.0, np.nan, 1 - 2.0 ** -24], np.float32)
    order = np.argsort(-x[0].astype(np.float64), kind="stable")
    for k, top_p, last in ((40, 1.0, order[39]), (3000, 1.0, order[2999]), (0, 1e-9, order[0])):
        tok, _ = _call(torch.as_tensor(x).cuda(), _params(6, temperature=1.0, top_k=k, top_p=top_p, min_p=0.0, u=u))
        assert tok[0] == tok[3] == tok[4] == order[0]
        assert tok[1] == tok[2] == tok[5] == last


@pytest.mark.parametrize("off", ["temperature", "top_k", "top_p", "min_p", None])
@pytest.mark.parametrize("V", VS)
def test_parameters_one_by_one_left_out(V, off):
    off = {off: None} if off else dict.fromkeys(("temperature", "top_k", "top_p", "min_p"))
    _check(_logits(8, V, 83), _params(8, seed=83, **off))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,off", [(1, 0), (3, 1), (0, 2), (5, 3), (7, 7)])
def test_rows_that_start_anywhere(dtype, pad, off):
    """Slices of rows that start and end inside 16 bytes, between large logits."""
    T, V = 7, 50257
    x = torch.as_tensor(_logits(T, V, 84)).to(dtype)
    buf = torch.full((T * (V + pad) + off + 8,), 1e30, dtype=dtype, device="cuda")
    view = buf[off:off + T * (V + pad)].view(T, V + pad)[:, :V]
    view.copy_(x)
    p = _params(T, seed=84)
    tok, prob = _call(view, p)
    want, want_p = _expect(x.double().numpy(), p)
    np.testing.assert_array_equal(tok, want)
    assert (np.abs(prob - want_p) <= 2.0 ** -23 * want_p + 1e-30).all()


@pytest.mark.parametrize("T,V", [(1, 50257), (2, 50257), (4, 50257), (17, 50257), (64, 50257), (4, 151936),
                                 (1, 9001), (17, 9001), (64, 41000)])
def test_verify_in_both_forms(T, V):
    """Every number of kept drafts at the ends and in the middle; greedy rows,
    and rows with nothing to draw (token -1, which no draft is)."""
    x = _logits(T, V, 85 + T)
    if T > 2:
        x[T - 2] = -np.inf
    p = _params(T, seed=85)
    p["temperature"][::3] = 0.0
    want, want_p = _expect(x.astype(np.float64), p)
    xs = torch.as_tensor(x).cuda()
    for kept in sorted({0, 1, T // 2, T - 2, T - 1} & set(range(T))):
        draft = np.maximum(want[:T - 1], 0)
        if kept < T - 1:
            draft[kept] = (want[kept] + 1) % V
        n_want = next((i for i in range(T - 1) if draft[i] != want[i]), T - 1) + 1
        tok, prob, n = _call(xs, p, draft=draft, verify=True)
        np.testing.assert_array_equal(tok, want)
        assert (np.abs(prob - want_p) <= 2.0 ** -23 * want_p + 1e-30).all()
        assert n == n_want


def test_rows_alone_and_in_batches_of_either_form():
    """40,009 logits: 64 rows take a workgroup each, 61 and 1 go in slices."""
    V = 40009
    x = torch.as_tensor(_logits(64, V, 86)).cuda()
    p = _params(64, seed=86)
    tok, prob = _call(x, p)
    for rows in [slice(0, 60), slice(4, 64)] + [slice(t, t + 1) for t in (0, 13, 40, 63)]:
        a, b = _call(x[rows], {k: v[rows] for k, v in p.items()})
        np.testing.assert_array_equal(a, tok[rows])
        np.testing.assert_array_equal(b, prob[rows])


@pytest.mark.parametrize("V", VS)
def test_replayed_verify_pass(V):
    """Captured once; new logits, numbers and drafts between the replays."""
    import routed_expert_ffn_gemv_amd as moe
    T = 5
    p = _params(T, seed=87)
    par = {k: torch.as_tensor(v, device="cuda") for k, v in p.items() if k != "u"}
    logits, u = torch.zeros((T, V), device="cuda"), torch.zeros(T, device="cuda")
    draft = torch.zeros(T - 1, dtype=torch.int32, device="cuda")
    tok = torch.zeros(T, dtype=torch.int32, device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_sample_workspace_size(T, V), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_verify_sample(logits, T, V, draft, u, tok, n, ws, stream=side, **par)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_verify_sample(logits, T, V, draft, u, tok, n, ws, **par)
    for kept, seed in ((4, 90), (0, 91), (2, 92), (3, 93)):
        x = _logits(T, V, seed)
        p["u"] = np.random.default_rng(seed).random(T, dtype=np.float32)
        want, _ = _expect(x.astype(np.float64), p)
        d = want[:T - 1].astype(np.int32)
        if kept < T - 1:
            d[kept] = (d[kept] + 1) % V
        logits.copy_(torch.as_tensor(x))
        u.copy_(torch.as_tensor(p["u"]))
        draft.copy_(torch.as_tensor(d))
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(tok.cpu().numpy(), want)
        assert int(n) == kept + 1
        _call(logits, p)


def test_more_logits_than_31_bits_count():
    """16,384 rows of 151,936: the far rows' tokens, masked elsewhere."""
    import routed_expert_ffn_gemv_amd as moe
    T, V = 16384, 151936
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("12 GB of GPU memory wanted")
    x = torch.full((T, V), float("-inf"), dtype=torch.bfloat16, device="cuda")
    row = torch.arange(T, device="cuda")
    want = (row * 9973 + 5) % V
    x[row, want] = 1.5
    full = _logits(4, V, 88)
    far = [0, 14134, 14135, T - 1]           # element 2^31 lies in row 14,134
    for i, t in enumerate(far):
        x[t] = torch.as_tensor(full[i]).to(torch.bfloat16)
    p = _params(T, seed=88, temperature=0.8, top_k=50, top_p=0.9, min_p=0.0)
    par = {k: torch.as_tensor(v, device="cuda") for k, v in p.items()}
    u = par.pop("u")
    tok = torch.zeros(T, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_sample_workspace_size(T, V), dtype=torch.uint8, device="cuda")
    moe.moe_sample(x, T, V, u, tok, ws, **par)
    torch.cuda.synchronize()
    ref, _ = _expect(torch.as_tensor(full).to(torch.bfloat16).double().numpy(), {k: v[far] for k, v in p.items()})
    want = want.to(torch.int32)
    want[far] = torch.as_tensor(ref, dtype=torch.int32, device="cuda")
    assert torch.equal(tok, want)


def _largest_vocabulary():
    """2^26 logits, and of them those that a top-k of 40 can keep."""
    V = 1 << 26
    x = np.random.default_rng(95).standard_normal((2, V), dtype=np.float32) * 3
    x[1, 1 << 25:] = -np.inf
    few = [np.sort(np.argpartition(-r, 400)[:400]) for r in x]      # in the order of their indexes
    p = _params(2, temperature=[0.9, 2.0], top_k=40, top_p=[0.9, 1.0], min_p=0.0, u=[0.41, 0.77])
    want = []
    for t in range(2):
        tok, prob, slack = around.sample_row(x[t, few[t]], float(p["u"][t]), float(p["temperature"][t]), 40,
                                             float(p["top_p"][t]))
        assert slack > 2.0 ** -14                # w is held to 2^-17 of itself here
        want.append((few[t][tok], prob))
    return x, p, want


def test_the_largest_vocabulary():
    x, p, want = _largest_vocabulary()
    tok, prob = _call(torch.as_tensor(x).cuda(), p)
    assert tok.tolist() == [w[0] for w in want]
    assert (np.abs(prob - [w[1] for w in want]) <= 2.0 ** -16 * np.array([w[1] for w in want])).all()


def test_one_value_in_a_very_long_row():
    """2^24 + 3 equal logits: the token is the u-th part of them exactly."""
    V = (1 << 24) + 3
    x = torch.full((1, V), -2.5, dtype=torch.bfloat16, device="cuda")
    p = _params(1, temperature=0.7, top_k=None, top_p=None, min_p=None, u=0.618)
    tok, prob = _call(x, p)
    assert tok[0] == int(np.floor(np.float64(p["u"][0]) * V))
    assert abs(prob[0] * V - 1) <= 2.0 ** -23
