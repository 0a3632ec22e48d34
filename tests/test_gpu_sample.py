"""GPU parity of moe_sample and moe_verify_sample with the definition in 64
bits: tokens equal, probabilities to fp32's rounding.

A weight is held to 2^-(6 + frac) of itself, frac = min(28, 63 - 2 ceil(log2
V)): 2^-33 for the largest vocabulary here, half of that off at most.  A sum of
weights is off by less than 6e-11 of itself, and a bin's mass is rounded to
2^-43 of the largest weight besides.  A draw or a top-p cut nearer than SLACK to
the border between two tokens would be the test's mistake; none here is
(asserted).  prob: the token's weight is evaluated to 1e-14 and the kept sum as
above, then fp32's half step (2^-24)."""

import numpy as np
import pytest
import torch

from oracle import around

pytestmark = pytest.mark.gpu

SLACK = 1e-10


def _params(T, **kw):
    rng = np.random.default_rng(kw.pop("seed", 1))
    p = {
        "temperature": rng.uniform(0.4, 1.6, T).astype(np.float32),
        "top_k": rng.choice([0, 1, 2, 20, 200, 5000], T).astype(np.int32),
        "top_p": rng.choice([0.0, 0.3, 0.8, 0.95, 0.999, 1.0], T).astype(np.float32),
        "min_p": rng.choice([0.0, 0.0, 0.001, 0.05, 0.5], T).astype(np.float32),
        "u": rng.random(T, dtype=np.float32),
    }
    for k, v in kw.items():
        if v is None:
            p[k] = None
        else:
            p[k] = np.broadcast_to(np.asarray(v, np.int32 if k == "top_k" else np.float32), (T,)).copy()
    return p


def _call(logits, p, draft=None, verify=False, stream=None):
    """logits: a CUDA tensor [T][V].  Outputs have a guard entry."""
    import routed_expert_ffn_gemv_amd as moe
    T, V = logits.shape
    d = {k: None if v is None else torch.as_tensor(v, device="cuda") for k, v in p.items()}
    u = d.pop("u")
    tok = torch.full((T + 1,), -5, dtype=torch.int32, device="cuda")
    prob = torch.full((T + 1,), -5.0, device="cuda")
    n = torch.full((2,), -5, dtype=torch.int32, device="cuda")
    ws = torch.full((moe.moe_sample_workspace_size(T, V),), 0xA5, dtype=torch.uint8, device="cuda")
    if verify:
        dr = torch.as_tensor(np.asarray(draft, np.int32), device="cuda") if T > 1 else None
        moe.moe_verify_sample(logits, T, V, dr, u, tok, n, ws, prob=prob, stream=stream, **d)
    else:
        moe.moe_sample(logits, T, V, u, tok, ws, prob=prob, stream=stream, **d)
    torch.cuda.synchronize()
    tok, prob, n = tok.cpu().numpy(), prob.cpu().numpy(), n.cpu().numpy()
    assert tok[T] == -5 and prob[T] == -5 and n[1] == -5
    return (tok[:T], prob[:T], int(n[0])) if verify else (tok[:T], prob[:T])


def _expect(logits, p):
    off = {"temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0}
    toks, probs = [], []
    for t in range(logits.shape[0]):
        a = {k: (off[k] if p[k] is None else p[k][t].item()) for k in off}
        tok, prob, slack = around.sample_row(logits[t], float(p["u"][t]), **a)
        assert slack > SLACK, f"row {t}: the draw lies on a border"
        toks.append(tok)
        probs.append(prob)
    return np.array(toks), np.array(probs)


def _check(logits, p):
    """logits: numpy fp32, or a CPU bf16 tensor."""
    t = torch.as_tensor(logits)
    tok, prob = _call(t.cuda(), p)
    want, want_p = _expect(t.double().numpy(), p)
    np.testing.assert_array_equal(tok, want)
    assert (np.abs(prob - want_p) <= 2.0 ** -23 * want_p + 1e-30).all()


def _logits(T, V, seed, fall=1.2):
    """Falling off with the rank as a language model's, plus noise."""
    rng = np.random.default_rng(seed)
    x = np.stack([-fall * np.log1p(rng.permutation(V)) for _ in range(T)])
    return (x + 0.5 * rng.standard_normal((T, V)) + 5).astype(np.float32)


@pytest.mark.parametrize("V", [1, 2, 3, 7, 63, 64, 65, 500, 4095, 4096, 4097, 8200, 32000, 50257, 151936])
def test_vocabularies(V):
    """Whole and ragged slices; every filter on and off."""
    T = 24 if V < 60000 else 12
    _check(_logits(T, V, V), _params(T, seed=V))


@pytest.mark.parametrize("T", [1, 2, 63, 300, 1500])
def test_batches(T):
    """The rows are split over fewer workgroups as there are more of them."""
    V = 20011 if T <= 300 else 5003
    _check(_logits(T, V, T), _params(T, seed=T))


@pytest.mark.parametrize("off", ["temperature", "top_k", "top_p", "min_p"])
def test_parameters_left_out(off):
    _check(_logits(16, 3001, 3), _params(16, seed=9, **{off: None}))


def test_all_parameters_left_out():
    _check(_logits(16, 3001, 4), _params(16, seed=9, temperature=None, top_k=None, top_p=None, min_p=None))


def test_flat_rows():
    """Normal logits: the kept set is most of the vocabulary."""
    x = np.random.default_rng(6).standard_normal((8, 151936)).astype(np.float32)
    _check(x, _params(8, seed=6, top_k=[0, 0, 0, 100000, 50000, 3, 0, 0], min_p=0.0,
                      top_p=[1, 0.9, 0.5, 0.9, 1, 1, 0.999, 0.01]))


@pytest.mark.parametrize("V", [300, 32000, 151936])
def test_sixteen_bit_logits_tie(V):
    """bf16 logits: long runs of equal ones, ordered by index."""
    x = torch.as_tensor(_logits(10, V, V + 1) * 2).to(torch.bfloat16)
    _check(x, _params(10, seed=V + 1, temperature=1.5))


@pytest.mark.parametrize("V", [100, 5000, 30000, 100003])
def test_equal_logits(V):
    """One value everywhere: the order is the index alone, and beyond 16,384
    candidates the row itself is searched."""
    x = np.full((6, V), 3.25, np.float32)
    _check(x, _params(6, top_k=[0, 0, V // 3, V - 1, 0, 70], top_p=[1, 0.77, 0.51, 1, 0.999, 0.31],
                      min_p=0.0, u=[0.0, 0.123456, 0.7654321, 0.999, 0.3, 0.56789]))


def test_few_values():
    """Two and three distinct logits, top-k and top-p cutting inside the runs."""
    rng = np.random.default_rng(0)
    x = rng.choice([0.0, 1.0, 1.5], (9, 60001)).astype(np.float32)
    _check(x, _params(9, top_k=[0, 100, 20001, 40000, 0, 0, 59999, 0, 7], min_p=0.0,
                      top_p=[1, 1, 0.9, 0.8, 0.37, 0.9999, 1, 0.6, 0.5], seed=2))


def test_masks_and_infinities():
    V = 9001
    x = _logits(9, V, 12)
    x[0, :] = -np.inf                        # nothing left
    x[1, :] = -np.inf
    x[1, 777] = -3.0                         # one left
    x[2, ::2] = -np.inf
    x[3, 5:] = np.finfo(np.float32).min      # the type's lowest value is a logit like another
    x[4, :] = np.finfo(np.float32).min
    x[5, ::3] = np.nan
    x[6, :] = np.nan
    x[7, [8, 100, 4000]] = np.inf            # equal infinities share the draw
    x[8, :] = -np.inf
    x[8, V - 1] = np.finfo(np.float32).min
    p = _params(9, temperature=0.9, top_k=0, top_p=0.97, min_p=0.0, seed=3)
    _check(x, p)
    tok, prob = _call(torch.as_tensor(x).cuda(), p)
    assert tok[0] == tok[6] == -1 and prob[0] == prob[6] == 0
    assert tok[1] == 777 and tok[8] == V - 1 and tok[7] in (8, 100, 4000)


def test_extreme_parameters():
    T, V = 16, 6000
    x = _logits(T, V, 13)
    x[3] = x[3, ::-1]
    p = _params(T, seed=4,
                temperature=[0, -1, np.nan, 1e-30, 1e-45, 1e30, np.inf, 1, 1, 1, 1, 1, 1, 1, 1, 100],
                top_k=[0, 0, 0, 0, 0, 0, 0, -4, 2 ** 31 - 1, V, V + 1, 1, 0, 0, 0, 0],
                top_p=[1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, np.nan, 1.5, -2, 0.9],
                min_p=[0, 0, 0, 0, 0, 0, 0, np.nan, -1, 0, 0, 0, 1, 2, 0, 0],
                u=[0.5, 0.5, 0.5, 0.5, 0.5, 0.31, 0.77, 0.2, 0.4, 0.6, 0.8, 0.9, 0.3, 0.9, 0.9, 0.77])
    _check(x, p)


def test_extreme_draws():
    """u = 0 takes the first token, u >= 1 and just below the last kept one,
    u < 0 and NaN the first."""
    V = 2500
    x = np.repeat(_logits(1, V, 14), 6, axis=0)
    u = np.array([0.0, 1.0, 5.0, -1.0, np.nan, 1 - 2.0 ** -24], np.float32)
    p = _params(6, temperature=1.0, top_k=40, top_p=1.0, min_p=0.0, u=u)
    tok, _ = _call(torch.as_tensor(x).cuda(), p)
    order = np.argsort(-x[0].astype(np.float64), kind="stable")
    assert tok[0] == tok[3] == tok[4] == order[0]
    assert tok[1] == tok[2] == tok[5] == order[39]


def test_draws_follow_the_probabilities():
    """With u spread evenly over [0, 1) every token is drawn its share of the
    times, to within one."""
    N, V = 4096, 50
    x = np.repeat(_logits(1, V, 15, fall=0.7), N, axis=0)
    u = ((np.arange(N) + 0.5) / N).astype(np.float32)
    tok, prob = _call(torch.as_tensor(x).cuda(),
                      _params(N, temperature=1.3, top_k=30, top_p=0.95, min_p=0.0, u=u))
    w = np.exp((x[0].astype(np.float64) - x[0].max()) / float(np.float32(1.3)))
    order = np.argsort(-w, kind="stable")[:30]
    cum = np.cumsum(w[order])
    kept = order[:int((cum < float(np.float32(0.95)) * cum[-1]).sum()) + 1]
    share = np.zeros(V)
    share[kept] = w[kept] / w[kept].sum()
    got = np.bincount(tok, minlength=V)
    assert (np.abs(got - N * share) <= 1).all()
    np.testing.assert_allclose(prob, share[tok], rtol=1e-6)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,off", [(1, 0), (3, 1), (0, 2), (5, 3)])
def test_strided_and_unaligned_rows(dtype, pad, off):
    T, V = 7, 4999
    x = torch.as_tensor(_logits(T, V, 16)).to(dtype)
    buf = torch.full((T * (V + pad) + off + 8,), 1e30, dtype=dtype, device="cuda")
    view = buf[off:off + T * (V + pad)].view(T, V + pad)[:, :V]
    view.copy_(x)
    p = _params(T, seed=8)
    tok, prob = _call(view, p)
    want, _ = _expect(x.double().numpy(), p)
    np.testing.assert_array_equal(tok, want)


def test_a_row_does_not_depend_on_its_batch():
    x = _logits(40, 30011, 17)
    p = _params(40, seed=17)
    tok, prob = _call(torch.as_tensor(x).cuda(), p)
    for t in (0, 13, 39):
        one = {k: v[t:t + 1] for k, v in p.items()}
        a, b = _call(torch.as_tensor(x[t:t + 1]).cuda(), one)
        assert a[0] == tok[t] and b[0] == prob[t]


@pytest.mark.parametrize("T", [1, 2, 4, 17, 64])
def test_verify(T):
    V = 32000
    x = _logits(T, V, 18 + T)
    p = _params(T, seed=18)
    want, _ = _expect(x.astype(np.float64), p)
    xs = torch.as_tensor(x).cuda()
    for kept in sorted({0, T // 2, T - 1}):
        draft = want[:T - 1].copy()
        if kept < T - 1:
            draft[kept] = (draft[kept] + 1) % V
        tok, _, n = _call(xs, p, draft=draft, verify=True)
        np.testing.assert_array_equal(tok, want)
        assert n == kept + 1


def test_verify_at_temperature_zero_is_the_greedy_acceptance():
    import oracle
    x = _logits(4, 32000, 30)
    g = x.argmax(axis=1)
    draft = np.array([g[0], g[1], (g[2] + 1) % 32000], np.int32)
    tok, _, n = _call(torch.as_tensor(x).cuda(), _params(4, temperature=0.0, top_k=0, top_p=1, min_p=0),
                      draft=draft, verify=True)
    np.testing.assert_array_equal(tok[:n], oracle.verify_accept(x, draft))


def test_replayed_graph_and_other_stream():
    """One capture, replayed on new logits and numbers, with eager work on
    another workspace between the replays."""
    import routed_expert_ffn_gemv_amd as moe
    T, V = 3, 20000
    logits = torch.zeros((T, V), device="cuda")
    u = torch.zeros(T, device="cuda")
    p = _params(T, seed=21)
    par = {k: torch.as_tensor(v, device="cuda") for k, v in p.items() if k != "u"}
    tok = torch.zeros(T, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_sample_workspace_size(T, V), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_sample(logits, T, V, u, tok, ws, stream=side, **par)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_sample(logits, T, V, u, tok, ws, **par)
    for seed in (40, 41, 42, 43):
        x = _logits(T, V, seed)
        logits.copy_(torch.as_tensor(x))
        p["u"] = np.random.default_rng(seed).random(T, dtype=np.float32)
        u.copy_(torch.as_tensor(p["u"]))
        g.replay()
        torch.cuda.synchronize()
        want, _ = _expect(x.astype(np.float64), p)
        np.testing.assert_array_equal(tok.cpu().numpy(), want)
        _call(logits, p)
