"""moe_rope_append with NaN and infinities: columns from R on stay as they are,
whatever else their lane holds; NaN stays in its head's row (or its pair)."""

import pytest
import torch

from oracle import around
from oracle import attention as ref
from paged import Setup

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def _run(s, x, Hq, R, interleaved, weight=None):
    """(q, keys, values, key scales, value scales) of every token, on the host."""
    import routed_expert_ffn_gemv_amd as moe
    cache, batch, d = s.device()
    q = torch.zeros((s.T, Hq * s.D), dtype=torch.bfloat16, device="cuda")
    freq = torch.as_tensor(ref.frequencies(R, 100.0)[0], device="cuda")
    w = None if weight is None else weight.cuda()
    moe.moe_rope_append(cache, batch, x.cuda(), s.T, Hq, q, freq=freq, interleaved=interleaved, q_weight=w, k_weight=w)
    torch.cuda.synchronize()
    at = [s.place(0, int(p)) for p in s.positions(0)]
    rows = [torch.stack([d[n][p].cpu() for p in at]) if d[n] is not None else None
            for n in ("k", "v", "k_scale", "v_scale")]
    return q.cpu().view(s.T, Hq, s.D), *rows


def _same(a, b):
    assert torch.equal(torch.isnan(a), torch.isnan(b))
    assert torch.equal(torch.nan_to_num(a.float(), nan=0.0), torch.nan_to_num(b.float(), nan=0.0))


@pytest.mark.parametrize("D,R", [(64, 2), (64, 10), (64, 50), (128, 20), (256, 102)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new", [3, 8200])
def test_columns_behind_the_rotated_ones_stay(D, R, interleaved, x_dtype, new):
    Hq, Hkv = 2, 1
    s = Setup([(new, new + 5)], Hkv, D, page=64)
    x = torch.randn((new, Hq + 2 * Hkv, D), generator=torch.Generator().manual_seed(R)).to(x_dtype)
    for t, h, c, v in ((0, 0, R, INF), (0, 1, R + 1, -INF), (1, 0, R + 3, NAN), (1, 2, R, INF), (2, 2, R + 1, NAN),
                       (new - 1, 1, D - 1, INF)):
        x[t, h, c] = v
    clean = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    rows = torch.arange(new) if new < 100 else torch.tensor([0, 1, 2, 3, new - 1])
    want = _run(s, clean.view(new, -1), Hq, R, interleaved)
    got = _run(s, x.view(new, -1), Hq, R, interleaved)
    for g, w, part in ((got[0], want[0], x[:, :Hq]), (got[1], want[1], x[:, Hq:Hq + Hkv])):
        assert torch.equal(g[rows][..., :R], w[rows][..., :R])
        _same(g[rows][..., R:], part[rows][..., R:].bfloat16())


@pytest.mark.parametrize("interleaved", [False, True])
def test_nan_behind_the_rotated_columns_in_8_bits(interleaved):
    """A NaN code in its own column, left out of the row's maximum."""
    D, R, Hq = 128, 10, 1
    s = Setup([(4, 9)], 1, D, "f8")
    x = torch.randn((4, 3, D), generator=torch.Generator().manual_seed(7))
    x[1, 1, 11] = x[2, 2, 5] = NAN
    clean = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    want = _run(s, clean.view(4, -1), Hq, R, interleaved)
    got = _run(s, x.view(4, -1), Hq, R, interleaved)
    for i in (3, 4):
        assert torch.equal(got[i], want[i])
    for i, (t, c) in ((1, (1, 11)), (2, (2, 5))):
        codes, w = got[i].clone(), want[i]
        assert int(codes[t, 0, c]) & 127 == 127
        codes[t, 0, c] = w[t, 0, c]
        assert torch.equal(codes, w)


@pytest.mark.parametrize("cache", ["bf16", "f8"])
@pytest.mark.parametrize("new", [4, 8200])
def test_rows_beside_stay(cache, new):
    """A NaN (or an infinity) makes NaN of its own head's row where there is a
    norm, and leaves every other row as it is."""
    D, Hq, Hkv, R = 64, 3, 2, 32
    s = Setup([(new, new)], Hkv, D, cache, page=64)
    x = torch.randn((new, Hq + 2 * Hkv, D), generator=torch.Generator().manual_seed(1))
    w = torch.rand(D) + 0.5
    want = _run(s, x.view(new, -1), Hq, R, False, w)
    bad = x.clone()
    bad[1, 1, 40] = NAN
    bad[2, Hq + 1, 3] = NAN
    got = _run(s, bad.view(new, -1), Hq, R, False, w)
    assert bool(torch.isnan(got[0][1, 1]).all())
    got[0][1, 1] = want[0][1, 1]
    k = got[1] if cache == "bf16" else torch.as_tensor(around.E4M3[got[1].numpy()])
    assert bool(torch.isnan(k[2, 1]).all())
    got[1][2, 1] = want[1][2, 1]
    if cache == "f8":
        assert float(got[3][2, 1]) == 2.0 ** -126
        got[3][2, 1] = want[3][2, 1]
    for g, v in zip(got, want):
        assert (g is None and v is None) or torch.equal(g, v)
