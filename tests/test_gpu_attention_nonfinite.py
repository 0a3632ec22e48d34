"""moe_paged_attention with NaN and infinities in queries and keys that are
seen: a row's result is what the formula gives, however its tile is cut, and
the rows beside it keep their bits."""

import numpy as np
import pytest
import torch

from paged import Setup
from test_gpu_attention import _run, _wide

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def _tall(height, rows, Hkv, D, cache, Hq):
    T = sum(n for n, _ in rows)
    need = max(-(-length // 8) for _, length in rows)
    return Setup(rows, Hkv, D, cache, page=8, max_pages=max(need, _wide(T, Hq, D, height, 8)))


def _cases():
    """(setup, query heads): tiles of 16 to 256 rows, whole and cut."""
    yield "16 whole", Setup([(1, 40), (1, 9)], 2, 128), 6
    yield "16 cut", Setup([(1, 20011)], 1, 128), 4
    yield "16 cut f8", Setup([(1, 9000)], 2, 256, "f8"), 8
    yield "32 cut", Setup([(4, 9001)], 1, 64), 7
    yield "64 cut", _tall(64, [(40, 3000)], 1, 128, "bf16", 8), 8
    yield "128 cut", _tall(128, [(40, 3000)], 1, 128, "f8", 8), 8
    yield "256 cut", _tall(256, [(70, 2000)], 1, 256, "bf16", 8), 8
    yield "256 whole", _tall(256, [(70, 90)], 2, 64, "bf16", 8), 8


CASES = {name: (s, Hq) for name, s, Hq in _cases()}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_a_query_that_is_not_finite(name, bad):
    """NaN in every column of its own head's row, the others untouched."""
    s, Hq = CASES[name]
    want = ("out", "x8") if s.D > 64 else ("out",)
    q, out, x8, scale = _run(s, Hq, want=want)
    t, h = s.T // 2, Hq - 2
    worse = q.clone()
    worse[t, h * s.D + 5] = bad
    _, got, got8, got_scale = _run(s, Hq, want=want, q=worse)
    cols = slice(h * s.D, (h + 1) * s.D)
    assert bool(torch.isnan(got[t, cols]).all())
    got[t, cols] = out[t, cols]
    assert torch.equal(got, out)
    if "x8" in want:
        blocks = slice(h * s.D // 128, (h + 1) * s.D // 128)
        assert bool((got8[t, cols] & 127 == 127).all()) and bool((got_scale[t, blocks] == 2.0 ** -126).all())
        got8[t, cols], got_scale[t, blocks] = x8[t, cols], scale[t, blocks]
        assert torch.equal(got8, x8) and torch.equal(got_scale, scale)


def _formula(q, k, v, pos, scale):
    """One row [D] over keys and values [L][D] in 64 bits, NaN and infinities
    as the formula's own operations give them."""
    with np.errstate(all="ignore"):
        s = (k[:pos + 1] * q).sum(axis=1) * scale
        w = np.exp(s - s.max())
        return (w[:, None] * v[:pos + 1]).sum(axis=0) / w.sum()


@pytest.mark.parametrize("new,length,height", [(1, 1, 64), (1, 50, 64), (1, 9000, 64), (3, 700, 64), (50, 300, 64),
                                               (50, 300, 128), (50, 300, 256)])
@pytest.mark.parametrize("value", [-INF, INF, NAN])
def test_keys_that_are_not_finite(new, length, height, value):
    """A score of -infinity weighs nothing, a row of no other (or with one of
    +infinity or NaN) is NaN."""
    D, Hq = 64, 8
    s = Setup([(new, length)], 1, D, page=8, max_pages=max(_wide(new, Hq, D, height, 8), -(-length // 8)))
    s.k[s.place(0, length // 2)][:, 0] = value
    q = torch.randn((new, Hq, D), generator=torch.Generator().manual_seed(3)).bfloat16()
    q[..., 0] = torch.where(torch.arange(Hq) % 2 == 0, 1.0, -1.0)       # (either sign of an infinite score)
    _, out, _, _ = _run(s, Hq, q=q.view(new, -1))
    got = out.double().numpy().reshape(new, Hq, D)
    k, v, _ = s.sequence(0)
    some = set()
    for t in sorted({0, new // 2, new - 1}):
        for h in range(Hq):
            want = _formula(q[t, h].double().numpy(), k[:, 0], v[:, 0], length - new + t, D ** -0.5)
            assert np.array_equal(np.isnan(got[t, h]), np.isnan(want)), (t, h)
            some.add(bool(np.isnan(want).any()))
            if not np.isnan(want).any():
                # weights off by less than 1.1 * 2^-8, the output by 2^-8 more
                assert (np.abs(got[t, h] - want) <= 2.2 * 2.0 ** -8 * np.abs(v).max()).all()
    assert some == ({True} if value != value or length == 1 else {True, False})


@pytest.mark.parametrize("name", ["16 whole", "16 cut", "64 cut", "256 cut"])
def test_scores_of_minus_infinity_alone(name):
    """No finite score: NaN, as 0 / 0 is; a later finite one takes it all."""
    s, Hq = CASES[name]
    s = Setup(s.rows, s.Hkv, s.D, "bf16", s.page, max_pages=s.max_pages)
    q, _, _, _ = _run(s, Hq)
    q.view(s.T, Hq, s.D)[..., 0] = 1.0
    s.k[..., 0] = -INF
    _, out, _, _ = _run(s, Hq, q=q)
    assert bool(torch.isnan(out).all())
    for b in range(len(s.rows)):
        last = int(s.positions(b)[0])
        s.k[s.place(b, last)][:, 0] = 0.0
    _, out, _, _ = _run(s, Hq, q=q)
    for b in range(len(s.rows)):
        page, slot = s.place(b, int(s.positions(b)[0]))
        want = s.v[page, slot].repeat_interleave(Hq // s.Hkv, dim=0).reshape(1, -1)
        rows = out[s.off[b]:s.off[b + 1]].float()
        # (one weight: its own rounding to bf16 cancels in the quotient but for 2^-16)
        assert bool(((rows - want.float()).abs() <= 2.0 ** -8 * want.float().abs()).all())


@pytest.mark.parametrize("cache", ["bf16", "f8"])
def test_rows_that_see_nothing_stay_zeros(cache):
    """Whatever their queries hold."""
    s = Setup([(5, 3), (1, 30), (2, 0)], 2, 64, cache, page=8)
    s.table[1] = -1
    q = torch.full((8, 4 * 64), NAN, dtype=torch.bfloat16)
    _, out, _, _ = _run(s, 4, q=q)
    none = [0, 1, 5, 6, 7]
    assert bool((out[none] == 0).all()) and bool(torch.isnan(out[2:5]).all())
