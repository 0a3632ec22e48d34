"""The weights of moe_paged_attention, to more bits than an output shows: values
are ones at places of their own, so that an 8-bit output's fp32 scale is one
weight over the row's sum."""

import math

import numpy as np
import pytest
import torch

from oracle import attention as ref
from paged import Setup
from test_gpu_attention import _run, _wide

# Of a weight 2^x, x > -13: x is rounded at 2^-21 (half a step below 16), the
# factor log2(e) and an 8-bit key's score at 2^-24 of themselves (at most 4.4),
# after ln 2 together 2^-20.5; exp2 is off by 2^-23, the largest weight, which is
# most of the sum, by as much; the waves' maxima differ by less than 8, which adds
# 2^-22 and another exp2 on either side; sum, quotient and scale are fewer than
# eight roundings of 2^-24.  All of it is less than 2^-18.8.
OFF = 2.0 ** -18.5
PARTS = {2: 2.0 ** -16, 3: 2.0 ** -24}     # what bf16 numbers in turn leave of a weight


def _bf16(a):
    return torch.as_tensor(a, dtype=torch.float32).bfloat16().double().numpy()


def _heights(n, D, cache):
    """n distances below the row's maximum, one per position of their own."""
    x = np.random.default_rng(D).uniform(0.3 if cache == "bf16" else 1.5, 3.0, n)
    return _bf16(x) if cache == "bf16" else x.astype(np.float32).astype(np.float64)


def _setup(D, cache, rows, max_pages=None):
    """Position i < D scores -x_i with a query that is one in column i (others
    -12 or less) and has a one in column i of its value; position D scores 0."""
    s = Setup(rows, 1, D, cache, page=16, max_pages=max_pages)
    s.table[:] = s.table[:1]                          # (all texts are one)
    x = _heights(D, D, cache)
    length = rows[0][1]
    scale = torch.rand(length, generator=torch.Generator().manual_seed(5)) * 0.5 + 0.5
    for p in range(length):
        at = s.place(0, p)
        if cache == "bf16":
            s.k[at] = 0.0 if p == D else -12.0
            s.v[at] = 0.0
            if p < D:
                s.k[at][0, p], s.v[at][0, p] = -x[p], 1.0
        else:
            s.k[at] = 0 if p == D else 0xD0           # -8
            s.v[at] = 0
            s.k_scale[at], s.v_scale[at] = (x[p] if p < D else 2.0), float(scale[p])
            if p < D:
                s.k[at][0, p], s.v[at][0, p] = 0xB8, 0x38       # -1, 1
    return s


def _check(s, Hq, parts):
    D, T = s.D, s.T
    q = torch.zeros((T, Hq, D), dtype=torch.bfloat16)
    place = (torch.arange(T * Hq) % D).view(T, Hq)
    q.scatter_(2, place[..., None], 1.0)
    _, _, _, scale = _run(s, Hq, q=q.view(T, -1), scale=1.0, want=("x8",))
    got = scale.double().numpy().reshape(T, Hq, D // 128) * 448
    k, v, seen = s.sequence(0)
    for b in range(len(s.rows)):
        t = np.arange(s.off[b], s.off[b + 1])
        out, _, _, _ = ref.attend(q[t].double().numpy(), k, v, s.positions(b), seen, 1.0)
        # (of each row's blocks the one with its own column)
        block = (place[t] // 128).numpy()[..., None]
        want = np.take_along_axis(out.reshape(len(t), Hq, D // 128, 128).max(axis=3), block, axis=2)
        off = np.abs(np.take_along_axis(got[t], block, axis=2) / want - 1)
        assert off.max() <= OFF + PARTS[parts], (b, off.max(), np.argwhere(off > OFF + PARTS[parts])[:5].tolist())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("cache", ["bf16", "f8"])
@pytest.mark.parametrize("new,Hq", [(1, 16), (1, 5), (2, 16), (4, 8)])
def test_three_parts(D, cache, new, Hq):
    """Up to 32 rows: every position of a step, in tiles of 16 and of 32."""
    n = -(-D // (new * Hq))
    _check(_setup(D, cache, [(new, D + 1 + new)] * n), Hq, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("cache", ["bf16", "f8"])
@pytest.mark.parametrize("height,new,Hq", [(64, 8, 8), (64, 5, 12), (128, 16, 8), (256, 32, 8), (256, 17, 15)])
def test_two_parts(D, cache, height, new, Hq):
    n = -(-D // (new * Hq))
    s = _setup(D, cache, [(new, D + 1 + new)] * n, max_pages=_wide(new * n, Hq, D, height))
    _check(s, Hq, 2)


def _left(w, parts):
    """What `parts` bf16 numbers leave of weights, relative."""
    rest = torch.as_tensor(w, dtype=torch.float32)
    for _ in range(parts):
        rest = rest - rest.bfloat16().float()
    return (rest.double().abs() / torch.as_tensor(w, dtype=torch.float32).double()).numpy()


@pytest.mark.parametrize("D", [128, 256])
def test_a_missing_part_would_show(D):
    """On the host: the weights that these tests take are not those that fewer
    parts hold, whatever power of two (or wave's own maximum) they go by."""
    x = _heights(D, D, "bf16")
    for base in (0.0, 8 / math.log2(math.e)):
        w = np.exp(-x - base)
        assert (_left(w, 2) > 1.5 * (OFF + PARTS[3])).sum() > D // 16
        assert (_left(w, 1) > 20 * (OFF + PARTS[2])).sum() > D // 2
    rng = np.random.default_rng(1)
    x, scale = _heights(D, D, "f8"), rng.uniform(0.5, 1.0, D).astype(np.float32)
    assert (_left(np.exp(-x) * scale, 2) > 1.5 * (OFF + PARTS[3])).sum() > D // 16
    assert (_left(np.exp(-x) * scale, 1) > 20 * (OFF + PARTS[2])).sum() > D // 2


# One position of weight 1, the others of 2^-27.05 (18.75 in natural units): a
# lane's step of eight adds 2^-24.05, less than half a step of fp32 at 1.
SMALL = 18.75
LONG = 65536


def _plain_sum(weights):
    s = np.float32(0)
    for w in weights:
        s = np.float32(s + w)
    return float(s)


def test_a_sum_without_its_roundings_would_show():
    """On the host: the lane that has the large weight loses its share of the
    small ones, 1 of 16 for a row in 16 lanes."""
    w = math.exp(-SMALL)
    steps = [np.float32(1 + 7 * w)] + [np.float32(8 * w)] * (LONG // 128 - 1)
    lost = 1 + 7 * w + (LONG // 128 - 1) * 8 * w - _plain_sum(steps)
    assert lost > 4 * OFF


@pytest.mark.gpu
def test_long_sums():
    """One large weight among 65,536, in tiles that one workgroup walks over
    alone: as many texts as there are workgroups, all in the same pages."""
    D, Hq, B = 128, 16, 512
    s = _one_text(D, B)
    q = torch.zeros((B, Hq, D), dtype=torch.bfloat16)
    q[..., 0] = 1.0
    _, out, _, scale = _run(s, Hq, q=q.view(B, -1), scale=1.0, want=("out", "x8"))
    want = 1 / (1 + (LONG - 1) * math.exp(-SMALL))
    got = scale.double().numpy() * 448
    assert np.abs(got / want - 1).max() <= OFF
    assert bool((out.double().view(B, Hq, D)[..., 0] / want - 1).abs().max() <= 2.0 ** -8)


def _one_text(D, B):
    s = Setup([(1, LONG)], 1, D, page=64, spare=0)
    s.k.zero_()
    s.v.zero_()
    s.k[..., 0] = -SMALL
    first = s.place(0, 0)
    s.k[first][0, 0] = 0.0
    s.v[first][0, 0] = 1.0
    s.rows = [(1, LONG)] * B
    s.off = list(range(B + 1))
    s.T = B
    s.table = s.table.expand(B, -1).contiguous()
    s.kv_len = torch.full((B,), LONG, dtype=torch.int32)
    return s
