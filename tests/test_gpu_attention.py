"""GPU parity of moe_paged_attention against its definition in 64 bits.

Tolerances.  A score is a sum of D exact products in fp32, off by less than
(D + 16) 2^-24 times scale * sum |q k|, its exponent's rounding and exp2's
included: a weight is off by that much of itself twice over (its own and the
maximum's).  The weight is then rounded to bf16 (2^-8); with a bf16 cache the
divisor is the sum of the rounded weights, so that an error e of the weights
moves the output by e times the weighted mean of |v - out| at most; with an
8-bit one the divisor is the unrounded sum and 2^-8 counts against the weighted
mean of |v|.  The fp32 sums of the outputs add less than 2^-18 of that mean.  The
output's own rounding: 2^-8 (bf16); e4m3 2^-4 of the value, 2^-10 of the scale where the
code is subnormal."""

import numpy as np
import pytest
import torch

from oracle import around
from oracle import attention as ref
from paged import Setup

pytestmark = pytest.mark.gpu


def _off(f8, D, out, spread, level, mag):
    e = 2 * (D + 16) * 2.0 ** -24 * mag
    return (1.02 * 2.0 ** -8 + e) * (level if f8 else spread) + (e + 2.0 ** -18) * level


def _run(s, Hq, window=0, scale=None, seed=1, sharp=1.5, want=("out",), stream=None, pad=0, off=0, q=None):
    """(q, out, x8, x8_scale) on the host, rows behind the last token's among
    them, which must be as they were."""
    import routed_expert_ffn_gemv_amd as moe
    D, T = s.D, s.T
    g = torch.Generator().manual_seed(seed)
    if q is None:
        q = (torch.randn((T, Hq * D), generator=g) * sharp).bfloat16()
    cache, batch, d = s.device()
    rows = T + 1
    qbuf = torch.full((rows * (Hq * D + pad) + off + 8,), 3.0, dtype=torch.bfloat16, device="cuda")
    qv = qbuf[off:off + rows * (Hq * D + pad)].view(rows, Hq * D + pad)[:, :Hq * D]
    qv[:T].copy_(q)
    obuf = torch.full((rows * (Hq * D + pad) + off + 8,), -7.0, dtype=torch.bfloat16, device="cuda")
    out = obuf[off:off + rows * (Hq * D + pad)].view(rows, Hq * D + pad)[:, :Hq * D]
    x8 = torch.full((rows, Hq * D), 0x55, dtype=torch.uint8, device="cuda")
    sc = torch.full((rows, max(1, Hq * D // 128)), -7.0, device="cuda")
    n = moe.moe_paged_attention_workspace_size(T, len(s.rows), Hq, s.Hkv, D)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    moe.moe_paged_attention(cache, batch, qv, T, Hq, D ** -0.5 if scale is None else scale, ws,
                            out=out if "out" in want else None, x8=x8 if "x8" in want else None,
                            x8_scale=sc if "x8" in want else None, window=window, stream=stream)
    torch.cuda.synchronize()
    o, c, w = out.cpu(), x8.cpu(), sc.cpu()
    rest = np.ones(rows, bool)
    rest[s.off[0]:s.off[-1]] = False
    assert (o[rest] == -7).all() and (c[rest] == 0x55).all() and (w[rest] == -7).all()
    if "out" not in want:
        assert (o == -7).all()
    if "x8" not in want:
        assert (c == 0x55).all() and (w == -7).all()
    gap = torch.ones(obuf.numel(), dtype=torch.bool)
    gap[off:off + rows * (Hq * D + pad)].view(rows, Hq * D + pad)[:, :Hq * D] = False
    assert (obuf.cpu()[gap] == -7).all()
    return q, o[:T], c[:T], w[:T]


def _check(s, Hq, window=0, scale=None, rows=None, want=("out",), **kw):
    """rows: how many tokens of a sequence are compared (spread over it)."""
    q, out, x8, x8_scale = _run(s, Hq, window, scale, want=want, **kw)
    D = s.D
    sc = float(np.float32(D ** -0.5 if scale is None else scale))
    worst = 0.0
    for b, (new, _) in enumerate(s.rows):
        if not new:
            continue
        pick = np.arange(new) if rows is None or new <= rows else np.unique(
            np.linspace(0, new - 1, rows).astype(int))
        k, v, seen = s.sequence(b)
        t = s.off[b] + pick
        qb = q[t].double().numpy().reshape(len(pick), Hq, D)
        o, *scales = ref.attend(qb, k, v, s.positions(b)[pick], seen, sc, window)
        off = _off(s.f8, D, o, *scales)
        if "out" in want:
            got = out[t].double().numpy().reshape(o.shape)
            err = np.abs(got - o) - 2.0 ** -8 * np.abs(o) - 1.01 * off
            assert (err <= 1e-30).all(), f"sequence {b}: {err.max()} too far at {np.argwhere(err > 1e-30)[:4].tolist()}"
            worst = max(worst, float((np.abs(got - o) / (np.abs(o) + off + 1e-30)).max()))
        if "x8" in want:
            blocks = o.reshape(len(pick), -1, 128)
            boff = off.reshape(blocks.shape)
            amax = np.abs(blocks).max(axis=2)
            got_scale = x8_scale[t].double().numpy()
            assert (np.abs(got_scale - np.maximum(amax, around.SCALE_FLOOR) / 448)
                    <= boff.max(axis=2) / 448 + 2.0 ** -22 * amax / 448).all()
            got = around.E4M3[x8[t].numpy()].reshape(blocks.shape) * got_scale[:, :, None]
            assert (np.abs(got - blocks) <= 2.0 ** -4 * (np.abs(blocks) + boff) + 2.0 ** -10 * got_scale[:, :, None]
                    + boff).all()
    return worst


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cache", ["bf16", "f8"])
@pytest.mark.parametrize("length", [1, 2, 31, 32, 33, 127, 128, 129, 300])
def test_one_token(D, cache, length):
    _check(Setup([(1, length)], 2, D, cache), 6)


def _wide(T, Hq, D, height, page=16):
    """Pages of a table so wide that tiles get `height` rows (they are at most
    64, 128 or 256 tall below 2.5e9, below 5e9 and from 5e9 products of the
    step on, which the host counts by the table's width)."""
    return int({64: 0, 128: 3.5e9, 256: 6e9}[height] / (T * Hq * D * page)) + 40


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cache", ["bf16", "f8"])
@pytest.mark.parametrize("new,height", [(2, 64), (9, 64), (17, 64), (40, 64), (33, 128), (40, 256), (70, 256)])
@pytest.mark.parametrize("before", [0, 1, 77])
def test_chunks(D, cache, new, height, before):
    """All tile heights (16 to 256 rows), with and without a past."""
    _check(Setup([(new, before + new)], 2, D, cache, max_pages=_wide(new, 8, D, height)), 8, rows=24)


@pytest.mark.parametrize("D,cache", [(64, "bf16"), (128, "f8"), (256, "bf16"), (256, "f8")])
@pytest.mark.parametrize("height", [64, 128, 256])
def test_tall_tiles(D, cache, height):
    """Several tiles per sequence, cut and whole, ragged, windows, 8-bit
    outputs, pages that are not there, at every height."""
    want = ("out", "x8") if D > 64 else ("out",)
    rows = [(150, 700), (0, 3), (97, 97), (1, 400)]
    T, Hq = 248, 12
    s = Setup(rows, 2, D, cache, page=8, max_pages=_wide(T, Hq, D, height, 8))
    _check(s, Hq, want=want, rows=5)
    _check(s, Hq, want=want, rows=5, window=70)
    s.table[0, 30:41] = -1
    _check(s, Hq, want=want, rows=5)
    # few rows that one sequence brings to a long text: every tile is cut
    _check(Setup([(33, 3001)], 1, D, cache, page=32, max_pages=_wide(33, 8, D, height, 32)), 8, rows=3)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 5), (6, 2), (7, 1), (33, 1), (48, 1), (100, 1), (200, 1)])
@pytest.mark.parametrize("cache", ["bf16", "f8"])
def test_head_groups(Hq, Hkv, cache):
    _check(Setup([(3, 50), (1, 7)], Hkv, 64, cache), Hq)


@pytest.mark.parametrize("layout", ["slots", "heads", "both"])
@pytest.mark.parametrize("page", [1, 2, 8, 16, 64, 256])
@pytest.mark.parametrize("cache", ["bf16", "f8"])
def test_layouts(layout, page, cache):
    _check(Setup([(1, 150), (5, 40)], 2, 64, cache, page, layout), 4)


@pytest.mark.parametrize("D,want", [(128, ("x8",)), (128, ("out", "x8")), (256, ("x8",)), (256, ("out", "x8"))])
@pytest.mark.parametrize("new", [1, 5, 70])
def test_outputs_in_8_bits(D, want, new):
    _check(Setup([(new, 200 + new), (1, 3)], 2, D), 4, want=want, rows=12)
    _check(Setup([(new, 90 + new)], 1, D, "f8"), 5, want=want, rows=12)


@pytest.mark.parametrize("window", [1, 2, 31, 64, 100, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("new", [1, 3, 40, 200])
def test_windows(window, new):
    for cache, D in (("bf16", 64), ("f8", 128)):
        _check(Setup([(new, 300 + new), (min(new, 9), 40)], 2, D, cache), 4, window=window, rows=12)


@pytest.mark.parametrize("cache", ["bf16", "f8"])
def test_long_texts_are_cut(cache):
    """One sequence over all workgroups, for one token, a verify pass and a
    chunk; more pages than a workgroup holds numbers of."""
    _check(Setup([(1, 20011)], 1, 128, cache, 16), 4)
    _check(Setup([(4, 9001)], 2, 256, cache, 1), 16, rows=2)
    _check(Setup([(130, 7001)], 1, 64, cache, 2), 4, rows=4)


def test_more_pages_than_one_workgroup_holds_numbers_of():
    """Runs of several spans of page numbers: many sequences, pages of one
    and of two positions."""
    _check(Setup([(1, 2500 + 3 * b) for b in range(150)], 4, 64, "f8", 1), 4, sharp=1.0)
    _check(Setup([(40, 2500 + 3 * b) for b in range(10)], 8, 64, "f8", 2), 32, rows=2)


def test_ragged_batch():
    rows = [(1, 1 + (97 * b) % 700) for b in range(70)]
    _check(Setup(rows, 2, 64, page=32), 6)
    rows = [(0, 55), (3, 3), (0, 0), (1, 300), (20, 61), (0, 9), (2, 129)]
    _check(Setup(rows, 2, 128, "f8", first=2, behind=3), 6)


def test_more_sequences_than_threads():
    _check(Setup([(b % 2, 3 + b % 50) for b in range(700)], 1, 64, behind=1), 2)


def test_mixed_batch():
    """One sequence brings a chunk, the others one token each."""
    rows = [(1, 40 + 11 * b) for b in range(9)]
    rows[4] = (333, 700)
    _check(Setup(rows, 2, 64), 6, rows=9)
    _check(Setup(rows, 2, 256, "f8"), 16, rows=5, want=("x8",))


def test_rows_that_see_nothing():
    """More new tokens than positions, no positions, pages that are not
    there: zeros, and the other rows as if nothing were missing."""
    for cache in ("bf16", "f8"):
        for D in (64, 256):
            s = Setup([(5, 3), (4, 0), (2, 40), (1, 16), (3, 30)], 2, D, cache, page=8, max_pages=5)
            s.table[2, 1:3] = torch.tensor([-1, s.pages], dtype=torch.int32)
            s.table[3] = -5
            s.table[4, 3] = 2 ** 31 - 1
            s.table[4, 0] = -2 ** 31
            want = ("out", "x8") if D == 256 else ("out",)
            _check(s, 4, want=want)
            q, out, x8, sc = _run(s, 4, want=want)
            none = [0, 1, 5, 6, 7, 8, 11]
            assert (out[none] == 0).all()
            if D == 256:
                assert (x8[none] & 127 == 0).all() and (sc[none] == 2.0 ** -126).all()
            _check(s, 4, window=9)
            for window in (2 ** 30 - 1, 2 ** 30, 2 ** 31 - 1):       # (and positions below zero)
                _check(s, 4, window=window)
    # rows before and behind the text's start in one wave
    s = Setup([(40, 25), (16, 9)], 2, 64)
    for window in (0, 3, 2 ** 31 - 1):
        _check(s, 4, window=window)


def test_positions_behind_the_table():
    s = Setup([(3, 100), (1, 64)], 2, 64, page=16, max_pages=4)
    _check(s, 4)


@pytest.mark.parametrize("cache", ["bf16", "f8"])
def test_what_lies_elsewhere_has_no_effect(cache):
    """NaN and infinities in later slots of the last page and in other pages."""
    for new, length in ((1, 37), (3, 130), (70, 90)):
        s = Setup([(new, length)], 2, 128, cache, page=32, spare=3)
        q, want, _, _ = _run(s, 6)
        used = torch.zeros((s.pages, s.page), dtype=torch.bool)
        for p in range(length):
            used[s.place(0, p)] = True
        for t in (s.k, s.v):
            t[~used] = 0x7F if cache == "f8" else float("nan")
        if cache == "f8":
            for t in (s.k_scale, s.v_scale):
                t[~used] = float("inf")
        else:
            s.v[~used] = float("inf")
        _, got, _, _ = _run(s, 6, q=q)
        assert torch.equal(got, want)


def test_scores_of_any_size():
    """Flat rows, one position far above all others, a maximum that rises with
    every step, and one that falls."""
    s = Setup([(2, 400)], 1, 64)
    _check(s, 2, scale=1e-6)
    _check(s, 2, scale=30.0)
    s = Setup([(2, 700)], 1, 64, page=16)
    q = torch.zeros((2, 128), dtype=torch.bfloat16)
    q[:, ::64] = 16.0
    for sign in (1, -1):
        for p in range(700):
            s.k[s.place(0, p)] = 0
            s.k[s.place(0, p)][:, 0] = sign * p * 0.25
        _check(s, 2, q=q, scale=1.0)
        _check(s, 2, q=q, scale=0.01)
    s.k.zero_()
    _check(s, 2, q=q)


def test_large_values():
    s = Setup([(2, 90)], 2, 64)
    s.v *= 2.0 ** 100
    _check(s, 4)
    s.v *= 2.0 ** -200
    _check(s, 4)


@pytest.mark.parametrize("pad,off", [(8, 0), (5, 1), (0, 3)])
def test_strides_and_alignment(pad, off):
    _check(Setup([(5, 60), (1, 200)], 2, 128), 6, pad=pad, off=off)


def test_same_bits_again():
    s = Setup([(1, 5000), (1, 20), (30, 900)], 2, 128)
    _, a, _, _ = _run(s, 8)
    for _ in range(3):
        assert torch.equal(_run(s, 8)[1], a)


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 elements whose last pages are used, alone
    and among first ones."""
    import routed_expert_ffn_gemv_amd as moe
    D, Hkv, page = 256, 8, 256
    pages = 2 ** 32 // (page * Hkv * D) + 9
    small = Setup([(1, 600), (3, 300)], Hkv, D, page=page)
    k = torch.empty((pages, page, Hkv, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    table = small.table.clone()
    for i in range(small.pages):
        at = pages - 1 - i if i % 2 == 0 else i
        k[at].copy_(small.k[i])
        v[at].copy_(small.v[i])
        table[small.table == i] = at
    q = torch.randn((4, 16 * D), generator=torch.Generator().manual_seed(2)).bfloat16()
    _, want, _, _ = _run(small, 16, q=q)
    d = lambda t: t.to("cuda")  # noqa: E731
    batch = moe.KVBatch(d(torch.tensor(small.off, dtype=torch.int32)), d(small.kv_len), d(table))
    out = torch.zeros((4, 16 * D), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_paged_attention_workspace_size(4, 2, 16, Hkv, D), dtype=torch.uint8, device="cuda")
    moe.moe_paged_attention(moe.KVCache(k, v), batch, d(q), 4, 16, D ** -0.5, ws, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want)


def test_two_streams_and_a_replayed_graph():
    """Two calls at once with workspaces of their own; one graph replayed on
    other lengths, tables and queries, eager calls in between."""
    import routed_expert_ffn_gemv_amd as moe
    a = Setup([(1, 4000), (2, 33)], 2, 128, seed=1)
    b = Setup([(2, 100), (1, 3000)], 2, 128, seed=2, max_pages=a.max_pages)
    sets = []
    for s in (a, b):
        cache, batch, d = s.device()
        q = torch.randn((3, 8 * 128), generator=torch.Generator().manual_seed(s.rows[0][1])).bfloat16().cuda()
        n = moe.moe_paged_attention_workspace_size(3, 2, 8, 2, 128)
        sets.append((cache, batch, d, q, torch.empty(n, dtype=torch.uint8, device="cuda"),
                     torch.zeros_like(q), torch.cuda.Stream()))
    call = lambda st, out, ws, stream=None, batch=None: moe.moe_paged_attention(  # noqa: E731
        st[0], batch or st[1], st[3], 3, 8, 0.09, ws, out=out, stream=stream)
    want = []
    for st in sets:
        o = torch.zeros_like(st[3])
        call(st, o, st[4])
        torch.cuda.synchronize()
        want.append(o)
    for _ in range(10):
        for st in sets:
            call(st, st[5], st[4], st[6])
    torch.cuda.synchronize()
    for st, w in zip(sets, want):
        assert torch.equal(st[5], w)
    # the graph reads a's cache; its batch takes turns
    st = sets[0]
    q_off, kv_len, table = (st[2][n].clone() for n in ("q_off", "kv_len", "table"))
    batch = moe.KVBatch(q_off, kv_len, table)
    out = torch.zeros_like(st[3])
    call(st, out, st[4], batch=batch)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(st, out, st[4], batch=batch)
    for i in range(5):
        st[3].copy_(torch.randn(st[3].shape, generator=torch.Generator().manual_seed(i)).bfloat16())
        other = sets[i % 2][2]
        q_off.copy_(other["q_off"])
        kv_len.copy_(other["kv_len"])
        table.copy_(other["table"].clamp(max=a.pages - 1))
        graph.replay()
        o = torch.zeros_like(out)
        call(st, o, sets[1][4], batch=batch)
        torch.cuda.synchronize()
        assert torch.equal(o, out) and bool((o != 0).any())
