"""GPU parity of moe_rope_append against its definition in 64 bits.

Tolerances.  The norm: up to 13 additions of squares, a mean, a root, a
division and two products in fp32, together less than 2^-20 of a value.
The rotation: a turn's fp32 rest is off by 2^-25 turns (2^-22 radians), sine
and cosine by 2 units of 2^-24, their products and sum by 2^-23 more: with
the norm's share less than 2^-19 times (|a1| + |a2|) * max(rot_scale, 1).
Then bf16's half step (2^-8) or, in 8 bits, e4m3's (2^-4 of the value, 2^-10
of the scale where the code is subnormal)."""

import numpy as np
import pytest
import torch

from oracle import around
from oracle import attention as ref
from paged import Setup

pytestmark = pytest.mark.gpu

EPS = 1e-5
OFF = 2.0 ** -19


def _want(s, qkv, Hq, freq, rot_scale, interleaved, qw, kw):
    """Per row of a sequence: (t, b, pos, q, k, v and their error scales)."""
    D, Hkv = s.D, s.Hkv
    x = qkv.double().numpy()
    for b in range(len(s.rows)):
        pos = s.positions(b)
        for i, p in enumerate(pos):
            t = s.off[b] + i
            heads = x[t].reshape(Hq + 2 * Hkv, D)
            q = ref.head_norm(heads[:Hq], qw, EPS)
            k = ref.head_norm(heads[Hq:Hq + Hkv], kw, EPS)
            (q, qm), (k, km) = (ref.rotate(a, np.full(len(a), p), freq, rot_scale, interleaved) for a in (q, k))
            yield t, b, int(p), (q, qm), (k, km), heads[Hq + Hkv:]


def _in_8_bits(codes, scale, value, mag):
    """codes [Hkv][D] with scales [Hkv] against values off by OFF * mag."""
    off = OFF * mag
    amax = np.abs(value).max(axis=1)
    want = np.maximum(amax, around.SCALE_FLOOR) / 448
    assert (np.abs(scale - want) <= off.max(axis=1) / 448 + 2.0 ** -23 * want).all()
    got = around.E4M3[codes] * scale[:, None]
    assert (np.abs(got - value) <= 2.0 ** -4 * (np.abs(value) + off) + 2.0 ** -10 * scale[:, None] + off).all()


def _check(s, Hq, R, interleaved=False, norm=True, x_dtype=torch.bfloat16, w_dtype=torch.bfloat16, theta=1e4,
           rot_scale=1.0, seed=1, in_place=False, stream=None, pad=0, off=0):
    import routed_expert_ffn_gemv_amd as moe
    g = torch.Generator().manual_seed(seed)
    D, Hkv, T = s.D, s.Hkv, s.T
    width = (Hq + 2 * Hkv) * D
    qkv = (torch.randn((T, width), generator=g) * 2).to(x_dtype)
    qw = kw = None
    if norm:
        qw, kw = ((1 + 0.3 * torch.randn(D, generator=g)).to(w_dtype) for _ in "qk")
    freq, _ = ref.frequencies(R, theta)
    cache, batch, d = s.device()
    buf = torch.full((T * (width + pad) + off + 8,), 3.0, dtype=x_dtype, device="cuda")
    x = buf[off:off + T * (width + pad)].view(T, width + pad)[:, :width]
    x.copy_(qkv)
    if in_place:
        q = x[:, :Hq * D]
    else:
        qbuf = torch.full((T * (Hq * D + pad) + off + 8,), -7.0, dtype=torch.bfloat16, device="cuda")
        q = qbuf[off:off + T * (Hq * D + pad)].view(T, Hq * D + pad)[:, :Hq * D]
    before = q.cpu().clone()
    moe.moe_rope_append(cache, batch, x, T, Hq, q, freq=torch.as_tensor(freq, device="cuda") if R else None,
                        rot_scale=rot_scale, interleaved=interleaved, q_weight=None if qw is None else qw.cuda(),
                        k_weight=None if kw is None else kw.cuda(), eps=EPS, stream=stream)
    torch.cuda.synchronize()
    host = {n: d[n].cpu().contiguous() for n in ("k", "v", "k_scale", "v_scale") if d[n] is not None}
    left = {n: getattr(s, n).clone() for n in host}     # what must be as it was
    got_q = q.cpu()
    rest = np.ones(T, bool)
    e = float(np.float32(EPS))
    assert abs(e - EPS) < 1e-12
    w64 = [None if w is None else w.double().numpy() for w in (qw, kw)]
    for t, b, p, (qr, qm), (kr, km), vr in _want(s, qkv, Hq, freq, rot_scale, interleaved, *w64):
        rest[t] = False
        gq = got_q[t].double().numpy().reshape(Hq, D)
        assert (np.abs(gq - qr) <= 2.0 ** -8 * np.abs(qr) + 1.01 * OFF * qm).all(), (t, b, p)
        where = s.place(b, p)
        if where is None:
            continue
        for n, value, mag in (("k", kr, km), ("v", vr, np.zeros_like(vr))):
            got = host[n][where]
            if s.f8:
                _in_8_bits(got.numpy(), host[n + "_scale"][where].double().numpy(), value, mag)
                host[n + "_scale"][where] = left[n + "_scale"][where]
            else:
                gv = got.double().numpy()
                assert (np.abs(gv - value) <= 2.0 ** -8 * np.abs(value) + 1.01 * OFF * mag).all(), (n, t, b, p)
                if n == "v":
                    assert torch.equal(got.reshape(-1), torch.as_tensor(value).to(x_dtype).bfloat16().reshape(-1))
            host[n][where] = left[n][where]
    for n in host:
        assert torch.equal(host[n], left[n]), f"{n}: written outside the new positions"
    assert torch.equal(got_q[rest], before[rest])
    if pad and not in_place:
        gap = torch.ones(qbuf.numel(), dtype=torch.bool)
        gap[off:off + T * (Hq * D + pad)].view(T, Hq * D + pad)[:, :Hq * D] = False
        assert (qbuf.cpu()[gap] == -7).all()
    return got_q


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("R", [0, 2, 10, 50, 64])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotations(D, R, interleaved):
    _check(Setup([(3, 9), (1, 40)], 2, D), 3, R, interleaved)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cache", ["bf16", "f8"])
@pytest.mark.parametrize("norm", [False, True])
def test_formats(D, x_dtype, cache, norm):
    _check(Setup([(5, 21), (2, 2)], 3, D, cache), 4, D, norm=norm, x_dtype=x_dtype,
           w_dtype=torch.float32 if D == 64 else torch.bfloat16, rot_scale=1.25)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (16, 2), (7, 7), (33, 1)])
@pytest.mark.parametrize("cache", ["bf16", "f8"])
def test_heads(Hq, Hkv, cache):
    _check(Setup([(2, 30)], Hkv, 128, cache), Hq, 32)


@pytest.mark.parametrize("layout", ["slots", "heads", "both"])
@pytest.mark.parametrize("page", [1, 2, 16, 128])
@pytest.mark.parametrize("cache", ["bf16", "f8"])
def test_layouts(layout, page, cache):
    _check(Setup([(4, 19), (0, 5), (1, 1), (6, 6)], 2, 64, cache, page, layout), 2, 64)


def test_many_sequences_and_rows_of_none():
    """More sequences than one round of the search takes, empty ones among
    them, rows before the first and behind the last sequence."""
    rows = [(b % 3, 5 + b % 40) for b in range(300)]
    _check(Setup(rows, 1, 64, first=3, behind=5), 2, 16)


def test_one_token_in_many_sequences():
    _check(Setup([(1, 1 + (7 * b) % 90) for b in range(130)], 2, 128, "f8", 32), 4, 64)


def test_more_than_a_thousand_tokens():
    """A workgroup per token, which walks over all of its rows."""
    _check(Setup([(1100, 1500), (13, 13)], 2, 64, page=32), 9, 50, True)


@pytest.mark.parametrize("D,Hq,interleaved,x_dtype,cache", [
    (64, 1, False, torch.float32, "bf16"), (128, 5, True, torch.bfloat16, "f8"), (256, 14, False, torch.bfloat16, "bf16")])
def test_four_tokens_per_workgroup(D, Hq, interleaved, x_dtype, cache):
    """More than 8192 rows: sequences that end inside a workgroup's four, rows
    of none, positions that are not there, rows in several rounds."""
    rows = [(8001, 8050), (0, 7), (3, 2), (170, 200), (1, 1), (19, 40)]
    _check(Setup(rows, 2, D, cache, page=32, first=2, behind=3), Hq, D // 2, interleaved, x_dtype=x_dtype)


def test_positions_that_are_not_there():
    """Pages out of range, positions behind the table and before the start:
    keys and values dropped, queries written."""
    s = Setup([(6, 30), (4, 40), (5, 3)], 2, 64, page=8, max_pages=4)
    s.table[0, 3] = -1
    s.table[1, 2] = s.pages
    s.table[1, 3] = 2 ** 31 - 1
    _check(s, 2, 64)


@pytest.mark.parametrize("pos", [100_000, 16_777_217, 2 ** 30 - 5])
def test_far_positions(pos):
    s = Setup([(3, 1)], 1, 64, page=2 ** 16, spare=1, max_pages=2 ** 14)
    s.kv_len[0] = pos + 3
    s.rows = [(3, pos + 3)]
    s.table[0, pos >> 16] = 1
    s.table[0, (pos + 2) >> 16] = 1
    _check(s, 2, 64, theta=10.0)


@pytest.mark.parametrize("pad,off", [(0, 0), (8, 0), (5, 1), (0, 3)])
@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
def test_strides_and_alignment(pad, off, x_dtype):
    _check(Setup([(5, 21)], 2, 128), 3, 128, x_dtype=x_dtype, pad=pad, off=off)


@pytest.mark.parametrize("D", [64, 256])
def test_in_place(D):
    a = _check(Setup([(5, 21), (2, 2)], 2, D), 9, 32, in_place=True, pad=8)
    b = _check(Setup([(5, 21), (2, 2)], 2, D), 9, 32)
    assert torch.equal(a, b)


def test_zeros_and_subnormals():
    """Rows of zeros (scale at its floor) and values near the smallest."""
    import routed_expert_ffn_gemv_amd as moe
    s = Setup([(2, 2)], 1, 64, "f8")
    cache, batch, d = s.device()
    x = torch.zeros((2, 3 * 64), device="cuda")
    x[1] = 1e-40
    q = torch.ones((2, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    moe.moe_rope_append(cache, batch, x, 2, 1, q, q_weight=w, k_weight=w, eps=0.0 + 1e-6)
    torch.cuda.synchronize()
    assert (q[0] == 0).all()
    p = s.place(0, 0)
    assert (d["k"][p] == 0).all() and (d["v"][p] == 0).all()
    assert float(d["k_scale"][p][0]) == float(d["v_scale"][p][0]) == 2.0 ** -126


def test_other_stream_and_replayed_graph():
    """Captured once, replayed on other rows, lengths, tables and offsets."""
    import routed_expert_ffn_gemv_amd as moe
    s = Setup([(3, 20), (1, 9)], 2, 128, "f8")
    t = Setup([(1, 35), (3, 7)], 2, 128, "f8", seed=5, max_pages=s.max_pages + 1)
    s = Setup([(3, 20), (1, 9)], 2, 128, "f8", max_pages=t.max_pages, spare=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _check(s, 4, 64, stream=side)
    cache, batch, d = s.device()
    g = torch.Generator().manual_seed(3)
    freq = torch.as_tensor(ref.frequencies(64, 1e4)[0], device="cuda")
    x = torch.zeros((4, 8 * 128), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((4, 4 * 128), dtype=torch.bfloat16, device="cuda")
    call = lambda c, b, out: moe.moe_rope_append(c, b, x, 4, 4, out, freq=freq)  # noqa: E731
    call(cache, batch, q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(cache, batch, q)
    for i in range(4):
        x.copy_(torch.randn(x.shape, generator=g).bfloat16())
        other = (s, t)[i % 2]
        d["q_off"].copy_(torch.tensor(other.off, dtype=torch.int32))
        d["kv_len"].copy_(other.kv_len)
        d["table"].copy_(other.table.clamp(max=s.pages - 1))
        state = {n: d[n].clone() for n in ("k", "v", "k_scale", "v_scale")}
        graph.replay()
        q2 = torch.zeros_like(q)
        c2 = moe.KVCache(state["k"], state["v"], state["k_scale"], state["v_scale"])
        call(c2, batch, q2)
        torch.cuda.synchronize()
        assert torch.equal(q, q2) and bool((q != 0).any())
        for n in state:
            assert torch.equal(state[n], d[n]), n
