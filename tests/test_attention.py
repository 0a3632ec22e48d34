"""The attention half of a layer on the host: refused arguments (before any
HIP call, so no GPU is needed), frequencies and the references' own pins."""

import ctypes
import math

import numpy as np
import pytest
import torch

import routed_expert_ffn_gemv_amd as moe
from oracle import attention as ref

FAKE = 1 << 20      # an aligned non-null address; never dereferenced here
F32, BF16, E4M3 = moe.MOE_W_F32, moe.MOE_W_BF16, moe.MOE_W_E4M3
OK, INVALID, UNSUPPORTED, WORKSPACE = (moe.MOE_OK, moe.MOE_ERR_INVALID, moe.MOE_ERR_UNSUPPORTED,
                                       moe.MOE_ERR_WORKSPACE)


def _cache(**kw):
    a = dict(num_pages=10, page_size=16, Hkv=2, D=128, fmt=BF16, k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE,
             page_stride=16 * 2 * 128, slot_stride=2 * 128, head_stride=128)
    a.update(kw)
    return moe.moe_kv_cache(*a.values())


def _batch(**kw):
    a = dict(B=3, max_pages=8, q_off=FAKE, kv_len=FAKE, page_table=FAKE, table_stride=8)
    a.update(kw)
    return moe.moe_kv_batch(*a.values())


def _append(cache=None, batch=None, **kw):
    a = dict(qkv=FAKE, fmt=BF16, stride=8 * 128, T=5, Hq=4, freq=FAKE, R=64, inter=0, rs=1.0, qw=FAKE, kw=FAKE,
             wf=BF16, eps=1e-6, q=2 * FAKE, qs=4 * 128)
    a.update(kw)
    cache = _cache() if cache is None else cache
    batch = _batch() if batch is None else batch
    return moe.lib.moe_rope_append(ctypes.byref(cache), ctypes.byref(batch), *a.values(), None)


CACHE_REFUSALS = [
    (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(Hkv=0), INVALID), (dict(D=0), INVALID),
    (dict(fmt=F32), UNSUPPORTED), (dict(fmt=2), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
    (dict(page_size=24), UNSUPPORTED), (dict(Hkv=257), UNSUPPORTED), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(k=FAKE + 8), INVALID), (dict(v=FAKE + 8), INVALID),
    (dict(fmt=E4M3, k_scale=None), INVALID), (dict(fmt=E4M3, v_scale=None), INVALID),
    (dict(fmt=E4M3, k_scale=FAKE + 2), INVALID), (dict(fmt=E4M3, v_scale=FAKE + 1), INVALID),
    (dict(page_stride=127), INVALID), (dict(slot_stride=132), INVALID), (dict(head_stride=0), INVALID),
    (dict(head_stride=-128), INVALID), (dict(page_stride=(1 << 30) + 128), UNSUPPORTED), (dict(fmt=E4M3, head_stride=136), INVALID),
]
BATCH_REFUSALS = [
    (dict(B=0), INVALID), (dict(B=4097), UNSUPPORTED), (dict(max_pages=0), INVALID), (dict(table_stride=7), INVALID),
    (dict(max_pages=(1 << 26) + 1, table_stride=1 << 30), UNSUPPORTED), (dict(q_off=None), INVALID),
    (dict(kv_len=None), INVALID), (dict(page_table=None), INVALID), (dict(q_off=FAKE + 2), INVALID),
    (dict(kv_len=FAKE + 2), INVALID), (dict(page_table=FAKE + 2), INVALID),
]


def _attend(cache=None, batch=None, **kw):
    a = dict(q=FAKE, qs=4 * 128, T=5, Hq=4, scale=0.1, window=0, out=FAKE, os=4 * 128, x8=FAKE, sc=FAKE, ws=FAKE,
             size=1 << 30)
    a.update(kw)
    cache = _cache() if cache is None else cache
    batch = _batch() if batch is None else batch
    return moe.lib.moe_paged_attention(ctypes.byref(cache), ctypes.byref(batch), *a.values(), None)


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS)
def test_cache_refusals(kw, status):
    assert _append(cache=_cache(**kw)) == status
    assert _attend(cache=_cache(**kw)) == status


@pytest.mark.parametrize("kw,status", BATCH_REFUSALS)
def test_batch_refusals(kw, status):
    assert _append(batch=_batch(**kw)) == status
    assert _attend(batch=_batch(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), OK), (dict(T=-1), INVALID), (dict(T=(1 << 22) + 1), UNSUPPORTED), (dict(Hq=0), INVALID),
    (dict(Hq=5), INVALID), (dict(Hq=1026), UNSUPPORTED), (dict(Hq=516), UNSUPPORTED), (dict(q=None), INVALID),
    (dict(q=FAKE + 1), INVALID), (dict(qs=511), INVALID), (dict(out=None, x8=None, sc=None), INVALID),
    (dict(x8=None), INVALID), (dict(sc=None), INVALID), (dict(out=FAKE + 1), INVALID), (dict(os=511), INVALID),
    (dict(sc=FAKE + 2), INVALID), (dict(scale=0.0), INVALID), (dict(scale=1e-30), INVALID), (dict(scale=1e30), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(window=-1), INVALID),
    (dict(ws=None), INVALID), (dict(ws=FAKE + 64), INVALID), (dict(size=1000), WORKSPACE),
])
def test_attend_refusals(kw, status):
    assert _attend(**kw) == status


def test_attend_in_8_bits_wants_whole_blocks():
    cache = _cache(D=64, page_stride=16 * 2 * 64, slot_stride=128, head_stride=64)
    assert _attend(cache=cache) == UNSUPPORTED
    assert _attend(cache=cache, T=0, x8=None, sc=None) == OK


def test_attend_workspace_size():
    n = ctypes.c_size_t(0)
    size = moe.lib.moe_paged_attention_workspace_size
    assert size(1, 1, 16, 2, 256, None) == INVALID
    assert size(-1, 1, 16, 2, 256, ctypes.byref(n)) == INVALID
    assert size(1, 0, 16, 2, 256, ctypes.byref(n)) == INVALID
    assert size(1, 1, 15, 2, 256, ctypes.byref(n)) == INVALID
    for bad in ((1, 4097, 16, 2, 256), (1, 1, 16, 2, 96), (1, 1, 514, 2, 64), (1 << 23, 1, 16, 2, 64)):
        assert size(*bad, ctypes.byref(n)) == UNSUPPORTED
    for Hq, Hkv, D in ((16, 2, 256), (7, 7, 64), (256, 1, 128)):
        last = 0
        for T in (0, 1, 2, 5, 17, 100, 5000, 1 << 22):
            a = moe.moe_paged_attention_workspace_size(T, 1, Hq, Hkv, D)
            assert a >= last and a % 256 == 0 and a == moe.moe_paged_attention_workspace_size(T, 64, Hq, Hkv, D)
            last = a
    a = moe.moe_paged_attention_workspace_size(5, 3, 4, 2, 128)
    assert _attend(size=a - 1) == WORKSPACE


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), OK), (dict(T=-1), INVALID), (dict(T=(1 << 22) + 1), UNSUPPORTED), (dict(Hq=0), INVALID),
    (dict(Hq=1025), UNSUPPORTED), (dict(fmt=E4M3), UNSUPPORTED), (dict(wf=E4M3), UNSUPPORTED),
    (dict(R=-2), INVALID), (dict(R=63), INVALID), (dict(R=130), INVALID), (dict(freq=None), INVALID),
    (dict(freq=FAKE + 4), INVALID), (dict(qkv=None), INVALID), (dict(q=None), INVALID), (dict(q=FAKE + 1), INVALID),
    (dict(qkv=FAKE + 1), INVALID), (dict(fmt=F32, qkv=FAKE + 2), INVALID), (dict(stride=8 * 128 - 1), INVALID),
    (dict(qs=4 * 128 - 1), INVALID), (dict(qw=FAKE + 1), INVALID), (dict(wf=F32, kw=FAKE + 2), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(rs=float("inf")), INVALID),
    (dict(q=FAKE), INVALID), (dict(q=FAKE, qs=8 * 128, fmt=F32), INVALID),     # in place: stride and format
])
def test_append_refusals(kw, status):
    assert _append(**kw) == status


def test_null_cache_and_batch():
    args = (FAKE, BF16, 1024, 5, 4, FAKE, 64, 0, 1.0, None, None, BF16, 1e-6, 2 * FAKE, 512, None)
    assert moe.lib.moe_rope_append(None, ctypes.byref(_batch()), *args) == INVALID
    assert moe.lib.moe_rope_append(ctypes.byref(_cache()), None, *args) == INVALID


def test_binding_refusals():
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    c8, sc = torch.zeros((4, 16, 2, 64), dtype=torch.uint8), torch.zeros((4, 16, 2))
    n32 = torch.zeros(4, dtype=torch.int32)
    for bad in (
        lambda: moe.KVCache(k, k),                                           # not on a GPU
        lambda: moe.KVCache(k[0], k[0]),
        lambda: moe.KVCache(k, k[:3]),
        lambda: moe.KVCache(k, k.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)),
        lambda: moe.KVCache(k.float(), k.float()),
        lambda: moe.KVCache(k, c8),
        lambda: moe.KVCache(k.transpose(2, 3), k.transpose(2, 3)),
        lambda: moe.KVCache(c8, c8),                                         # scales wanted
        lambda: moe.KVCache(k, k, sc, sc),
        lambda: moe.KVCache(c8, c8, sc, sc[:3]),
        lambda: moe.KVCache(c8, c8, sc.double(), sc),
        lambda: moe.KVBatch(n32, n32[:3], n32.view(2, 2)),
        lambda: moe.KVBatch(n32, n32, n32.view(4, 1)),
        lambda: moe.KVBatch(n32.long(), n32[:3], torch.zeros((3, 5), dtype=torch.int32)),
        lambda: moe.KVBatch(n32, n32[:3], torch.zeros((3, 5))),
        lambda: moe.KVBatch(n32, n32[:3], torch.zeros((5, 3), dtype=torch.int32).t()),
        lambda: moe.KVBatch(n32, n32[:3], torch.zeros((3, 5), dtype=torch.int32)),   # not on a GPU
    ):
        with pytest.raises(ValueError):
            bad()


class _Anywhere:
    """Stands for a KVCache and a KVBatch, on no GPU."""
    D, Hkv, device, ref = 64, 2, 0, None


def test_call_binding_refusals():
    c = b = _Anywhere()
    x, q = torch.zeros((5, 8 * 64), dtype=torch.bfloat16), torch.zeros((5, 4 * 64), dtype=torch.bfloat16)
    w, freq, ws = torch.ones(64), torch.ones(16, dtype=torch.float64), torch.zeros(64, dtype=torch.uint8)
    append, attend = moe.moe_rope_append, moe.moe_paged_attention
    for bad in (
        lambda: append(c, b, x, 5, 4, q),                                    # not on a GPU
        lambda: append(c, b, x.double(), 5, 4, q),
        lambda: append(c, b, x, 6, 4, q),
        lambda: append(c, b, x, 5, 5, q),
        lambda: append(c, b, x, 5, 4, q.float()),
        lambda: append(c, b, x, 5, 4, q[:, :255]),
        lambda: append(c, b, x, 5, 4, q, freq=freq.float()),
        lambda: append(c, b, x, 5, 4, q, q_weight=w[:63]),
        lambda: append(c, b, x, 5, 4, q, q_weight=w, k_weight=w.bfloat16()),
        lambda: attend(c, b, q, 5, 4, 0.1, ws, out=q),                       # not on a GPU
        lambda: attend(c, b, q.float(), 5, 4, 0.1, ws, out=q),
        lambda: attend(c, b, q, 6, 4, 0.1, ws, out=q),
        lambda: attend(c, b, q, 5, 4, 0.1, ws, out=q.float()),
        lambda: attend(c, b, q, 5, 4, 0.1, ws, out=q[:4]),
        lambda: attend(c, b, q, 5, 4, 0.1, ws.float(), out=q),
        lambda: attend(c, b, q, 5, 4, 0.1, ws, x8=q, x8_scale=torch.zeros((5, 2))),
        lambda: attend(c, b, q, 5, 4, 0.1, ws, x8=torch.zeros((5, 256), dtype=torch.uint8),
                       x8_scale=torch.zeros((5, 1))),
    ):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("kw", [
    dict(R=64, theta=1e4), dict(R=2, theta=1e6), dict(R=256, theta=5e5, scaling="linear", factor=8.0),
    dict(R=64, theta=1e4, scaling="base", factor=4.0), dict(R=128, theta=1e6, scaling="bands", factor=4.0, context=32768),
    dict(R=64, theta=1e4, scaling="bands", factor=40.0, context=4096, fast=32.0, slow=1.0),
    dict(R=4, theta=1e4, scaling="bands", factor=2.0, context=10, fast=3.0, slow=2.9),
])
def test_frequencies(kw):
    freq, rs = moe.moe_rope_frequencies(**kw)
    want, want_rs = ref.frequencies(**kw)
    # pow, log and the mixture round a few times each: 2^-52 per rounding, exponents up to ln(theta)
    np.testing.assert_allclose(freq.numpy(), want, rtol=1e-14)
    assert abs(rs - want_rs) <= 2.0 ** -24 * want_rs


def test_frequencies_ends_of_the_bands():
    """Pairs that turn often keep their frequency, slow ones are divided."""
    freq, rs = moe.moe_rope_frequencies(128, 1e4, "bands", 8.0, 4096)
    plain, one = moe.moe_rope_frequencies(128, 1e4)
    assert one == 1.0 and rs == pytest.approx(0.1 * math.log(8) + 1)
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(freq[turns > 40], plain[turns > 40])
    np.testing.assert_allclose(freq[turns < 0.8].numpy(), plain[turns < 0.8].numpy() / 8, rtol=1e-15)
    assert (freq <= plain).all() and (freq >= plain / 8 * (1 - 1e-15)).all()


@pytest.mark.parametrize("kw,status", [
    (dict(R=0), INVALID), (dict(R=7), INVALID), (dict(R=258), UNSUPPORTED), (dict(theta=1.0), INVALID),
    (dict(theta=float("nan")), INVALID), (dict(theta=float("inf")), INVALID),
    (dict(scaling="linear", factor=0.5), INVALID), (dict(scaling="linear", factor=float("nan")), INVALID),
    (dict(scaling="base", R=2, factor=2.0), INVALID), (dict(scaling="bands", factor=2.0, context=0), INVALID),
    (dict(scaling="bands", factor=2.0, context=100, fast=1.0, slow=1.0), INVALID),
    (dict(scaling="bands", factor=2.0, context=100, slow=0.0), INVALID),
])
def test_frequency_refusals(kw, status):
    a = dict(R=64, theta=1e4)
    a.update(kw)
    with pytest.raises(moe.MoEError) as err:
        moe.moe_rope_frequencies(**a)
    assert err.value.status == status


def test_frequency_refusals_of_pointers_and_kinds():
    buf = (ctypes.c_double * 32)()
    f = moe.lib.moe_rope_frequencies
    assert f(64, 1e4, 0, 1.0, 0, 32.0, 1.0, None, None) == INVALID
    assert f(64, 1e4, 4, 1.0, 0, 32.0, 1.0, buf, None) == UNSUPPORTED
    assert f(64, 1e4, -1, 1.0, 0, 32.0, 1.0, buf, None) == UNSUPPORTED
    assert f(64, 1e4, 0, 0.0, 0, 0.0, 0.0, buf, None) == OK and buf[0] == 1.0
    with pytest.raises(ValueError):
        moe.moe_rope_frequencies(64, 1e4, "other")


def test_rotation_by_hand():
    """A quarter turn per position swaps a pair's columns."""
    f = np.array([math.pi / 2, 0.0])
    a = np.array([[1.0, 2.0, 3.0, 4.0, 5.0]])
    np.testing.assert_allclose(ref.rotate(a, [1], f, 1.0, False)[0], [[-3, 2, 1, 4, 5]], atol=1e-15)
    np.testing.assert_allclose(ref.rotate(a, [1], f, 2.0, True)[0], [[-4, 2, 6, 8, 5]], atol=1e-15)
    np.testing.assert_allclose(ref.rotate(a, [4], f, 1.0, False)[0], a, atol=1e-14)


def test_scores_of_rotated_heads_depend_on_the_distance():
    rng = np.random.default_rng(1)
    f, _ = ref.frequencies(16, 1e4)
    q, k = rng.standard_normal((2, 1, 16))
    for inter in (False, True):
        s = [float((ref.rotate(q, [p + 7], f, 1.0, inter)[0] * ref.rotate(k, [p], f, 1.0, inter)[0]).sum())
             for p in (0, 5, 1000)]
        np.testing.assert_allclose(s, s[0], rtol=1e-9)


def test_attend_by_hand():
    """Equal scores average the values seen; no position: zeros."""
    q, k = np.zeros((2, 2, 4)), np.ones((3, 1, 4))
    v = np.arange(3.0)[:, None, None] * np.ones((3, 1, 4))
    seen = np.array([True, True, True])
    out, spread, level, _ = ref.attend(q, k, v, [1, 2], seen, 1.0)
    np.testing.assert_allclose(out[:, 0, 0], [0.5, 1.0])
    np.testing.assert_allclose(spread[:, 1, 0], [0.5, 2 / 3])
    np.testing.assert_allclose(level[:, 1, 0], [0.5, 1.0])
    assert ref.attend(q, k, v, [1, 2], seen, 1.0, window=1)[0][:, 0, 0].tolist() == [1.0, 2.0]
    assert (ref.attend(q, k, v, [1, 2], ~seen, 1.0)[0] == 0).all()
    assert ref.attend(q, k, v, [-1, 0], seen, 1.0)[0][:, 0, 0].tolist() == [0.0, 0.0]
    q[0, 0] = [np.log(2), 0, 0, 0]
    k[1] = 0
    out, _, _, mag = ref.attend(q, k, v, [1, 2], seen, 1.0)
    assert out[0, 0, 0] == pytest.approx(1 / 3) and mag[0, 0, 0] == pytest.approx(np.log(2))
