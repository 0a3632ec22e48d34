"""Outputs of the attention half that share memory with what the call still
reads: refused before any HIP call, and views beside each other are not."""

import pytest
import torch

import routed_expert_ffn_gemv_amd as moe
from oracle import attention as ref
from paged import Setup
from test_attention import FAKE, INVALID, _append, _attend

W = 4 * 128 * 2     # bytes of a row of queries


@pytest.mark.parametrize("kw", [
    dict(out=FAKE), dict(out=FAKE + 2), dict(out=FAKE + 5 * W - 2), dict(out=FAKE - 5 * W + 2),
    dict(qs=1024, os=1024, out=FAKE + 1022), dict(qs=1024, os=1024, out=FAKE - 2), dict(qs=2000, os=1024, out=FAKE + 3000),
    dict(T=1, out=FAKE + W - 2), dict(qs=1024, os=1024, out=FAKE + 3 * 2048 + 2), dict(qs=600, os=520, out=FAKE + 4 * 1200),
    dict(qs=1024, os=1024, out=FAKE + 4 * 2048 + W - 2), dict(qs=1024, os=1024, out=FAKE - 4 * 2048 - W + 2),
    dict(out=None, x8=FAKE, sc=3 * FAKE), dict(out=None, x8=FAKE + 5 * W - 1, sc=3 * FAKE),
    dict(out=None, x8=3 * FAKE, sc=FAKE + 4), dict(out=None, x8=3 * FAKE, sc=FAKE - 5 * 16 + 4),
])
def test_outputs_within_the_queries(kw):
    a = dict(out=2 * FAKE, x8=None, sc=None)
    a.update(kw)
    assert _attend(**a) == INVALID


PLACES = [(0, 512, 5 * 512, 512), (5 * 512, 512, 0, 512), (0, 1024, 512, 1024), (512, 1024, 0, 1024),
          (0, 1024, 5 * 1024, 1024), (0, 1024, 3 * 1024 + 512, 1024), (0, 1024, 4 * 1024 + 512, 1024),
          (4 * 1024 + 512, 1024, 0, 1024), (0, 10000, 512, 512), (0, 10000, 10512, 700), (600, 5000, 1200, 520)]


@pytest.mark.gpu
@pytest.mark.parametrize("q_at,q_stride,at,stride,x8", [(*p, False) for p in PLACES] + [
    (*p, True) for p in PLACES if p[1] == 10000 or p[3] == 512])        # (8-bit outputs are contiguous)
def test_outputs_beside_the_queries(q_at, q_stride, at, stride, x8):
    """In one allocation, before, behind and between the queries' rows."""
    T, Hq, D = 5, 4, 128
    s = Setup([(3, 200), (2, 9)], 2, D)
    cache, batch, _ = s.device()
    buf = torch.zeros(60000, dtype=torch.bfloat16, device="cuda")
    rows = lambda a, n: buf[a:a + T * n].as_strided((T, Hq * D), (n, 1))  # noqa: E731
    q, out = rows(q_at, q_stride), rows(at, stride)
    if x8 and q_stride == 10000:
        out = buf[at:at + T * 256].view(torch.uint8).view(T, Hq * D)
    elif x8:
        out = buf[at:at + T * 512].view(torch.uint8)[:T * 512].view(T, Hq * D)
    q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(1)))
    want = q.clone()
    ws = torch.empty(moe.moe_paged_attention_workspace_size(T, 2, Hq, 2, D), dtype=torch.uint8, device="cuda")
    scale = [torch.zeros((T, Hq), device="cuda") for _ in "ab"]
    apart = torch.zeros((T, Hq * D), dtype=out.dtype, device="cuda")
    for o, sc in ((apart, scale[0]), (out, scale[1])):
        kw = dict(x8=o, x8_scale=sc) if x8 else dict(out=o)
        moe.moe_paged_attention(cache, batch, q, T, Hq, 0.1, ws, **kw)
    torch.cuda.synchronize()
    assert torch.equal(apart, out) and torch.equal(*scale) and bool((apart != 0).any())
    assert torch.equal(q, want)
    with pytest.raises(moe.MoEError):
        moe.moe_paged_attention(cache, batch, q, T, Hq, 0.1, ws, out=q)


ROW = 8 * 128           # elements of a row of queries, keys and values


@pytest.mark.parametrize("kw", [
    dict(q=FAKE + 2, qs=ROW), dict(q=FAKE + W, qs=ROW), dict(q=FAKE + 2 * ROW - 2, qs=ROW + 8), dict(q=FAKE + 2),
    dict(q=FAKE - 2, qs=ROW), dict(q=FAKE + 4 * 2 * ROW, qs=ROW), dict(q=FAKE + 5 * 2 * ROW - 2), dict(q=FAKE - 4 * 2 * ROW, qs=ROW),
    dict(fmt=moe.MOE_W_F32, q=FAKE + 4, qs=2 * ROW), dict(fmt=moe.MOE_W_F32, q=FAKE + 5 * 4 * ROW - 2), dict(T=1, q=FAKE + 2 * ROW - 2),
])
def test_queries_within_other_parts_of_the_rows(kw):
    assert _append(**kw) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
def test_queries_beside_the_rows(x_dtype):
    """Queries in the gap behind each row of one allocation, as elsewhere."""
    T, Hq, Hkv, D, R = 7, 3, 2, 64, 32
    s = Setup([(T, 20)], Hkv, D)
    wide = (2 if x_dtype == torch.float32 else 1) * (Hq + 2 * Hkv) * D      # in bf16 columns
    buf = torch.zeros((T, wide + Hq * D), dtype=torch.bfloat16, device="cuda")
    x = buf.view(x_dtype)[:, :(Hq + 2 * Hkv) * D]
    x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(1)))
    freq = torch.as_tensor(ref.frequencies(R, 1e4)[0], device="cuda")
    got = []
    for q in (torch.zeros((T, Hq * D), dtype=torch.bfloat16, device="cuda"), buf[:, wide:]):
        cache, batch, d = s.device()
        moe.moe_rope_append(cache, batch, x, T, Hq, q, freq=freq)
        torch.cuda.synchronize()
        got.append((q.clone(), d["k"], d["v"]))
    for a, b in zip(*got):
        assert torch.equal(a, b)
