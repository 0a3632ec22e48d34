"""Both calls of the attention half at the largest number of sequences."""

import numpy as np
import pytest
import torch

import routed_expert_ffn_gemv_amd as moe

pytestmark = pytest.mark.gpu

B, PAGE, D, Hq = 4096, 16, 64, 2


@pytest.mark.parametrize("longest", [16, 41])
def test_4096_sequences(longest):
    """One new token or none each, appended and attended to: texts of 1 to
    `longest` positions, in pages of their own."""
    per = -(-longest // PAGE)
    length = torch.arange(B) * 7 % longest + 1
    new = (torch.arange(B) % 5 != 2).int()
    off = torch.cat((torch.zeros(1, dtype=torch.int32), new.cumsum(0).int()))
    T = int(off[-1])
    g = torch.Generator().manual_seed(longest)
    k, v = (torch.randn((B * per, PAGE, 1, D), generator=g).bfloat16().cuda() for _ in "kv")
    table = torch.randperm(B * per, generator=g).int().view(B, per)
    x = torch.randn((T, (Hq + 2) * D), generator=g).bfloat16()
    i32 = lambda t: t.int().cuda()  # noqa: E731
    cache, batch = moe.KVCache(k, v), moe.KVBatch(i32(off), i32(length), table.cuda())
    q = torch.zeros((T, Hq * D), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.empty(moe.moe_paged_attention_workspace_size(T, B, Hq, 1, D), dtype=torch.uint8, device="cuda")
    moe.moe_rope_append(cache, batch, x.cuda(), T, Hq, q)
    moe.moe_paged_attention(cache, batch, q, T, Hq, D ** -0.5, ws, out=out)
    torch.cuda.synchronize()
    assert torch.equal(q.cpu(), x[:, :Hq * D])
    rows = torch.arange(B)[new.bool()]
    last = length[rows] - 1
    kk, vv = (t.cpu()[table.long()].view(B, per * PAGE, D)[rows] for t in (k, v))
    assert torch.equal(kk[torch.arange(T), last], x[:, Hq * D:(Hq + 1) * D])
    assert torch.equal(vv[torch.arange(T), last], x[:, (Hq + 1) * D:])
    kk, vv, qq = (t.double().numpy() for t in (kk, vv, x[:, :Hq * D].view(T, Hq, D)))
    s = np.matmul(qq, kk.transpose(0, 2, 1)) * float(np.float32(D ** -0.5))
    s[np.broadcast_to((np.arange(per * PAGE) > last.numpy()[:, None])[:, None], s.shape)] = -np.inf
    w = np.exp(s - s.max(axis=2, keepdims=True))
    w /= w.sum(axis=2, keepdims=True)
    want = np.matmul(w, vv)
    # scores off by 2 (D + 16) 2^-24 of sum |q k| * scale, weights by that and (in three parts) 2^-24, sums by 2^-18
    e = 2 * (D + 16) * 2.0 ** -24 * (np.matmul(np.abs(qq), np.abs(kk).transpose(0, 2, 1)) * D ** -0.5).max(axis=2, keepdims=True)
    level = np.matmul(w, np.abs(vv))
    err = np.abs(out.cpu().double().numpy().reshape(T, Hq, D) - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + (2 * e + 2.0 ** -17) * level).all()
