"""moe_rope_append: the same rows give the same bits whether few tokens or many
are appended at once, and 8-bit values are the codes that their definition in
fp32 gives."""

import numpy as np
import pytest
import torch

from oracle import around
from oracle import attention as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _append(cache, x, first, n, Hq, **kw):
    """Rows first .. first + n - 1 of x at positions of the same numbers, into
    a cache of their own; (q, k, v, k_scale, v_scale) of these rows."""
    import routed_expert_ffn_gemv_amd as moe
    Hkv, D, page, f8 = cache["Hkv"], cache["D"], 64, cache["f8"]
    pages = -(-(first + n) // page)
    e = lambda *s, dtype: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    k, v = (e(pages, page, Hkv, D, dtype=torch.uint8 if f8 else BF16) for _ in "kv")
    ks, vs = (e(pages, page, Hkv, dtype=F32) if f8 else None for _ in "kv")
    i32 = lambda a: torch.as_tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = moe.KVBatch(i32([0, n]), i32([first + n]), i32(np.arange(pages)[None]))
    q = e(n, Hq * D, dtype=BF16)
    moe.moe_rope_append(moe.KVCache(k, v, ks, vs), batch, x[first:first + n], n, Hq, q, **kw)
    torch.cuda.synchronize()
    return [q] + [None if t is None else t.flatten(0, 1)[first:] [:n] for t in (k, v, ks, vs)]


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 9, 3), (128, 5, 1), (256, 16, 2)])
@pytest.mark.parametrize("R", [0, 10, 64])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("x_dtype,f8", [(F32, True), (BF16, True), (BF16, False)])
def test_the_same_bits_for_few_tokens_and_many(D, Hq, Hkv, R, interleaved, norm, x_dtype, f8):
    T = 8197
    g = torch.Generator(device="cuda").manual_seed(D + R)
    x = (torch.randn((T, (Hq + 2 * Hkv) * D), device="cuda", generator=g) * 3).to(x_dtype)
    kw = dict(freq=torch.as_tensor(ref.frequencies(R, 1e5)[0], device="cuda") if R else None, interleaved=interleaved,
              rot_scale=1.1386)
    if norm:
        kw["q_weight"], kw["k_weight"] = (1 + 0.3 * torch.randn(D, device="cuda", generator=g) for _ in "qk")
    cache = dict(Hkv=Hkv, D=D, f8=f8)
    many = _append(cache, x, 0, T, Hq, **kw)
    for first, n in ((3000, 1), (700, 37), (5000, 1021), (2, 1024), (1500, 5001)):
        for a, b in zip(_append(cache, x, first, n, Hq, **kw), many):
            if a is not None:
                assert torch.equal(a.view(torch.uint8), b[first:first + n].view(torch.uint8)), (first, n)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("x_dtype", [F32, BF16])
@pytest.mark.parametrize("T", [300, 8193])
def test_codes_of_values(D, x_dtype, T):
    """Values are not computed: scale and codes are what fp32 gives, to the bit."""
    x = torch.randn((T, 3 * D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(D))
    x = (x * torch.logspace(-30, 30, T, device="cuda")[:, None]).to(x_dtype)
    _, _, v, _, scale = _append(dict(Hkv=1, D=D, f8=True), x, 0, T, 1)
    a = x[:, 2 * D:].float().cpu().numpy()
    want = np.maximum(np.abs(a).max(axis=1), np.float32(around.SCALE_FLOOR)) / np.float32(448)
    assert np.array_equal(scale[:, 0].cpu().numpy(), want)
    codes = torch.as_tensor(a / want[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(v[:, 0].cpu(), codes)
