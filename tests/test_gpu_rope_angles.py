"""The rotation of moe_rope_append to more bits than its outputs show: of a key
that is one in a pair's first column and zero elsewhere, an 8-bit cache's fp32
scale is the larger of cosine and sine over 448."""

import numpy as np
import pytest
import torch

import routed_expert_ffn_gemv_amd as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("freq", [1.0, 0.31830988618, 1e-3])
@pytest.mark.parametrize("first", [0, 100_000, 2 ** 30 - 9000])
@pytest.mark.parametrize("T", [700, 8200])
@pytest.mark.parametrize("interleaved", [False, True])
def test_cosines_and_sines(freq, first, T, interleaved):
    D, page = 64, 2 ** 16
    shape = (2, page, 1, D)
    k, v = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in "kv")
    ks, vs = (torch.zeros(shape[:3], device="cuda") for _ in "kv")
    table = torch.full((1, 2 ** 14), -1, dtype=torch.int32, device="cuda")
    pages = sorted({first // page, (first + T - 1) // page})
    for i, p in enumerate(pages):
        table[0, p] = i
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.zeros((T, 3, D), device="cuda")
    x[:, 1, 0] = 1.0
    q = torch.zeros((T, D), dtype=torch.bfloat16, device="cuda")
    f = torch.tensor([freq], dtype=torch.float64)
    moe.moe_rope_append(moe.KVCache(k, v, ks, vs), moe.KVBatch(i32([0, T]), i32([first + T]), table), x.view(T, 3 * D),
                        T, 1, q, freq=f.cuda(), rot_scale=1.25, interleaved=interleaved)
    torch.cuda.synchronize()
    pos = np.arange(first, first + T)
    scale = ks[:, :, 0].double().cpu().numpy()
    got = np.array([scale[pages.index(p // page), p % page] for p in pos]) * 448
    angle = pos * freq
    want = 1.25 * np.maximum(np.abs(np.cos(angle)), np.abs(np.sin(angle)))
    # the factor times cosine or sine rounded once, the scale rounded once, and of the angle 2^-51 (its product with
    # the frequency and with 1 / (2 pi) in 64 bits, here and there)
    assert (np.abs(got / want - 1) <= 1.001 * 2.0 ** -23 + 2.0 ** -51 * np.abs(angle)).all()
