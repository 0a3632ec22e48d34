"""moe_add_rmsnorm with NaN and infinities: they stay in their rows (also where
rows share a wave), and reach the product that reads the codes."""

import numpy as np
import pytest
import torch

from test_gpu_norm import EPS, _cpu, _inputs, _run

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("H", [96, 256, 272, 1000, 2048])
@pytest.mark.parametrize("r_dtype", [F32, BF16])
def test_rows_beside_stay(H, r_dtype):
    y, r, w = _inputs(9, H, F32, r_dtype, F32, H)
    clean = _run(y, r, w)
    y[2, 5] = float("nan")
    r[4, H - 1] = float("inf")
    y[7, :] = float("-inf")
    got = _run(y, r, w)
    v, n, x, _, _ = _cpu(y, r, w)
    kept = [0, 1, 3, 5, 6, 8]
    for k in clean:
        assert torch.equal(got[k][kept].view(torch.uint8), clean[k][kept].view(torch.uint8)), k
    assert torch.equal(torch.isnan(got["x"]), torch.isnan(x))
    assert torch.equal(torch.isnan(got["resid"]), torch.isnan(v))
    codes = got["x8"] & 127
    assert torch.equal(codes == 127, torch.isnan(n))                # a NaN column is a NaN code
    assert bool((codes[4, :H - 1] == 0).all()) and bool((got["x"][4, :H - 1] == 0).all())


def test_nan_reaches_the_product():
    import routed_expert_ffn_gemv_amd as moe
    T, H, N = 5, 256, 300
    y, r, w = (t.cuda() for t in _inputs(T, H, F32, F32, F32, 1))
    r[3, 100] = float("nan")
    x8 = torch.zeros((T, H), dtype=torch.uint8, device="cuda")
    xs = torch.zeros((T, 2), device="cuda")
    moe.moe_add_rmsnorm(T, H, y, r, w, EPS, x8=x8, x8_scale=xs)
    w8 = torch.as_tensor(np.random.default_rng(0).integers(0, 120, (N, H), dtype=np.uint8), device="cuda")
    for dtype in (F32, BF16):
        out = torch.zeros((T, N), dtype=dtype, device="cuda")
        moe.moe_scaled_linear(x8, xs, T, w8, torch.ones((3, 2), device="cuda"), N, H, out)
        torch.cuda.synchronize()
        assert torch.isnan(out).any(dim=1).tolist() == [False, False, False, True, False]
        assert bool(torch.isnan(out[3]).all())
