"""moe_add_rmsnorm beyond 2^31 elements, bit for bit against the definition's
fp32 steps on the CPU."""

import pytest
import torch

from test_gpu_norm import EPS, _cpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pad", [0, 3])
def test_more_elements_than_31_bits_count(pad):
    import routed_expert_ffn_gemv_amd as moe
    if torch.cuda.mem_get_info()[0] < 32 << 30:
        pytest.skip("32 GiB of GPU memory wanted")
    T, H = 2 ** 21 + 3, 1032                  # element 2^31 is in row 2,080,895 (2,074,863 with the pad)
    g = torch.Generator(device="cuda")
    g.manual_seed(pad)
    resid = torch.empty((T, H + pad), dtype=torch.bfloat16, device="cuda")
    resid.normal_(generator=g)
    y = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    y.normal_(generator=g)
    weight = (1 + 0.1 * torch.randn(H, device="cuda", generator=g)).float()
    rows = [0, 1, 2 ** 20, 2 ** 31 // (H + pad) - 1, 2 ** 31 // (H + pad), 2 ** 31 // H, 2 ** 31 // H + 1, T - 2, T - 1]
    v, n, x_want, x8_want, s_want = _cpu(y[rows].cpu(), resid[rows, :H].cpu(), weight.cpu())
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x8 = torch.zeros((T, H), dtype=torch.uint8, device="cuda")
    scale = torch.zeros((T, (H + 127) // 128), device="cuda")
    beside = resid[:, H:].clone()
    moe.moe_add_rmsnorm(T, H, y, resid[:, :H], weight, EPS, resid_out=resid[:, :H], x=x, x8=x8, x8_scale=scale)
    torch.cuda.synchronize()
    assert torch.equal(resid[rows, :H].cpu(), v)
    assert torch.equal(x[rows].cpu(), x_want)
    assert torch.equal(x8[rows].cpu(), x8_want.view(torch.uint8))
    assert torch.equal(scale[rows].cpu(), s_want)
    assert torch.equal(resid[:, H:], beside)
    assert bool((scale > 0).all())            # every row was written
