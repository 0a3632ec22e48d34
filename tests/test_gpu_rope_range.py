"""moe_rope_append normalises rows of any size."""

import numpy as np
import pytest
import torch

from oracle import attention as ref
from paged import Setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("new", [6, 8200])
def test_rows_of_any_size_are_normalised(eps, new):
    """Rows whose squares leave fp32's range at either end; bounds as for other
    rows: 2^-19 of the pair's magnitude and bf16's half step."""
    import routed_expert_ffn_gemv_amd as moe
    D, R = 128, 32
    s = Setup([(new, new)], 1, D, page=64)
    g = torch.Generator().manual_seed(4)
    size = torch.tensor([1e37, 1e20, 1e-18, 1e-25, 1e-36, 1.0])[torch.arange(new) % 6]
    x = torch.randn((new, 3 * D), generator=g) * size[:, None]
    w = 1 + 0.3 * torch.randn(D, generator=g)
    freq = ref.frequencies(R, 1e3)[0]
    cache, batch, d = s.device()
    q = torch.zeros((new, D), dtype=torch.bfloat16, device="cuda")
    moe.moe_rope_append(cache, batch, x.cuda(), new, 1, q, freq=torch.as_tensor(freq, device="cuda"), q_weight=w.cuda(),
                        k_weight=w.cuda(), eps=eps)
    torch.cuda.synchronize()
    e = float(np.float32(eps))
    for i, got in ((0, q.cpu()), (1, torch.stack([d["k"][s.place(0, t)][0] for t in range(new)]).cpu())):
        a = ref.head_norm(x[:, i * D:(i + 1) * D].double().numpy(), w.double().numpy(), e)
        r, m = ref.rotate(a, np.arange(new), freq, 1.0, False)
        err = np.abs(got.double().numpy() - r)
        # (what is below 2^-126 may be flushed)
        assert (err <= 2.0 ** -8 * np.abs(r) + 1.01 * 2.0 ** -19 * m + 2.0 ** -125).all()
