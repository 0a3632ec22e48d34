"""The calls around the layer on the host: refused arguments (before any HIP
call, so no GPU is needed) and the references' own pins."""

import numpy as np
import pytest
import torch

import routed_expert_ffn_gemv_amd as moe
from oracle import around

FAKE = 1 << 20      # an aligned non-null address; never dereferenced here
F32, BF16 = moe.MOE_W_F32, moe.MOE_W_BF16
OK, INVALID, UNSUPPORTED, WORKSPACE = (moe.MOE_OK, moe.MOE_ERR_INVALID, moe.MOE_ERR_UNSUPPORTED,
                                       moe.MOE_ERR_WORKSPACE)


def _norm(**kw):
    a = dict(T=4, H=256, y=FAKE, y_fmt=F32, ys=256, r=FAKE, r_fmt=BF16, rs=256, w=FAKE, w_fmt=BF16,
             eps=1e-6, ro=FAKE, ros=256, x=FAKE, xs=256, x8=FAKE, sc=FAKE)
    a.update(kw)
    return moe.lib.moe_add_rmsnorm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), OK), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=32769), UNSUPPORTED),
    (dict(T=(1 << 22) + 1), UNSUPPORTED),
    (dict(r=None), INVALID), (dict(w=None), INVALID), (dict(x=None, x8=None, sc=None, ro=None), INVALID),
    (dict(x8=None), INVALID), (dict(sc=None), INVALID),
    (dict(r_fmt=moe.MOE_W_Q2B32), UNSUPPORTED), (dict(w_fmt=9), UNSUPPORTED), (dict(y_fmt=-1), UNSUPPORTED),
    (dict(ys=255), INVALID), (dict(rs=255), INVALID), (dict(ro=FAKE * 2, ros=255), INVALID),
    (dict(xs=0), INVALID), (dict(ros=264), INVALID),            # in place with another stride
    (dict(y=FAKE + 2), INVALID), (dict(r=FAKE + 1, ro=None), INVALID), (dict(x=FAKE + 1), INVALID),
    (dict(sc=FAKE + 2), INVALID), (dict(w=FAKE + 1), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
])
def test_norm_refusals(kw, status):
    assert _norm(**kw) == status


def test_norm_binding_refusals():
    """Formats, shapes and places are checked before the library is called."""
    r = torch.zeros((4, 256))
    w = torch.ones(256)
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    call = moe.moe_add_rmsnorm
    for bad in (
        lambda: call(4, 256, None, r, w, 1e-6, x=x),                       # not on a GPU
        lambda: call(5, 256, None, r, w, 1e-6, x=x),                       # too few rows
        lambda: call(4, 257, None, r, w, 1e-6, x=x),
        lambda: call(4, 256, r.half(), r, w, 1e-6, x=x),
        lambda: call(4, 256, None, r, w[:255], 1e-6, x=x),
        lambda: call(4, 256, None, r, w, 1e-6, x=r),                       # x is bf16
        lambda: call(4, 256, None, r, w, 1e-6, resid_out=x),               # another format
        lambda: call(4, 256, None, r.t().contiguous().t(), w, 1e-6, x=x),  # columns apart
        lambda: call(4, 256, None, r, w, 1e-6, x8=x, x8_scale=r),
        lambda: call(4, 256, None, r, w, 1e-6, x8=torch.zeros((4, 256), dtype=torch.uint8),
                     x8_scale=r[:1, :7]),
    ):
        with pytest.raises(ValueError):
            bad()


def test_e4m3_values_are_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(around.E4M3, t)
