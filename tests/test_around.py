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


def _sample(verify=False, **kw):
    a = dict(x=FAKE, fmt=F32, T=4, V=1000, stride=1000, par=None, u=FAKE)
    if verify:
        a["draft"] = FAKE
    a.update(tok=FAKE, prob=FAKE)
    if verify:
        a["n"] = FAKE
    a.update(ws=FAKE, size=1 << 30)
    a.update(kw)
    f = moe.lib.moe_verify_sample if verify else moe.lib.moe_sample
    return f(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), OK), (dict(T=-1), INVALID), (dict(V=0, stride=0), INVALID),
    (dict(T=16385), UNSUPPORTED), (dict(V=(1 << 26) + 1, stride=1 << 27), UNSUPPORTED),
    (dict(fmt=moe.MOE_W_Q4B32), UNSUPPORTED), (dict(x=None), INVALID), (dict(x=FAKE + 2), INVALID),
    (dict(fmt=BF16, x=FAKE + 1), INVALID), (dict(stride=999), INVALID), (dict(u=None), INVALID),
    (dict(u=FAKE + 2), INVALID), (dict(tok=None), INVALID), (dict(tok=FAKE + 1), INVALID),
    (dict(prob=FAKE + 2), INVALID), (dict(ws=None), INVALID), (dict(ws=FAKE + 64), INVALID),
    (dict(size=1000), WORKSPACE),
])
def test_sample_refusals(kw, status):
    assert _sample(**kw) == status
    if kw != dict(T=0) and kw != dict(T=16385):
        assert _sample(verify=True, **kw) == status


def test_verify_sample_refusals():
    import ctypes
    assert _sample(verify=True, T=0) == INVALID
    assert _sample(verify=True, T=65) == UNSUPPORTED
    assert _sample(verify=True, draft=None) == INVALID
    assert _sample(verify=True, n=None) == INVALID
    assert _sample(verify=True, n=FAKE + 2) == INVALID
    assert _sample(verify=True, draft=FAKE + 2) == INVALID
    n = ctypes.c_size_t(0)
    size = moe.lib.moe_sample_workspace_size
    assert size(4, 1000, None) == INVALID and size(-1, 1000, ctypes.byref(n)) == INVALID
    assert size(4, 0, ctypes.byref(n)) == INVALID and size(16385, 9, ctypes.byref(n)) == UNSUPPORTED
    assert size(4, 1000, ctypes.byref(n)) == OK and n.value % 256 == 0 and n.value > 0
    assert _sample(size=n.value - 1) == WORKSPACE
    bad = moe.moe_sample_params(FAKE, FAKE, FAKE + 2, FAKE)
    assert _sample(par=ctypes.byref(bad)) == INVALID


def test_sample_binding_refusals():
    x = torch.zeros((4, 100))
    u, tok = torch.zeros(4), torch.zeros(4, dtype=torch.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    call = moe.moe_sample
    for bad in (
        lambda: call(x, 4, 100, u, tok, ws),                                    # not on a GPU
        lambda: call(x, 5, 100, u, tok, ws),
        lambda: call(x, 4, 101, u, tok, ws),
        lambda: call(x.double(), 4, 100, u, tok, ws),
        lambda: call(x, 4, 100, u.double(), tok, ws),
        lambda: call(x, 4, 100, u, tok.long(), ws),
        lambda: call(x, 4, 100, u, tok, ws, top_k=u),
        lambda: call(x, 4, 100, u, tok, ws, temperature=u[:3]),
        lambda: call(x, 4, 100, u, tok, ws, prob=tok),
        lambda: moe.moe_verify_sample(x, 4, 100, tok[:2], u, tok, tok, ws),     # 3 drafts wanted
        lambda: moe.moe_verify_sample(x, 4, 100, tok, u, tok, u, ws),
    ):
        with pytest.raises(ValueError):
            bad()


def test_sample_reference_by_hand():
    """Probabilities 4/8, 2/8, 1/8, 1/8 (logits in powers of two)."""
    x = np.log(np.array([1.0, 4.0, 2.0, 1.0]))
    row = around.sample_row
    assert [row(x, u)[0] for u in (0.0, 0.49, 0.51, 0.74, 0.76, 0.87, 0.88)] == [1, 1, 2, 2, 0, 0, 3]
    assert row(x, 0.8, top_k=2)[:1] == (2,) and abs(row(x, 0.8, top_k=2)[1] - 1 / 3) < 1e-12
    assert row(x, 0.99, top_p=0.6)[0] == 2 and row(x, 0.99, top_p=0.4)[0] == 1
    assert row(x, 0.99, min_p=0.3)[0] == 2 and row(x, 0.99, min_p=2.0)[0] == 1
    assert row(x, 0.99, temperature=0.0)[0] == 1
    assert row(np.full(3, -np.inf), 0.5)[0] == -1
    assert row(x, 0.99)[0] == 3 and row(x, 0.99, temperature=1e-3)[0] == 1


def _linear(**kw):
    a = dict(x8=FAKE, xs=FAKE, T=4, w8=FAKE, ws_=FAKE, N=300, K=256, out=FAKE, fmt=F32, stride=300,
             ws=FAKE, size=1 << 30)
    a.update(kw)
    return moe.lib.moe_scaled_linear(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), OK), (dict(T=-1), INVALID), (dict(N=0, stride=0), INVALID), (dict(K=0), INVALID),
    (dict(K=200), INVALID), (dict(K=8), INVALID), (dict(K=32784), UNSUPPORTED),
    (dict(N=(1 << 24) + 1, stride=1 << 25), UNSUPPORTED), (dict(T=(1 << 22) + 1), UNSUPPORTED),
    (dict(fmt=moe.MOE_W_Q2B32), UNSUPPORTED), (dict(stride=299), INVALID),
    (dict(x8=None), INVALID), (dict(xs=None), INVALID), (dict(w8=None), INVALID),
    (dict(ws_=None), INVALID), (dict(out=None), INVALID), (dict(x8=FAKE + 8), INVALID),
    (dict(w8=FAKE + 8), INVALID), (dict(xs=FAKE + 2), INVALID), (dict(ws_=FAKE + 2), INVALID),
    (dict(out=FAKE + 2), INVALID), (dict(fmt=BF16, out=FAKE + 1), INVALID),
])
def test_linear_refusals(kw, status):
    assert _linear(**kw) == status


def test_linear_binding_refusals():
    x8, w8 = torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((300, 256), dtype=torch.uint8)
    xs, ws = torch.zeros((4, 2)), torch.zeros((3, 2))
    out = torch.zeros((4, 300))
    call = moe.moe_scaled_linear
    for bad in (
        lambda: call(x8, xs, 4, w8, ws, 300, 256, out),                     # not on a GPU
        lambda: call(x8, xs, 5, w8, ws, 300, 256, out),
        lambda: call(x8, xs[:, :1], 4, w8, ws, 300, 256, out),
        lambda: call(x8, xs, 4, w8, ws[:2], 300, 256, out),
        lambda: call(x8, xs, 4, w8[:299], ws, 300, 256, out),
        lambda: call(x8, xs, 4, w8, ws, 300, 256, out[:, :299]),
        lambda: call(x8.float(), xs, 4, w8, ws, 300, 256, out),
        lambda: call(x8, xs.double(), 4, w8, ws, 300, 256, out),
        lambda: call(x8, xs, 4, w8, ws, 300, 256, out.half()),
        lambda: call(x8, xs, 4, w8.t().contiguous().t(), ws, 300, 256, out),
    ):
        with pytest.raises(ValueError):
            bad()


def test_linear_reference_by_hand():
    x8 = np.array([[0x38, 0x40] + [0] * 14], np.uint8)        # 1, 2
    w8 = np.array([[0x38, 0xB8] + [0] * 14, [0x08, 0x01] + [0] * 14], np.uint8)   # 1, -1; 2^-6, 2^-9
    out, mag = around.scaled_linear(x8, np.array([[2.0]], np.float32), w8, np.array([[4.0]], np.float32))
    np.testing.assert_array_equal(out, [[-8.0, 8 * (2.0 ** -6 + 2.0 ** -8)]])
    np.testing.assert_array_equal(mag, [[24.0, 8 * (2.0 ** -6 + 2.0 ** -8)]])
