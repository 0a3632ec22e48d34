"""GPU parity of moe_add_rmsnorm: bit for bit against the same fp32 steps on
the CPU, and within the roundings of the formula in 64 bits.

Tolerances: inv is rounded once (2^-24) and n = (v * inv) * weight twice
more, so n is off by less than 2^-22 of itself; x adds bf16's half step
(2^-8), a scale one division (2^-24), a code e4m3's half step (2^-4, or
2^-10 scales where the code is subnormal)."""

import numpy as np
import pytest
import torch

from oracle import around

pytestmark = pytest.mark.gpu

EPS = 1e-6
N_OFF = 2.0 ** -22


def _cpu(y, resid, weight, eps=EPS):
    """The definition's fp32 steps: (v, n, x, x8 codes, scales)."""
    T, H = resid.shape
    v = resid if y is None else (resid.float() + y.float()).to(resid.dtype)
    f = v.float()
    inv = (1.0 / torch.sqrt(f.double().square().mean(dim=1, keepdim=True) + np.float64(np.float32(eps)))).float()
    n = f * inv * weight.float()
    nb = -(-H // 128)
    blocks = torch.nn.functional.pad(n, (0, nb * 128 - H)).view(T, nb, 128)
    scale = blocks.abs().amax(dim=2).clamp_min(around.SCALE_FLOOR) / 448.0
    x8 = (blocks / scale[:, :, None]).reshape(T, nb * 128)[:, :H].to(torch.float8_e4m3fn)
    return v, n, n.to(torch.bfloat16), x8, scale


def _inputs(T, H, y_dtype, r_dtype, w_dtype, seed, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    y = None if y_dtype is None else torch.randn((T, H), generator=g).to(y_dtype)
    resid = (torch.randn((T, H), generator=g) * scale).to(r_dtype)
    weight = (1 + 0.3 * torch.randn(H, generator=g)).to(w_dtype)
    return y, resid, weight


def _run(y, resid, weight, eps=EPS, want=("resid", "x", "x8"), stream=None):
    """On the GPU, outputs with a guard row behind the last one."""
    import routed_expert_ffn_gemv_amd as moe
    T, H = resid.shape
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    nb = -(-H // 128)
    out = {
        "resid": torch.full((T + 1, H), -77.0, dtype=resid.dtype, device="cuda"),
        "x": torch.full((T + 1, H), -77.0, dtype=torch.bfloat16, device="cuda"),
        "x8": torch.full((T + 1, H), 0x55, dtype=torch.uint8, device="cuda"),
        "scale": torch.full((T + 1, nb), -77.0, dtype=torch.float32, device="cuda"),
    }
    p = lambda k: out[k] if k in want else None  # noqa: E731
    moe.moe_add_rmsnorm(T, H, d(y), d(resid), d(weight), eps, resid_out=p("resid"), x=p("x"),
                        x8=p("x8"), x8_scale=out["scale"] if "x8" in want else None, stream=stream)
    torch.cuda.synchronize()
    out = {k: t.cpu() for k, t in out.items()}
    for k in ("resid", "x", "scale"):
        assert (out[k][T] == -77).all(), f"{k}: the row behind the last one was written"
        if k not in want and not (k == "scale" and "x8" in want):
            assert (out[k] == -77).all()
    assert (out["x8"][T] == 0x55).all()
    return {k: t[:T] for k, t in out.items()}


def _check(y, resid, weight, eps=EPS, **kw):
    got = _run(y, resid, weight, eps, **kw)
    v, n, x, x8, scale = _cpu(y, resid, weight, eps)
    assert torch.equal(got["resid"], v)
    assert torch.equal(got["scale"], scale)
    assert torch.equal(got["x"].view(torch.int16), x.view(torch.int16))
    assert torch.equal(got["x8"], x8.view(torch.uint8))
    ref = around.rms_norm(v.double().numpy(), weight.double().numpy(), float(np.float32(eps)))
    tiny = 2.0 ** -126
    assert (np.abs(got["x"].double().numpy() - ref) <= (2.0 ** -8 + N_OFF) * np.abs(ref) + tiny).all()
    s = around.block_scales(ref)
    assert (np.abs(got["scale"].double().numpy() - s) <= (N_OFF + 2.0 ** -24) * s).all()
    sg = np.repeat(got["scale"].double().numpy(), 128, axis=1)[:, :ref.shape[1]]
    val = around.E4M3[got["x8"].numpy()] * sg
    assert (np.abs(val - ref) <= (2.0 ** -4 + 4 * N_OFF) * np.abs(ref) + 2.0 ** -10 * sg).all()


F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("H", [1, 7, 8, 64, 127, 128, 129, 504, 512, 1000, 1024, 1030, 2048, 2056,
                               4096, 5000, 8192, 10000, 16384, 20001, 32768])
def test_widths(H):
    """Every variant of the split, whole and ragged rows, at 1 and 6 rows."""
    for T in (1, 6):
        y, r, w = _inputs(T, H, F32, BF16, BF16, seed=H + T)
        _check(y, r, w)


@pytest.mark.parametrize("y_dtype", [None, F32, BF16])
@pytest.mark.parametrize("r_dtype", [F32, BF16])
@pytest.mark.parametrize("w_dtype", [F32, BF16])
def test_formats(y_dtype, r_dtype, w_dtype):
    for H in (96, 2048):
        _check(*_inputs(9, H, y_dtype, r_dtype, w_dtype, seed=5))


@pytest.mark.parametrize("scale", [1e-42, 1e-25, 1e12, 1e30])
def test_ranges(scale):
    """Subnormal rows, rows whose squares pass the fp32 range."""
    _check(None, *_inputs(4, 640, None, F32, F32, 3, scale)[1:])


def test_zero_rows_and_blocks():
    y, r, w = _inputs(5, 512, F32, F32, F32, 2)
    r[1], y[1] = 0.0, 0.0
    r[2, 128:256], y[2, 128:256] = 0.0, 0.0
    y[3] = -r[3]
    _check(y, r, w)
    _check(y, r, torch.zeros_like(w))
    got = _run(torch.zeros_like(y), torch.zeros_like(r), w, eps=1e-6)
    assert (got["x8"] & 127 == 0).all() and (got["scale"] == 2.0 ** -126).all()


def test_many_rows():
    y, r, w = _inputs(3001, 256, BF16, F32, BF16, 8)
    _check(y, r, w)


@pytest.mark.parametrize("H", [9, 100, 250, 255, 256, 257, 513, 2049, 4099])
@pytest.mark.parametrize("T", [1, 3, 8, 21])
def test_rows_that_share_a_workgroup_or_start_anywhere(T, H):
    for y, r in ((F32, BF16), (BF16, F32)):
        _check(*_inputs(T, H, y, r, BF16, T + H))


def test_more_rows_than_one_grid_dimension_takes():
    """One workgroup per row, 2^20 + 5 rows: rows at both ends and around the
    border against the definition, and no row left out."""
    import routed_expert_ffn_gemv_amd as moe
    T, H = 2 ** 20 + 5, 1032
    resid = torch.empty((T, H), dtype=BF16, device="cuda")
    resid.copy_((torch.arange(T, device="cuda") % 251 + 1).to(BF16)[:, None].expand(T, H))
    resid[:, 7] = -3.0
    weight = torch.ones(H, device="cuda")
    x = torch.zeros((T, H), dtype=BF16, device="cuda")
    moe.moe_add_rmsnorm(T, H, None, resid, weight, EPS, x=x)
    torch.cuda.synchronize()
    rows = [0, 1, 2 ** 20 - 1, 2 ** 20, 2 ** 20 + 1, T - 1]
    want = _cpu(None, resid[rows].cpu(), weight.cpu())[2]
    assert torch.equal(x[rows].cpu(), want)
    assert bool((x[:, 0] != 0).all())


def test_outputs_one_by_one():
    y, r, w = _inputs(3, 384, F32, BF16, BF16, 4)
    v, n, x, x8, scale = _cpu(y, r, w)
    assert torch.equal(_run(y, r, w, want=("resid",))["resid"], v)
    assert torch.equal(_run(y, r, w, want=("x",))["x"], x)
    assert torch.equal(_run(y, r, w, want=("x8",))["x8"], x8.view(torch.uint8))


@pytest.mark.parametrize("pad,off", [(8, 0), (5, 0), (8, 1), (0, 3)])
def test_strided_unaligned_and_in_place(pad, off):
    """Rows inside wider buffers, starting at any element, updated in place;
    what lies between the rows stays."""
    import routed_expert_ffn_gemv_amd as moe
    T, H = 5, 2048
    y, r, w = _inputs(T, H, BF16, F32, BF16, 6)

    def wide(t, fill):
        buf = torch.full((T * (H + pad) + off + 16,), fill, dtype=t.dtype, device="cuda")
        view = buf[off:off + T * (H + pad)].view(T, H + pad)[:, :H]
        view.copy_(t)
        return buf, view

    yb, yv = wide(y, 9.0)
    rb, rv = wide(r, 9.0)
    xb, xv = wide(torch.zeros_like(y), 9.0)
    moe.moe_add_rmsnorm(T, H, yv, rv, w.cuda(), EPS, resid_out=rv, x=xv)
    torch.cuda.synchronize()
    v, n, x, _, _ = _cpu(y, r, w)
    assert torch.equal(rv.cpu(), v) and torch.equal(xv.cpu(), x)
    for buf in (rb, xb):
        rest = torch.ones(buf.numel(), dtype=torch.bool)
        rest[off:off + T * (H + pad)].view(T, H + pad)[:, :H] = False
        assert (buf.cpu()[rest] == 9.0).all()


def test_other_stream_and_replayed_graph():
    import routed_expert_ffn_gemv_amd as moe
    T, H = 4, 2048
    y, r, w = (t.cuda() for t in _inputs(T, H, F32, F32, BF16, 7))
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x8 = torch.zeros((T, H), dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.zeros((T, H // 128), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_add_rmsnorm(T, H, y, r, w, EPS, x=x, x8=x8, x8_scale=sc, stream=side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_add_rmsnorm(T, H, y, r, w, EPS, x=x, x8=x8, x8_scale=sc)
    for seed in (20, 21, 22):
        y2, r2, _ = _inputs(T, H, F32, F32, BF16, seed)
        y.copy_(y2)
        r.copy_(r2)
        g.replay()
        torch.cuda.synchronize()
        _, _, x_ref, x8_ref, s_ref = _cpu(y2, r2, w.cpu())
        assert torch.equal(x.cpu(), x_ref) and torch.equal(sc.cpu(), s_ref)
        assert torch.equal(x8.cpu().view(torch.uint8), x8_ref.view(torch.uint8))
