"""moe_scaled_linear where workgroups walk over several tiles, where rings of
LDS buffers are filled again and again, and beyond 2^31 bytes.  Whole outputs
are compared with the product in 64 bits; tolerances as in
test_gpu_scaled_linear.py."""

import pytest
import torch

from oracle import around

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _inputs(T, N, K, seed):
    """Codes of every magnitude and their scales, on the GPU."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def codes(rows):
        c = torch.randint(0, 256, (rows, K), dtype=torch.uint8, device="cuda", generator=g)
        for i in range(0, rows, 8192):     # (NaN codes to 1)
            part = c[i:i + 8192]
            part[(part & 127) == 127] = 0x38
        return c

    def scales(rows):
        return (0.2 + 1.8 * torch.rand((rows, -(-K // 128)), device="cuda", generator=g)) / 448

    return codes(T), scales(T), codes(N), scales(-(-N // 128))


def _values(codes, scale, table):
    rows, K = codes.shape
    v = table[codes.to(torch.int32)]
    for b in range(scale.shape[1]):
        v[:, b * 128:(b + 1) * 128] *= scale[:, b:b + 1]
    return v


def _reference(x8, xs, w8, ws, t, n):
    """(product, sum of absolute values) of rows t and weight rows n in 64 bits."""
    table = torch.as_tensor(around.E4M3, device="cuda")
    x = _values(x8[t], xs[t].double(), table)
    rows = torch.arange(w8.shape[0], device="cuda")[n]
    w = _values(w8[n], ws.double()[rows // 128], table).t().contiguous()
    return torch.mm(x, w), torch.mm(x.abs(), w.abs())


def _out(T, N, dtype, pad, off=0):
    buf = torch.full(((T + 1) * (N + pad) + off,), -776.0, dtype=dtype, device="cuda")
    return buf[off:].view(T + 1, N + pad)


def _call(x8, xs, w8, ws, out):
    import routed_expert_ffn_gemv_amd as moe
    T, K = x8.shape
    N = w8.shape[0]
    moe.moe_scaled_linear(x8, xs, T, w8, ws, N, K, out[:T, :N])
    torch.cuda.synchronize()
    assert bool((out[T] == -776).all()) and bool((out[:, N:] == -776).all()), "written outside the output"


def _compare(out, data, t, n):
    T, K = data[0].shape
    want, mag = _reference(*data, t, n)
    tol = (259 + K / 128) * 2.0 ** -24 * mag
    if out.dtype == BF16:
        if T > 16:
            tol = tol + 7 * 2.0 ** -13 * mag
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    bad = (out[:T, :data[2].shape[0]][t, n].double() - want).abs() > tol
    bad = bad | torch.isnan(out[:T, :data[2].shape[0]][t, n])
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


ALL = slice(None)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,N,K,pad", [
    (600, 40000, 640, 8), (600, 40000, 1008, 3), (600, 40000, 128, 8), (600, 40000, 48, 4),
    (300, 40000, 640, 8), (300, 40000, 1040, 8), (300, 40000, 112, 8), (512, 32768, 384, 0),
    (40, 100000, 640, 8), (40, 100000, 1040, 4), (50, 151936, 272, 0), (64, 98304, 256, 8),
    (5000, 4096, 640, 0), (5000, 4096, 80, 8), (3000, 4104, 528, 0), (2000, 9000, 400, 0),
    (32, 33004, 2064, 4), (24, 100000, 528, 8), (20, 33000, 1040, 8),
])
def test_workgroups_with_several_tiles(T, N, K, pad, dtype):
    """256 x 256, 256 x 128, 128 x 128 and 128 x 64 outputs per tile, up to
    three tiles per workgroup, one to nine blocks of columns; stores of 16
    bytes (left under way behind the next tile's loads), 8 and single ones."""
    data = _inputs(T, N, K, T + N + K)
    out = _out(T, N, dtype, pad)
    _call(*data, out)
    _compare(out, data, ALL, ALL)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_replayed_with_several_tiles(dtype):
    """Captured once, replayed on other inputs: bits of the eager call."""
    import routed_expert_ffn_gemv_amd as moe
    T, N, K = 600, 40000, 640
    data = _inputs(T, N, K, 1)
    out = torch.zeros((T, N), dtype=dtype, device="cuda")
    moe.moe_scaled_linear(*data[:2], T, *data[2:], N, K, out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_scaled_linear(*data[:2], T, *data[2:], N, K, out)
    eager = torch.zeros_like(out)
    for seed in (2, 3, 4):
        new = _inputs(T, N, K, seed)
        for a, b in zip(data, new):
            a.copy_(b)
        out.zero_()
        g.replay()
        moe.moe_scaled_linear(*new[:2], T, *new[2:], N, K, eager)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def _room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"{gib} GiB of GPU memory wanted")


@pytest.mark.parametrize("T,dtype", [(1, F32), (16, BF16), (40, F32), (100, BF16)])
def test_weights_beyond_31_bits(T, dtype):
    _room(16)
    N, K = 70000, 32768                       # byte 2^31 is weight row 65,536's first
    data = _inputs(T, N, K, T)
    out = _out(T, N, dtype, 8)
    _call(*data, out)
    for n in (slice(0, 256), slice(65400, 65700), slice(69700, N)):
        _compare(out, data, ALL, n)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_tokens_beyond_31_bits(dtype):
    _room(16)
    T, N, K = 70000, 64, 32768
    data = _inputs(T, N, K, 5)
    out = _out(T, N, dtype, 8)
    _call(*data, out)
    for t in (slice(0, 256), slice(65400, 65700), slice(69700, T)):
        _compare(out, data, t, ALL)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_outputs_beyond_31_bits(dtype):
    _room(24)
    T, N, K = 33000, 66000, 144               # element 2^31 is in row 32,534
    data = _inputs(T, N, K, 6)
    out = _out(T, N, dtype, 8)
    _call(*data, out)
    for t in (slice(0, 300), slice(16200, 16400), slice(32400, 32700), slice(32800, T)):
        for n in (slice(0, 300), slice(33000, 33300), slice(N - 300, N)):
            _compare(out, data, t, n)
