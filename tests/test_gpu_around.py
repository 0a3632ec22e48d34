"""The calls around the layer as they are used together: two layers with the
residual stream and its norm between them, then the output head and the
acceptance of sampled and of greedy drafts.  Every call's result is compared
with the 64-bit reference of what it was given."""

import numpy as np
import pytest
import torch

import oracle
import synth
from helpers import ORACLE_THREADS, TOL, DeviceLayer, host, rowwise_rel_err, small_cfg
from oracle import around

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _head(V, H, seed):
    """Codes and block scales of a [V][H] head, as a quantiser makes them."""
    w = np.random.default_rng(seed).standard_normal((V, H)).astype(np.float32) * 0.05
    vb, hb = -(-V // 128), -(-H // 128)
    pad = np.zeros((vb * 128, hb * 128), np.float32)
    pad[:V, :H] = w
    scale = np.maximum(np.abs(pad).reshape(vb, 128, hb, 128).max(axis=(1, 3)), 1e-30) / np.float32(448)
    full = np.repeat(np.repeat(scale, 128, 0)[:V], 128, 1)[:, :H].astype(np.float32)
    codes = (torch.as_tensor(w) / torch.as_tensor(full)).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.numpy(), scale.astype(np.float32)


@pytest.mark.parametrize("T", [1, 4, 16])
def test_two_layers_head_and_acceptance(T):
    import routed_expert_ffn_gemv_amd as moe
    H, V = 256, 5000
    rng = np.random.default_rng(T)
    cfg = small_cfg(E=32, k=4, H=H, I=64, T=T, layers=2)
    resid = torch.as_tensor(rng.standard_normal((T, H)).astype(np.float32), device="cuda")
    weights = [torch.as_tensor((1 + 0.1 * rng.standard_normal(H)).astype(np.float32), device="cuda")
               for _ in range(3)]
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    moe.moe_add_rmsnorm(T, H, None, resid, weights[0], EPS, x=x)
    y = None
    for layer in range(2):
        xb = host(x.view(torch.int16)).view(np.uint16).copy()
        L = DeviceLayer(cfg, layer, x=xb)
        o = L.outputs()
        ws = moe.workspace(L.desc, T)
        moe.moe_layer(L.desc, x, T, o["y"], o["idx"], o["gate"], o["slot_idx"], o["miss"], o["miss_off"], ws)
        torch.cuda.synchronize()
        ref = oracle.layer_from_synth(cfg, layer, xb, threads=ORACLE_THREADS)
        assert rowwise_rel_err(host(o["y"]), ref["y"]) <= TOL
        y = o["y"]
        if layer == 0:
            before = host(resid).copy()
            moe.moe_add_rmsnorm(T, H, y, resid, weights[1], EPS, resid_out=resid, x=x)
            torch.cuda.synchronize()
            np.testing.assert_array_equal(host(resid), before + host(y))
            n = around.rms_norm(host(resid), host(weights[1]), EPS)
            assert (np.abs(x.double().cpu().numpy() - n) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(n)).all()
    x8 = torch.empty((T, H), dtype=torch.uint8, device="cuda")
    xs = torch.empty((T, H // 128), device="cuda")
    moe.moe_add_rmsnorm(T, H, y, resid, weights[2], EPS, x8=x8, x8_scale=xs)
    w8, w_scale = _head(V, H, 7)
    logits = torch.empty((T, V), device="cuda")
    moe.moe_scaled_linear(x8, xs, T, torch.as_tensor(w8, device="cuda"),
                          torch.as_tensor(w_scale, device="cuda"), V, H, logits)
    torch.cuda.synchronize()
    want, mag = around.scaled_linear(host(x8), host(xs), w8, w_scale)
    assert (np.abs(host(logits) - want) <= (259 + H / 128) * 2.0 ** -24 * mag).all()

    u = rng.random(T, dtype=np.float32)
    lg = host(logits)
    tokens = [around.sample_row(lg[t], float(u[t]), temperature=float(np.float32(0.8)), top_k=50,
                                top_p=float(np.float32(0.9)))[0] for t in range(T)]
    draft = np.array(tokens[:T - 1], np.int32)
    if T > 2:
        draft[T - 2] = (draft[T - 2] + 1) % V
    full = lambda v, dtype: torch.full((T,), v, dtype=dtype, device="cuda")  # noqa: E731
    out, n_out = full(-5, torch.int32), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_sample_workspace_size(T, V), dtype=torch.uint8, device="cuda")
    dr = torch.as_tensor(draft, device="cuda") if T > 1 else None
    moe.moe_verify_sample(logits, T, V, dr, torch.as_tensor(u, device="cuda"), out, n_out, ws,
                          temperature=full(0.8, torch.float32), top_k=full(50, torch.int32),
                          top_p=full(0.9, torch.float32))
    torch.cuda.synchronize()
    assert host(out).tolist() == tokens
    assert int(host(n_out)[0]) == (T if T <= 2 else T - 1)

    # temperature 0 keeps what moe_verify_accept keeps
    g = lg.argmax(axis=1).astype(np.int32)
    gd = torch.as_tensor(g[:T - 1], device="cuda") if T > 1 else None
    moe.moe_verify_sample(logits, T, V, gd, torch.as_tensor(u, device="cuda"), out, n_out, ws,
                          temperature=full(0.0, torch.float32))
    out2, n2 = full(-5, torch.int32), torch.zeros(1, dtype=torch.int32, device="cuda")
    vws = torch.empty(max(moe.moe_verify_workspace_size(T, V), 256), dtype=torch.uint8, device="cuda")
    moe.moe_verify_accept(logits, T, V, gd, out2, n2, vws)
    torch.cuda.synchronize()
    assert host(out).tolist() == host(out2).tolist() == g.tolist()
    assert int(host(n_out)[0]) == int(host(n2)[0]) == T


def test_one_graph_from_norm_to_token():
    """Norm, head and sampling captured once and replayed on new inputs, with
    eager work on other buffers between the replays; every replay equals the
    eager result."""
    import routed_expert_ffn_gemv_amd as moe
    T, H, V = 3, 512, 40961
    rng = np.random.default_rng(1)
    w8, w_scale = (torch.as_tensor(v, device="cuda") for v in _head(V, H, 2))
    weight = torch.ones(H, device="cuda")
    temp = torch.full((T,), 0.7, device="cuda")

    def buffers():
        e = lambda *s, **k: torch.zeros(s, device="cuda", **k)  # noqa: E731
        return dict(y=e(T, H), resid=e(T, H), out=e(T, H), x8=e(T, H, dtype=torch.uint8), xs=e(T, H // 128),
                    logits=e(T, V), u=e(T), tok=e(T, dtype=torch.int32), prob=e(T),
                    ws=e(moe.moe_sample_workspace_size(T, V), dtype=torch.uint8))

    def step(b):
        moe.moe_add_rmsnorm(T, H, b["y"], b["resid"], weight, EPS, resid_out=b["out"], x8=b["x8"],
                            x8_scale=b["xs"])
        moe.moe_scaled_linear(b["x8"], b["xs"], T, w8, w_scale, V, H, b["logits"])
        moe.moe_sample(b["logits"], T, V, b["u"], b["tok"], b["ws"], temperature=temp, prob=b["prob"])

    a, b = buffers(), buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a)
    for _ in range(4):
        for key in ("y", "resid"):
            v = torch.as_tensor(rng.standard_normal((T, H)).astype(np.float32))
            a[key].copy_(v)
            b[key].copy_(v)
        v = torch.as_tensor(rng.random(T, dtype=np.float32))
        a["u"].copy_(v)
        b["u"].copy_(v)
        g.replay()
        step(b)
        torch.cuda.synchronize()
        for key in ("out", "x8", "xs", "logits", "tok", "prob"):
            assert torch.equal(a[key], b[key]), key


def test_two_streams_at_once():
    """The same calls on two streams with workspaces of their own."""
    import routed_expert_ffn_gemv_amd as moe
    T, V = 8, 90001
    rng = np.random.default_rng(5)
    sets = []
    for k in range(2):
        x = torch.as_tensor((rng.standard_normal((T, V)) * 2).astype(np.float32), device="cuda")
        u = torch.as_tensor(rng.random(T, dtype=np.float32), device="cuda")
        ws = torch.empty(moe.moe_sample_workspace_size(T, V), dtype=torch.uint8, device="cuda")
        sets.append((x, u, ws, torch.empty(T, dtype=torch.int32, device="cuda"), torch.cuda.Stream()))
    want = []
    for x, u, ws, tok, _ in sets:
        moe.moe_sample(x, T, V, u, tok, ws)
        torch.cuda.synchronize()
        want.append(tok.clone())
    torch.cuda.synchronize()
    for _ in range(10):
        for x, u, ws, tok, st in sets:
            moe.moe_sample(x, T, V, u, tok, ws, stream=st)
    torch.cuda.synchronize()
    for (_, _, _, tok, _), w in zip(sets, want):
        assert torch.equal(tok, w)
