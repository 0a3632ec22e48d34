"""The attention half of a layer as its calls are used together: norm, 8-bit
projection, append, attention, 8-bit projection, residual and norm, MoE layer,
over a prompt in chunks, a verify pass and single tokens.  Every call's result
is compared with the 64-bit reference of what it was given."""

import numpy as np
import pytest
import torch

import oracle
from helpers import ORACLE_THREADS, TOL, DeviceLayer, host, rowwise_rel_err, small_cfg
from oracle import around
from oracle import attention as ref
from test_gpu_around import _head
from test_gpu_attention import _off

pytestmark = pytest.mark.gpu

EPS = 1e-6


class Step:
    """A small model's layer and the buffers of one sequence."""

    def __init__(self, cache, H=256, Hq=4, Hkv=2, D=128, R=64, page=16, pages=20, T=64):
        import routed_expert_ffn_gemv_amd as moe
        self.moe, self.H, self.Hq, self.Hkv, self.D, self.R, self.page = moe, H, Hq, Hkv, D, R, page
        rng = np.random.default_rng(3)
        e = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        self.width = (Hq + 2 * Hkv) * D
        self.w_qkv, self.s_qkv = _head(self.width, H, 1)
        self.w_o, self.s_o = _head(H, Hq * D, 2)
        self.d = {n: torch.as_tensor(getattr(self, n), device="cuda") for n in ("w_qkv", "s_qkv", "w_o", "s_o")}
        self.norm = [torch.as_tensor((1 + 0.1 * rng.standard_normal(n)).astype(np.float32), device="cuda")
                     for n in (H, D, D, H)]
        freq, self.rot_scale = moe.moe_rope_frequencies(R, 1e4, "bands", 4.0, 128)
        self.freq = freq.cuda()
        f8 = cache == "f8"
        shape = (pages, page, Hkv, D)
        self.k, self.v = (e(*shape, dtype=torch.uint8 if f8 else torch.bfloat16) for _ in "kv")
        self.ks, self.vs = (e(*shape[:3]) if f8 else None for _ in "kv")
        self.cache = moe.KVCache(self.k, self.v, self.ks, self.vs)
        self.table = torch.as_tensor(rng.permutation(pages)[None].astype(np.int32), device="cuda")
        self.q_off, self.kv_len = e(2, dtype=torch.int32), e(1, dtype=torch.int32)
        self.batch = moe.KVBatch(self.q_off, self.kv_len, self.table)
        self.ws = e(moe.moe_paged_attention_workspace_size(T, 1, Hq, Hkv, D), dtype=torch.uint8)
        self.b = dict(x8=e(T, H, dtype=torch.uint8), xs=e(T, H // 128), qkv=e(T, self.width, dtype=torch.bfloat16),
                      q=e(T, Hq * D, dtype=torch.bfloat16), o8=e(T, Hq * D, dtype=torch.uint8), os=e(T, Hq * D // 128),
                      y=e(T, H, dtype=torch.bfloat16), x=e(T, H, dtype=torch.bfloat16))

    def run(self, resid, T):
        """resid [T][H] += the attention half; b["x"]: the MoE layer's input."""
        moe, b, d, D = self.moe, self.b, self.d, self.D
        moe.moe_add_rmsnorm(T, self.H, None, resid, self.norm[0], EPS, x8=b["x8"], x8_scale=b["xs"])
        moe.moe_scaled_linear(b["x8"], b["xs"], T, d["w_qkv"], d["s_qkv"], self.width, self.H, b["qkv"])
        moe.moe_rope_append(self.cache, self.batch, b["qkv"], T, self.Hq, b["q"], freq=self.freq,
                            rot_scale=self.rot_scale, q_weight=self.norm[1], k_weight=self.norm[2], eps=EPS)
        moe.moe_paged_attention(self.cache, self.batch, b["q"], T, self.Hq, D ** -0.5, self.ws, x8=b["o8"],
                                x8_scale=b["os"])
        moe.moe_scaled_linear(b["o8"], b["os"], T, d["w_o"], d["s_o"], self.H, self.Hq * D, b["y"])
        moe.moe_add_rmsnorm(T, self.H, b["y"], resid, self.norm[3], EPS, resid_out=resid, x=b["x"])

    def set(self, new, length):
        self.q_off.copy_(torch.tensor([0, new], dtype=torch.int32))
        self.kv_len.fill_(length)

    def cached(self, length):
        """Keys and values of the first positions in 64 bits."""
        at = np.arange(length)
        page, slot = host(self.table)[0][at // self.page], at % self.page
        out = []
        for t, s in ((self.k, self.ks), (self.v, self.vs)):
            if s is None:
                out.append(t.double().cpu().numpy()[page, slot])
            else:
                out.append(around.E4M3[host(t)][page, slot] * host(s).astype(np.float64)[page, slot][..., None])
        return out


@pytest.mark.parametrize("cache", ["bf16", "f8"])
def test_prompt_verify_and_tokens(cache):
    st = Step(cache)
    rng = np.random.default_rng(9)
    H, Hq, Hkv, D = st.H, st.Hq, st.Hkv, st.D
    keys = []           # what the cache must hold
    length = 0
    for step, T in enumerate((50, 64, 4, 1, 1)):
        start = length
        if step == 3:
            start = length = length - 2         # two of the drafts were not kept: their places are written again
            keys = keys[:length]
        length += T
        resid = torch.as_tensor(rng.standard_normal((T, H)).astype(np.float32), device="cuda")
        before = host(resid).copy()
        st.set(T, length)
        st.run(resid, T)
        torch.cuda.synchronize()
        b = {n: t[:T] for n, t in st.b.items()}
        want, mag = around.scaled_linear(host(b["x8"]), host(b["xs"]), st.w_qkv, st.s_qkv)
        qkv = b["qkv"].double().cpu().numpy()
        assert (np.abs(qkv - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -14 * mag).all()
        # queries, keys and values of what the projection gave
        pos = np.arange(start, length)
        heads = qkv.reshape(T, Hq + 2 * Hkv, D)
        w = [host(n).astype(np.float64) for n in st.norm]
        q, k = np.zeros((T, Hq, D)), np.zeros((T, Hkv, D))
        for h in range(Hq + Hkv):
            a = ref.head_norm(heads[:, h], w[1 if h < Hq else 2], EPS)
            r, m = ref.rotate(a, pos, host(st.freq), st.rot_scale, False)
            if h < Hq:
                q[:, h] = r
                got = b["q"].double().cpu().numpy().reshape(T, Hq, D)[:, h]
                assert (np.abs(got - r) <= 2.0 ** -8 * np.abs(r) + 2.0 ** -18.9 * m).all()
            else:
                k[:, h - Hq] = r
        keys += list(zip(k, heads[:, Hq + Hkv:]))
        ck, cv = st.cached(length)
        for p, (kk, vv) in enumerate(keys):
            for got, value in ((ck[p], kk), (cv[p], vv)):
                amax = np.abs(value).max(axis=1, keepdims=True)
                off = 2.0 ** -8 * np.abs(value) + 2.0 ** -17 * amax if cache == "bf16" else (
                    2.0 ** -4 * np.abs(value) + (2.0 ** -10 / 448 + 2.0 ** -17) * amax)
                assert (np.abs(got - value) <= off).all(), p
        # attention over what the cache holds, and the projection back
        gq = b["q"].double().cpu().numpy().reshape(T, Hq, D)
        o, *scales = ref.attend(gq, ck, cv, pos, np.ones(length, bool), float(np.float32(D ** -0.5)))
        off = _off(cache == "f8", D, o, *scales)
        sc = host(b["os"]).astype(np.float64).reshape(T, Hq, 1)
        got = around.E4M3[host(b["o8"])].reshape(T, Hq, D) * sc
        assert (np.abs(got - o) <= 2.0 ** -4 * (np.abs(o) + off) + 2.0 ** -10 * sc + off).all()
        want, mag = around.scaled_linear(host(b["o8"]), host(b["os"]), st.w_o, st.s_o)
        y = b["y"].double().cpu().numpy()
        assert (np.abs(y - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -14 * mag).all()
        np.testing.assert_array_equal(host(resid), before + b["y"].float().cpu().numpy())
        # and the MoE layer behind it
        if T <= 16:
            xb = host(b["x"].view(torch.int16)).view(np.uint16).copy()
            cfg = small_cfg(E=32, k=4, H=H, I=64, T=T, layers=1)
            L = DeviceLayer(cfg, 0, x=xb)
            out = L.outputs()
            st.moe.moe_layer(L.desc, b["x"], T, out["y"], out["idx"], out["gate"], out["slot_idx"], out["miss"],
                             out["miss_off"], st.moe.workspace(L.desc, T))
            torch.cuda.synchronize()
            layer = oracle.layer_from_synth(cfg, 0, xb, threads=ORACLE_THREADS)
            assert rowwise_rel_err(host(out["y"]), layer["y"]) <= TOL


@pytest.mark.parametrize("cache", ["bf16", "f8"])
def test_one_graph_for_every_step(cache):
    """The half captured once for 4 rows (rows of no sequence behind the last)
    and replayed as the text grows; every replay equals the eager calls."""
    a, b = Step(cache), Step(cache)
    resid = [torch.zeros((4, a.H), device="cuda") for _ in "ab"]
    a.set(4, 4)
    a.run(resid[0], 4)
    torch.cuda.synchronize()
    for t in (a.k, a.v):
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run(resid[0], 4)
    length = 0
    for i, T in enumerate((4, 4, 1, 3, 2)):
        length += T
        x = torch.as_tensor(np.random.default_rng(i).standard_normal((4, a.H)).astype(np.float32))
        for s, r in zip((a, b), resid):
            r.copy_(x)
            s.set(T, length)
        graph.replay()
        b.run(resid[1], 4)
        torch.cuda.synchronize()
        for n in ("q", "o8", "os"):
            assert torch.equal(a.b[n][:T], b.b[n][:T]), n
        assert torch.equal(resid[0][:T], resid[1][:T])
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
