"""Timed cases of the operators that surround the routed-MoE layer.

Between two layers the layer's output joins the residual stream, which is
normalised into the next layer's tokens (moe_add_rmsnorm); after the last one
an 8-bit block-scaled product gives the logits, or another dense projection
(moe_scaled_linear); from the logits a token is drawn per row, for a decode batch
(moe_sample) or for a verify pass (moe_verify_sample).

``own`` False: the operators in elementary torch operations; True: the
library's calls.  Both take what ``prepare`` returns.
"""

import math

import torch

own = False

BLOCK = 128          # columns (and weight rows) that share a scale
E4M3_MAX = 448.0
SCALE_FLOOR = 448.0 * 2.0 ** -126   # smallest block maximum that sets a scale

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- the cases

def listed():
    """Hidden 2048, a vocabulary of 151,936 and steps of 1, 4, 16 and 32,768
    tokens are the model's; the others are generic."""
    return [
        # one decoded token between two layers: latency
        {"name": "norm_token", "op": "norm", "T": 1, "H": 2048, "y": "f32", "resid": "f32", "out": "bf16"},
        # a 16-token step in front of the output head
        {"name": "norm_step_f8", "op": "norm", "T": 16, "H": 2048, "y": "f32", "resid": "bf16", "out": "f8"},
        # a packed batch of odd length, rows that end inside a block of 128
        {"name": "norm_ragged", "op": "norm", "T": 1237, "H": 1000, "y": "bf16", "resid": "f32", "out": "both"},
        # a long prompt, for the router (bf16) and a dense projection (8 bits)
        {"name": "norm_prompt", "op": "norm", "T": 32768, "H": 2048, "y": "f32", "resid": "bf16", "out": "both"},
        # the output head for one token: the weights are read once
        {"name": "head_token", "op": "linear", "T": 1, "N": 151936, "K": 2048, "out": "f32"},
        # the output head for a 16-token step
        {"name": "head_step", "op": "linear", "T": 16, "N": 151936, "K": 2048, "out": "f32"},
        # a projection of an odd batch, every size ending inside a tile
        {"name": "proj_ragged", "op": "linear", "T": 777, "N": 1000, "K": 2000, "out": "f32"},
        # a projection of a long prompt: matrix-core rate
        {"name": "proj_prompt", "op": "linear", "T": 32768, "N": 4096, "K": 2048, "out": "bf16"},
        # one chat request
        {"name": "sample_token", "op": "sample", "T": 1, "V": 151936, "logits": "f32", "masked": 0.0, "verify": False},
        # a verify pass: one token and three drafts
        {"name": "sample_verify", "op": "sample", "T": 4, "V": 151936, "logits": "f32", "masked": 0.0, "verify": True},
        # a batch under a grammar that forbids most tokens, 16-bit logits
        {"name": "sample_masked", "op": "sample", "T": 64, "V": 32000, "logits": "bf16", "masked": 0.9, "verify": False},
        # a large decode batch of mixed requests
        {"name": "sample_batch", "op": "sample", "T": 256, "V": 151936, "logits": "f32", "masked": 0.0, "verify": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "linear", "sample"))
    if op == "norm":
        H = _log_int(rng, 64, 8192)
        if rng.random() < 0.7:
            H = max(64, H // 32 * 32)
        return {"op": op, "T": _log_int(rng, 1, max(1, min(32768, 32768 * 2048 // H))), "H": H,
                "y": rng.choice(("f32", "bf16", "none")), "resid": rng.choice(("f32", "bf16")),
                "out": rng.choice(("bf16", "f8", "both"))}
    if op == "linear":
        N, K = _log_int(rng, 64, 151936), _log_int(rng, 128, 8192) // 16 * 16
        if rng.random() < 0.5:
            K = max(128, K // 128 * 128)
        N = min(N, 151936 * 2048 // K)
        out = rng.choice(("f32", "bf16"))
        most = min(32768, 32768 * 4096 * 2048 // (N * K), 32768 * 4096 // N)
        return {"op": op, "T": _log_int(rng, 1, max(1, most)), "N": N, "K": K, "out": out}
    V = _log_int(rng, 1000, 151936)
    verify = rng.random() < 0.3
    T = rng.randint(1, 8) if verify else _log_int(rng, 1, 256)
    return {"op": op, "T": T, "V": V, "logits": rng.choice(("f32", "bf16")),
            "masked": rng.choice((0.0, 0.0, 0.5, 0.9)), "verify": verify}


def work(case):
    T = case["T"]
    size = {"f32": 4, "bf16": 2, "none": 0}
    if case["op"] == "norm":
        H = case["H"]
        y, r = size[case["y"]], size[case["resid"]]
        out = {"bf16": 2 * H, "f8": H + 4 * -(-H // BLOCK), "both": 3 * H + 4 * -(-H // BLOCK)}[case["out"]]
        # without y the residual stays as it is and is not written
        return {"bytes": T * (H * (y + r + (r if y else 0)) + out) + 2 * H, "flops": 6 * T * H}
    if case["op"] == "linear":
        N, K = case["N"], case["K"]
        scales = 4 * -(-K // BLOCK) * (T + -(-N // BLOCK))
        return {"bytes": (T + N) * K + scales + T * N * size[case["out"]], "flops": 2 * T * N * K}
    return {"bytes": T * (case["V"] * size[case["logits"]] + 32), "flops": 4 * T * case["V"]}


# ---------------------------------------------------------------- inputs

def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _quantise(v, rows):
    """v [R][K] fp32 -> e4m3 codes and one scale per `rows` x 128 block."""
    R, K = v.shape
    rb, kb = -(-R // rows), -(-K // BLOCK)
    pad = torch.nn.functional.pad(v, (0, kb * BLOCK - K, 0, rb * rows - R))
    amax = pad.view(rb, rows, kb, BLOCK).abs().amax(dim=(1, 3))
    scale = amax.clamp_min(SCALE_FLOOR) / E4M3_MAX
    full = scale.repeat_interleave(rows, 0)[:R].repeat_interleave(BLOCK, 1)[:, :K]
    return (v / full).to(torch.float8_e4m3fn), scale


def _logits(case, seed):
    """Logits whose probabilities fall off as a power of a token's rank, as a
    language model's do, from sharp rows to flat ones, with noise."""
    T, V = case["T"], case["V"]
    g = _gen(seed, 3)
    rank = torch.argsort(torch.rand((T, V), device="cuda", generator=g), dim=1)
    fall = 0.7 + 1.6 * torch.rand((T, 1), device="cuda", generator=g)
    x = -fall * torch.log1p(rank.float()) + 0.4 * torch.randn((T, V), device="cuda", generator=g)
    x += 20.0 * torch.rand((T, 1), device="cuda", generator=g)
    if case["masked"]:
        drop = torch.rand((T, V), device="cuda", generator=g) < case["masked"]
        drop[:, V // 2] = False
        x = x.masked_fill(drop, -math.inf)
    return x.to(DTYPES[case["logits"]])


def prepare(case, seed):
    T, dev = case["T"], "cuda"
    s = {"case": case}
    if case["op"] == "norm":
        H = case["H"]
        g = _gen(seed, 1)
        s["y"] = None if case["y"] == "none" else (
            torch.randn((T, H), device=dev, generator=g) * 0.7).to(DTYPES[case["y"]])
        s["resid"] = (torch.randn((T, H), device=dev, generator=g) * 3.0).to(DTYPES[case["resid"]])
        s["weight"] = (1.0 + 0.2 * torch.randn(H, device=dev, generator=g)).to(torch.bfloat16)
        s["resid_out"] = None if s["y"] is None else torch.empty_like(s["resid"])
        s["x"] = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if case["out"] != "f8" else None
        s["x8"] = s["x8_scale"] = None
        if case["out"] != "bf16":
            s["x8"] = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=dev)
            s["x8_scale"] = torch.empty((T, -(-H // BLOCK)), dtype=torch.float32, device=dev)
    elif case["op"] == "linear":
        N, K = case["N"], case["K"]
        g = _gen(seed, 2)
        s["x8"], s["x8_scale"] = _quantise(torch.randn((T, K), device=dev, generator=g), 1)
        s["w8"], s["w8_scale"] = _quantise(torch.randn((N, K), device=dev, generator=g) * 0.02, BLOCK)
        s["out"] = torch.empty((T, N), dtype=DTYPES[case["out"]], device=dev)
        s["ws"] = None
        if own:
            import routed_expert_ffn_gemv_amd as moe
            n = moe.moe_scaled_linear_workspace_size(T, N, K)
            s["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
    else:
        V = case["V"]
        g = _gen(seed, 4)
        s["logits"] = _logits(case, seed)
        row = torch.arange(T, device=dev)

        def uniform():
            return torch.rand(T, device=dev, generator=g)

        # every fourth request or so leaves one of the filters off; an eighth is greedy
        s["temperature"] = torch.where(row % 8 == 5, torch.zeros_like(uniform()), 0.5 + 0.8 * uniform())
        s["top_k"] = torch.where(uniform() < 0.4, torch.zeros_like(row), (uniform() * 200).long() + 1).to(torch.int32)
        s["top_p"] = torch.where(uniform() < 0.25, torch.ones(T, device=dev), 0.7 + 0.29 * uniform())
        s["min_p"] = torch.where(uniform() < 0.5, torch.zeros(T, device=dev), 0.1 * uniform())
        s["u"] = uniform()
        s["tokens"] = torch.empty(T, dtype=torch.int32, device=dev)
        s["prob"] = torch.empty(T, dtype=torch.float32, device=dev)
        if case["verify"]:
            # drafts that the model often agrees with: its most likely tokens
            s["draft"] = s["logits"].float().argmax(dim=1).to(torch.int32)[: T - 1].contiguous()
            s["n_out"] = torch.empty(1, dtype=torch.int32, device=dev)
        if own:
            import routed_expert_ffn_gemv_amd as moe
            s["ws"] = torch.empty(moe.moe_sample_workspace_size(T, V), dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        import routed_expert_ffn_gemv_amd as moe
        return {"norm": _own_norm, "linear": _own_linear, "sample": _own_sample}[op](moe, state)
    return {"norm": _plain_norm, "linear": _plain_linear, "sample": _plain_sample}[op](state)


def _own_norm(moe, s):
    c = s["case"]
    moe.moe_add_rmsnorm(c["T"], c["H"], s["y"], s["resid"], s["weight"], 1e-6, resid_out=s["resid_out"],
                        x=s["x"], x8=s["x8"], x8_scale=s["x8_scale"])
    return {"resid": s["resid_out"], "x": s["x"], "x8": s["x8"], "x8_scale": s["x8_scale"]}


def _own_linear(moe, s):
    c = s["case"]
    moe.moe_scaled_linear(s["x8"], s["x8_scale"], c["T"], s["w8"], s["w8_scale"], c["N"], c["K"], s["out"], s["ws"])
    return s["out"]


def _own_sample(moe, s):
    c = s["case"]
    params = {"temperature": s["temperature"], "top_k": s["top_k"], "top_p": s["top_p"], "min_p": s["min_p"]}
    if c["verify"]:
        moe.moe_verify_sample(s["logits"], c["T"], c["V"], s["draft"], s["u"], s["tokens"], s["n_out"], s["ws"],
                              prob=s["prob"], **params)
        return {"tokens": s["tokens"], "n_out": s["n_out"], "prob": s["prob"]}
    moe.moe_sample(s["logits"], c["T"], c["V"], s["u"], s["tokens"], s["ws"], prob=s["prob"], **params)
    return {"tokens": s["tokens"], "prob": s["prob"]}


def _plain_norm(s):
    v = s["resid"].float()
    if s["y"] is not None:
        v = (v + s["y"].float()).to(s["resid"].dtype)
    kept, v = v, v.float()
    # a normalised value next to a border between two 8-bit codes: the mean square is taken in 64 bits
    inv = torch.rsqrt(v.double().square().mean(dim=1, keepdim=True) + 1e-6).float()
    n = v * inv * s["weight"].float()
    x8 = scale = None
    if s["x8"] is not None:
        T, H = n.shape
        kb = -(-H // BLOCK)
        blocks = torch.nn.functional.pad(n, (0, kb * BLOCK - H)).view(T, kb, BLOCK)
        scale = blocks.abs().amax(dim=2).clamp_min(SCALE_FLOOR) / E4M3_MAX
        x8 = (blocks / scale[:, :, None]).view(T, kb * BLOCK)[:, :H].contiguous().to(torch.float8_e4m3fn)
    return {"resid": kept if s["y"] is not None else None,
            "x": n.to(torch.bfloat16) if s["x"] is not None else None, "x8": x8, "x8_scale": scale}


def _plain_linear(s):
    T, K = s["x8"].shape
    N = s["w8"].shape[0]
    a = s["x8"].float() * s["x8_scale"].repeat_interleave(BLOCK, 1)[:, :K]
    b = s["w8"].float() * s["w8_scale"].repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return (a @ b.t()).to(s["out"].dtype)


def _plain_sample(s):
    # 64 bits: a draw may fall next to the border between two tokens
    x = s["logits"].double()
    T, V = x.shape
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    greedy = (s["temperature"] <= 0)[:, None]
    tau = torch.where(greedy, torch.ones_like(x[:, :1]), s["temperature"].double()[:, None])
    w = torch.exp((x - x[:, :1]) / tau)
    rank = torch.arange(V, device=x.device)[None, :]
    w = w * (w >= s["min_p"].double()[:, None])
    k = s["top_k"].long()[:, None]
    w = w * ((rank < k) | (k <= 0))
    w = w * ((rank == 0) | ~greedy)
    cum = torch.cumsum(w, dim=1)
    p = s["top_p"].double()[:, None]
    # token r stays while the tokens before it hold less than p
    stays = (cum - w < p * cum[:, -1:]) | (p >= 1)
    w = w * (stays | (rank == 0))
    cum = torch.cumsum(w, dim=1)
    at = (cum <= s["u"].double()[:, None] * cum[:, -1:]).sum(dim=1, keepdim=True)
    at = torch.minimum(at, (w > 0).sum(dim=1, keepdim=True) - 1)
    tokens = order.gather(1, at)[:, 0].to(torch.int32)
    prob = (w.gather(1, at) / cum[:, -1:])[:, 0].float()
    if not s["case"]["verify"]:
        return {"tokens": tokens, "prob": prob}
    agree = (tokens[: T - 1] == s["draft"]).to(torch.int32)
    n_out = (torch.cumprod(agree, dim=0).sum() + 1).to(torch.int32).view(1)
    return {"tokens": tokens, "n_out": n_out, "prob": prob}


# ---------------------------------------------------------------- in 64 bits

def _e4m3(v):
    """v (64 bits) to the nearest e4m3 value, ties to an even code."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), e.clamp_min(-5) - 4)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        r = s["resid"].to(torch.float64)
        if s["y"] is not None:
            r = (r + s["y"].to(torch.float64)).to(s["resid"].dtype).to(torch.float64)
        H = r.shape[1]
        rms = torch.sqrt((r * r).sum(dim=1) / H + 1e-6)
        n = r / rms[:, None] * s["weight"].to(torch.float64)
        codes = scales = None
        if s["x8"] is not None:
            codes, scales = torch.empty_like(n), []
            for b in range(0, H, BLOCK):
                part = n[:, b:b + BLOCK]
                scale = torch.clamp(part.abs().max(dim=1).values, min=SCALE_FLOOR) / E4M3_MAX
                codes[:, b:b + BLOCK] = _e4m3(part / scale[:, None])
                scales.append(scale)
            scales = torch.stack(scales, dim=1)
        return {"resid": r if s["y"] is not None else None, "x": n if s["x"] is not None else None,
                "x8": codes, "x8_scale": scales}
    if case["op"] == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        out = torch.zeros((T, N), dtype=torch.float64, device="cuda")
        wrow = torch.arange(N, device="cuda") // BLOCK
        for b in range(0, K, BLOCK):
            a = s["x8"][:, b:b + BLOCK].to(torch.float64) * s["x8_scale"][:, b // BLOCK, None].double()
            w = s["w8"][:, b:b + BLOCK].to(torch.float64) * s["w8_scale"][wrow, b // BLOCK].double()[:, None]
            out += torch.mm(a, w.t().contiguous())
        return out
    tokens, probs = [], []
    for t in range(case["T"]):
        x = s["logits"][t].to(torch.float64)
        tau, u = float(s["temperature"][t]), float(s["u"][t])
        top_k, top_p, min_p = int(s["top_k"][t]), float(s["top_p"][t]), float(s["min_p"][t])
        if tau <= 0:
            tokens.append(int((x == x.max()).nonzero()[0, 0]))
            probs.append(1.0)
            continue
        w = torch.exp(x / tau - x.max() / tau)
        ids = torch.nonzero(w >= max(min_p, 1e-300))[:, 0]
        ids = ids[torch.argsort(-x[ids], stable=True)]
        ids = ids[:top_k] if top_k > 0 else ids
        part = w[ids]
        if top_p < 1:
            n = int((torch.cumsum(part, 0) < top_p * part.sum()).sum()) + 1
            ids, part = ids[:n], part[:n]
        share = part / part.sum()
        at = min(int((torch.cumsum(share, 0) <= u).sum()), len(ids) - 1)
        tokens.append(int(ids[at]))
        probs.append(float(share[at]))
    out = {"tokens": torch.tensor(tokens), "prob": torch.tensor(probs, dtype=torch.float64)}
    if case["verify"]:
        drafts = s["draft"].tolist()
        kept = 0
        while kept < len(drafts) and drafts[kept] == tokens[kept]:
            kept += 1
        out["n_out"] = torch.tensor([kept + 1])
    return out
