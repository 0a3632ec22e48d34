"""Timed cases of the attention half of a decoder layer over a paged cache.

A dense projection gives each new token's query, key and value heads;
moe_rope_append normalises and rotates queries and keys and appends keys and
values to the pages of the token's sequence; moe_paged_attention attends from
the new tokens of every sequence to its pages.

``own`` False: the operators in elementary torch operations; True: the
library's calls.  Both take what ``prepare`` returns.
"""

import math
import random

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
SCALE_FLOOR = 448.0 * 2.0 ** -126   # smallest row (or block) maximum that sets a scale
BLOCK = 128                         # output columns that share an 8-bit scale

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- the cases
#
# Lengths: "seqs" sequences; "new" is the number of new tokens of each, "len"
# the longest cached length (new tokens included).  "spread" texts: "same": all
# alike; "ragged": lengths (and counts of more than one) spread below these;
# "mixed": one sequence brings the chunk, the others one token each.

def listed():
    """Steps of 1, 4 (one token and three drafts), 16 and 32,768 tokens are
    the model's; head counts, pages and lengths are generic."""
    return [
        # one decoded token: latency
        {"name": "append_token", "op": "append", "seqs": 1, "new": 1, "len": 1000, "spread": "same", "Hq": 16,
         "Hkv": 2, "D": 256, "R": 64, "pairs": "half", "norm": True, "x": "bf16", "cache": "bf16", "page": 16},
        # a decode step of 64 requests into an 8-bit cache
        {"name": "append_step_f8", "op": "append", "seqs": 64, "new": 1, "len": 4000, "spread": "ragged", "Hq": 16,
         "Hkv": 2, "D": 256, "R": 64, "pairs": "half", "norm": True, "x": "bf16", "cache": "f8", "page": 32},
        # chunks of odd lengths, odd head counts, interleaved pairs, part of the head, fp32 rows
        {"name": "append_ragged", "op": "append", "seqs": 7, "new": 401, "len": 1500, "spread": "ragged", "Hq": 9,
         "Hkv": 3, "D": 64, "R": 50, "pairs": "neighbours", "norm": False, "x": "f32", "cache": "bf16", "page": 16},
        # a long prompt
        {"name": "append_prompt", "op": "append", "seqs": 1, "new": 32768, "len": 32768, "spread": "same", "Hq": 16,
         "Hkv": 2, "D": 256, "R": 64, "pairs": "half", "norm": True, "x": "bf16", "cache": "bf16", "page": 64},
        # one chat request, one token
        {"name": "attend_token", "op": "attend", "seqs": 1, "new": 1, "len": 4097, "spread": "same", "Hq": 16,
         "Hkv": 2, "D": 256, "cache": "bf16", "page": 16, "window": 0, "out": "bf16"},
        # a verify pass of one token and three drafts at the end of a long text
        {"name": "attend_verify", "op": "attend", "seqs": 1, "new": 4, "len": 32768, "spread": "same", "Hq": 16,
         "Hkv": 2, "D": 256, "cache": "bf16", "page": 64, "window": 0, "out": "f8"},
        # a decode batch of mixed requests
        {"name": "attend_batch", "op": "attend", "seqs": 64, "new": 1, "len": 16384, "spread": "ragged", "Hq": 16,
         "Hkv": 2, "D": 256, "cache": "bf16", "page": 32, "window": 0, "out": "bf16"},
        # a large decode batch on an 8-bit cache
        {"name": "attend_batch_f8", "op": "attend", "seqs": 256, "new": 1, "len": 5000, "spread": "ragged", "Hq": 32,
         "Hkv": 4, "D": 128, "cache": "f8", "page": 16, "window": 0, "out": "f8"},
        # a step that decodes for most requests and reads a chunk of one prompt; odd head group
        {"name": "attend_mixed", "op": "attend", "seqs": 17, "new": 509, "len": 7001, "spread": "mixed", "Hq": 15,
         "Hkv": 5, "D": 64, "cache": "bf16", "page": 16, "window": 0, "out": "bf16"},
        # chunks under a sliding window
        {"name": "attend_window", "op": "attend", "seqs": 4, "new": 1000, "len": 20000, "spread": "ragged", "Hq": 20,
         "Hkv": 4, "D": 128, "cache": "bf16", "page": 32, "window": 1024, "out": "bf16"},
        # a prompt from its start
        {"name": "attend_prompt", "op": "attend", "seqs": 1, "new": 16384, "len": 16384, "spread": "same", "Hq": 16,
         "Hkv": 2, "D": 256, "cache": "bf16", "page": 64, "window": 0, "out": "bf16"},
        # a chunk of 4096 tokens late in a long text, 8-bit cache
        {"name": "attend_long_f8", "op": "attend", "seqs": 1, "new": 4096, "len": 65536, "spread": "same", "Hq": 32,
         "Hkv": 4, "D": 128, "cache": "f8", "page": 64, "window": 0, "out": "f8"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(("append", "attend", "attend"))
        D = rng.choice((64, 128, 256))
        Hkv = rng.randint(1, 8)
        c = {"op": op, "seqs": _log_int(rng, 1, 256), "new": 1, "len": 1, "spread": rng.choice(("same", "ragged")),
             "Hq": Hkv * _log_int(rng, 1, 16), "Hkv": Hkv, "D": D, "cache": rng.choice(("bf16", "f8")),
             "page": rng.choice((16, 32, 64, 128))}
        kind = rng.choice(("decode", "verify", "chunk", "mixed"))
        if kind == "verify":
            c["new"] = rng.randint(2, 16)
        elif kind != "decode":
            c["new"] = _log_int(rng, 17, 16384)
        if kind == "mixed":
            c["spread"] = "mixed"
        c["len"] = max(c["new"], _log_int(rng, 1, 65536))
        if op == "append":
            c["R"] = rng.choice((D, D // 2, D // 4, 2 * rng.randint(1, D // 2)))
            c["pairs"] = rng.choice(("half", "neighbours"))
            c["norm"], c["x"] = rng.random() < 0.6, rng.choice(("bf16", "f32"))
        else:
            c["window"] = rng.choice((0, 0, _log_int(rng, 16, 8192)))
            c["out"] = rng.choice(("bf16", "f8" if D >= BLOCK else "bf16"))
        w = work(c)
        tokens, cached = sum(_news(c)), sum(_pages(c)) * c["page"]
        held = cached * Hkv * D * 4
        if tokens <= 65536 and held <= 8e9 and w["bytes"] <= 9.3e8 and w["flops"] <= 4.2e12:
            return c


def _spread(case):
    """(new tokens, cached length) of every sequence, from the case alone."""
    rng = random.Random(case["seqs"] * 1000003 + case["new"] * 1009 + case["len"])
    rows = []
    for b in range(case["seqs"]):
        new, length = case["new"], case["len"]
        if case["spread"] == "mixed" and b != case["seqs"] // 2:
            new = 1
        if case["spread"] == "ragged" and b != case["seqs"] // 2:
            new = new if new == 1 else rng.randint(max(1, new // 4), new)
        if case["spread"] != "same" and b != case["seqs"] // 2:
            length = max(new, int(length * rng.random() ** 1.5))
        rows.append((new, length))
    return rows


def _news(case):
    return [new for new, _ in _spread(case)]


def _pages(case):
    return [-(-length // case["page"]) for _, length in _spread(case)]


def work(case):
    rows, D, Hq, Hkv = _spread(case), case["D"], case["Hq"], case["Hkv"]
    T = sum(new for new, _ in rows)
    kv = Hkv * (D * 2 if case["cache"] == "bf16" else D + 4)      # bytes of a position's keys (or values)
    if case["op"] == "append":
        read = (Hq + 2 * Hkv) * D * (2 if case["x"] == "bf16" else 4)
        return {"bytes": T * (read + Hq * D * 2 + 2 * kv), "flops": T * (Hq + Hkv) * (4 * D + 3 * case["R"])}
    span = case["window"] or 1 << 60
    seen = pairs = 0
    for new, length in rows:
        seen += min(length, span + new - 1)
        first = length - new + 1                                   # positions that the first new token attends
        full = max(0, min(new, length - span))                     # the last ones see a whole window
        ramp = new - full
        pairs += full * span + ramp * first + ramp * (ramp - 1) // 2
    out = {"bf16": 2 * D, "f8": D + 4 * D // BLOCK}[case["out"]]
    return {"bytes": seen * 2 * kv + T * Hq * (2 * D + out), "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------- inputs

def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _row_codes(v):
    """v [..., D] fp32 -> e4m3 codes and one scale per row."""
    scale = v.abs().amax(dim=-1).clamp_min(SCALE_FLOOR) / E4M3_MAX
    return (v / scale[..., None]).to(torch.float8_e4m3fn), scale


def _cache(case, seed, pages):
    """Keys and values of every page (a kept cache holds something in each)."""
    shape = (pages, case["page"], case["Hkv"], case["D"])
    g = _gen(seed, 1)
    s = {}
    for name in ("k", "v"):
        if case["cache"] == "bf16":
            s[name] = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        else:
            s[name] = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
            s[name + "_scale"] = torch.empty(shape[:3], device="cuda")
            for p in range(0, pages, 4096):
                part = torch.randn((min(4096, pages - p), *shape[1:]), device="cuda", generator=g)
                s[name][p:p + 4096], s[name + "_scale"][p:p + 4096] = _row_codes(part)
    return s


def prepare(case, seed):
    dev = "cuda"
    rows, D, Hq, Hkv = _spread(case), case["D"], case["Hq"], case["Hkv"]
    T, per = sum(new for new, _ in rows), _pages(case)
    pages = sum(per) + 3
    s = {"case": case, "T": T, "rows": rows}
    s.update(_cache(case, seed, pages))
    g = _gen(seed, 2)
    # pages were handed out as requests came and went: any order
    order = torch.randperm(pages, device=dev, generator=g).to(torch.int32)
    table = torch.full((len(rows), max(per)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    q_off = [0]
    for new, _ in rows:
        q_off.append(q_off[-1] + new)
    s["page_table"] = table
    s["q_off"] = torch.tensor(q_off, dtype=torch.int32, device=dev)
    s["kv_len"] = torch.tensor([length for _, length in rows], dtype=torch.int32, device=dev)
    if case["op"] == "append":
        R = case["R"]
        s["qkv"] = torch.randn((T, (Hq + 2 * Hkv) * D), device=dev, generator=g).to(DTYPES[case["x"]])
        # a large base, and frequencies divided as for a context four times as long
        s["freq"] = torch.tensor([1e6 ** (-2.0 * j / R) / 4.0 for j in range(R // 2)], dtype=torch.float64, device=dev)
        s["rot_scale"] = 0.1 * math.log(4.0) + 1.0
        for name in ("q_weight", "k_weight"):
            s[name] = None
            if case["norm"]:
                s[name] = (1.0 + 0.2 * torch.randn(D, device=dev, generator=g)).to(torch.bfloat16)
        s["q"] = torch.empty((T, Hq * D), dtype=torch.bfloat16, device=dev)
    else:
        # from heads that spread their weight to heads that look at few positions
        sharp = 0.5 + 2.5 * torch.rand(Hq, device=dev, generator=g)
        q = torch.randn((T, Hq, D), device=dev, generator=g) * sharp[:, None]
        s["q"] = q.to(torch.bfloat16).view(T, Hq * D)
        s["out"] = s["x8"] = s["x8_scale"] = None
        if case["out"] == "f8":
            s["x8"] = torch.empty((T, Hq * D), dtype=torch.float8_e4m3fn, device=dev)
            s["x8_scale"] = torch.empty((T, Hq * D // BLOCK), device=dev)
        else:
            s["out"] = torch.empty((T, Hq * D), dtype=torch.bfloat16, device=dev)
    if own:
        import routed_expert_ffn_gemv_amd as moe
        s["cache"] = moe.KVCache(s["k"], s["v"], s.get("k_scale"), s.get("v_scale"))
        s["batch"] = moe.KVBatch(s["q_off"], s["kv_len"], s["page_table"])
        if case["op"] == "attend":
            n = moe.moe_paged_attention_workspace_size(T, len(rows), Hq, Hkv, D)
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    append = state["case"]["op"] == "append"
    if own:
        import routed_expert_ffn_gemv_amd as moe
        return _own_append(moe, state) if append else _own_attend(moe, state)
    return _plain_append(state) if append else _plain_attend(state)


def _updated(s):
    return {n: s[n] for n in ("q", "k", "v", "k_scale", "v_scale") if n in s}


def _own_append(moe, s):
    c = s["case"]
    moe.moe_rope_append(s["cache"], s["batch"], s["qkv"], s["T"], c["Hq"], s["q"], freq=s["freq"],
                        rot_scale=s["rot_scale"], interleaved=c["pairs"] == "neighbours", q_weight=s["q_weight"],
                        k_weight=s["k_weight"], eps=EPS)
    return _updated(s)


def _own_attend(moe, s):
    c = s["case"]
    moe.moe_paged_attention(s["cache"], s["batch"], s["q"], s["T"], c["Hq"], c["D"] ** -0.5, s["ws"], out=s["out"],
                            x8=s["x8"], x8_scale=s["x8_scale"], window=c["window"])
    return {"out": s["out"], "x8": s["x8"], "x8_scale": s["x8_scale"]}


def _plain_append(s):
    c = s["case"]
    T, D, R, Hq, Hkv = s["T"], c["D"], c["R"], c["Hq"], c["Hkv"]
    t = torch.arange(T, device="cuda")
    off, length = s["q_off"].long(), s["kv_len"].long()
    b = torch.searchsorted(off[1:], t, right=True)
    pos = length[b] - off[b + 1] + t
    # far positions: the angle in 64 bits
    angle = pos.double()[:, None] * s["freq"]
    cos, sin = [(f(angle) * s["rot_scale"]).float()[:, None, :] for f in (torch.cos, torch.sin)]
    x = s["qkv"].float().view(T, Hq + 2 * Hkv, D)
    done = []
    for part, weight in ((x[:, :Hq], s["q_weight"]), (x[:, Hq:Hq + Hkv], s["k_weight"])):
        if weight is not None:
            part = part * torch.rsqrt(part.square().mean(dim=2, keepdim=True) + EPS) * weight.float()
        if c["pairs"] == "half":
            lo, hi = part[..., :R // 2], part[..., R // 2:R]
            turned = torch.cat((lo * cos - hi * sin, hi * cos + lo * sin), dim=2)
        else:
            lo, hi = part[..., 0:R:2], part[..., 1:R:2]
            turned = torch.stack((lo * cos - hi * sin, hi * cos + lo * sin), dim=3).flatten(2)
        done.append(torch.cat((turned, part[..., R:]), dim=2))
    s["q"].copy_(done[0].reshape(T, Hq * D))
    page, slot = s["page_table"][b, pos // c["page"]].long(), pos % c["page"]
    for name, rows in (("k", done[1]), ("v", x[:, Hq + Hkv:])):
        if c["cache"] == "bf16":
            s[name][page, slot] = rows.to(torch.bfloat16)
        else:
            # (indexed as bytes: 8-bit floats cannot be stored by index)
            codes, s[name + "_scale"][page, slot] = _row_codes(rows)
            s[name].view(torch.uint8)[page, slot] = codes.view(torch.uint8)
    return _updated(s)


def _plain_attend(s):
    c = s["case"]
    D, Hq, Hkv, ps = c["D"], c["Hq"], c["Hkv"], c["page"]
    G = Hq // Hkv
    out = torch.empty((s["T"], Hq, D), device="cuda")
    t0 = 0
    for b, (new, length) in enumerate(s["rows"]):
        first = max(0, length - new - c["window"] + 1) if c["window"] else 0
        p0 = first // ps
        pages = s["page_table"][b, p0:-(-length // ps)].long()
        kv = []
        for name in ("k", "v"):
            x = s[name].view(torch.uint8 if c["cache"] == "f8" else torch.bfloat16)[pages].view(s[name].dtype).float()
            if c["cache"] == "f8":
                x = x * s[name + "_scale"][pages][..., None]
            kv.append(x.view(-1, Hkv, D)[:length - p0 * ps].transpose(0, 1).contiguous())
        k, v = kv
        pos = p0 * ps + torch.arange(k.shape[1], device="cuda")
        step = max(1, (1 << 30) // (Hq * k.shape[1]))              # 4 GiB of scores at a time
        for i in range(0, new, step):
            n = min(step, new - i)
            at = length - new + i + torch.arange(n, device="cuda")
            q = s["q"][t0 + i:t0 + i + n].float().view(n, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * n, D)
            x = torch.matmul(q, k.transpose(1, 2)).view(Hkv, G, n, -1) * D ** -0.5
            hidden = pos[None, :] > at[:, None]
            if c["window"]:
                hidden |= pos[None, :] <= at[:, None] - c["window"]
            x = x.masked_fill_(hidden, -math.inf)
            x = torch.exp(x.sub_(x.amax(dim=3, keepdim=True)))
            o = torch.matmul(x.view(Hkv, G * n, -1), v).view(Hkv, G, n, D) / x.sum(dim=3, keepdim=True)
            out[t0 + i:t0 + i + n] = o.permute(2, 0, 1, 3).reshape(n, Hq, D)
        t0 += new
    out = out.view(s["T"], Hq * D)
    if c["out"] != "f8":
        return {"out": out.to(torch.bfloat16), "x8": None, "x8_scale": None}
    x8, scale = _row_codes(out.view(s["T"], Hq * D // BLOCK, BLOCK))
    return {"out": None, "x8": x8.view(s["T"], Hq * D), "x8_scale": scale}


# ---------------------------------------------------------------- in 64 bits

def _e4m3(v):
    """v (64 bits) to the nearest e4m3 value, ties to an even code."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), e.clamp_min(-5) - 4)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _in_8_bits(v):
    scale = torch.clamp(v.abs().max(dim=-1).values, min=SCALE_FLOOR) / E4M3_MAX
    return _e4m3(v / scale.unsqueeze(-1)), scale


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_append if case["op"] == "append" else _exact_attend)(case, s)


def _exact_append(case, s):
    D, R, Hq, Hkv = case["D"], case["R"], case["Hq"], case["Hkv"]
    half = R // 2
    first, second = ((list(range(half)), list(range(half, R))) if case["pairs"] == "half" else
                     (list(range(0, R, 2)), list(range(1, R, 2))))
    out = {n: s[n].to(torch.float64) for n in ("k", "v")}
    out.update({n: s[n].to(torch.float64) for n in ("k_scale", "v_scale") if n in s})
    x = s["qkv"].to(torch.float64)
    q = torch.empty((s["T"], Hq * D), dtype=torch.float64, device="cuda")
    freq = s["freq"]
    t0 = 0
    for b, (new, length) in enumerate(s["rows"]):
        at = torch.arange(length - new, length, device="cuda")
        z = torch.polar(torch.full((new, half), s["rot_scale"], dtype=torch.float64, device="cuda"),
                        at.to(torch.float64)[:, None] * freq[None, :])
        page, slot = s["page_table"][b][at // case["page"]].long(), at % case["page"]
        for h in range(Hq + 2 * Hkv):
            r = x[t0:t0 + new, h * D:(h + 1) * D].clone()
            if h < Hq + Hkv:
                w = s["q_weight"] if h < Hq else s["k_weight"]
                if w is not None:
                    r = r / torch.sqrt((r * r).sum(dim=1, keepdim=True) / D + EPS) * w.to(torch.float64)
                turned = torch.complex(r[:, first], r[:, second]) * z
                r[:, first], r[:, second] = turned.real, turned.imag
            if h < Hq:
                q[t0:t0 + new, h * D:(h + 1) * D] = r
                continue
            name, head = ("k", h - Hq) if h < Hq + Hkv else ("v", h - Hq - Hkv)
            if case["cache"] == "f8":
                r, scale = _in_8_bits(r)
                out[name + "_scale"][page, slot, head] = scale
            out[name][page, slot, head] = r
        t0 += new
    return {"q": q, **out}


def _exact_attend(case, s):
    D, Hq, Hkv, ps = case["D"], case["Hq"], case["Hkv"], case["page"]
    out = torch.zeros((s["T"], Hq * D), dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (new, length) in enumerate(s["rows"]):
        where = torch.arange(length, device="cuda")
        page, slot = s["page_table"][b][where // ps].long(), where % ps
        for head in range(Hkv):
            rows = []
            for name in ("k", "v"):
                x = s[name].view(torch.uint8)[page, slot, head].view(s[name].dtype).to(torch.float64)
                if case["cache"] == "f8":
                    x = x * s[name + "_scale"][page, slot, head].to(torch.float64)[:, None]
                rows.append(x)
            k, v = rows
            kt = k.t().contiguous()
            for h in range(head * (Hq // Hkv), (head + 1) * (Hq // Hkv)):
                for i in range(0, new, 4096):
                    n = min(4096, new - i)
                    at = torch.arange(length - new + i, length - new + i + n, device="cuda")
                    score = torch.mm(s["q"][t0 + i:t0 + i + n, h * D:(h + 1) * D].to(torch.float64), kt) / math.sqrt(D)
                    seen = where[None, :] <= at[:, None]
                    if case["window"]:
                        seen &= where[None, :] > at[:, None] - case["window"]
                    score = torch.where(seen, score, torch.full_like(score, -math.inf))
                    out[t0 + i:t0 + i + n, h * D:(h + 1) * D] = torch.mm(torch.softmax(score, dim=1), v)
        t0 += new
    if case["out"] != "f8":
        return {"out": out, "x8": None, "x8_scale": None}
    x8, scale = _in_8_bits(out.view(s["T"], Hq * D // BLOCK, BLOCK))
    return {"out": None, "x8": x8.view(s["T"], Hq * D), "x8_scale": scale}
