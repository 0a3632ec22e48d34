"""Paged caches and batches for the tests of moe_rope_append and
moe_paged_attention: built on the host, copied to the device."""

import numpy as np
import torch

from oracle import around

CODES = torch.float8_e4m3fn


class Setup:
    """A cache of random contents and the sequences `rows` = [(new tokens,
    cached length), ...] over pages in random order.  layout: "slots" ([page]
    [slot][head][D]), "heads" ([page][head][slot][D]) or "both" (keys and
    values of a page next to each other)."""

    def __init__(self, rows, Hkv, D, cache="bf16", page=16, layout="slots", seed=0, spare=2, max_pages=None,
                 first=0, behind=0):
        g = torch.Generator().manual_seed(seed)
        self.rows, self.Hkv, self.D, self.f8, self.page = rows, Hkv, D, cache == "f8", page
        per = [max(0, -(-length // page)) for _, length in rows]
        self.pages = sum(per) + spare
        self.max_pages = max_pages or max(max(per), 1)
        shape = (self.pages, page, Hkv, D)
        if self.f8:
            k, v = (torch.randint(0, 256, shape, generator=g, dtype=torch.uint8) for _ in "kv")
            for t in (k, v):
                t[(t & 127) == 127] = 0x38      # no NaN codes
            self.k_scale, self.v_scale = (torch.rand(shape[:3], generator=g) * 0.01 + 0.002 for _ in "kv")
            # (codes are spread over the exponents: about as large as normal numbers)
            self.k, self.v = k, v
        else:
            self.k, self.v = (torch.randn(shape, generator=g).bfloat16() for _ in "kv")
            self.k_scale = self.v_scale = None
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        table = torch.full((len(rows), self.max_pages), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(per):
            n = min(n, self.max_pages)
            table[b, :n] = order[at:at + n]
            at += n
        self.table = table
        off = [first]
        for new, _ in rows:
            off.append(off[-1] + new)
        self.off = off
        self.T = off[-1] + behind
        self.layout = layout
        self.kv_len = torch.tensor([length for _, length in rows], dtype=torch.int32)

    def device(self, device="cuda"):
        """(KVCache, KVBatch, dict of the device tensors)."""
        import routed_expert_ffn_gemv_amd as moe

        def put(t):
            if self.layout == "heads":
                return t.permute(0, 2, 1, 3).contiguous().to(device).permute(0, 2, 1, 3)
            return t.contiguous().to(device)
        if self.layout == "both":
            kv = torch.stack((self.k, self.v), dim=1).contiguous().to(device)
            k, v = kv[:, 0], kv[:, 1]
        else:
            k, v = put(self.k), put(self.v)
        d = {"k": k, "v": v, "k_scale": None, "v_scale": None}
        if self.f8:
            d["k_scale"], d["v_scale"] = self.k_scale.to(device), self.v_scale.to(device)
        d["q_off"] = torch.tensor(self.off, dtype=torch.int32, device=device)
        d["kv_len"] = self.kv_len.to(device)
        d["table"] = self.table.to(device)
        return (moe.KVCache(k, v, d["k_scale"], d["v_scale"]),
                moe.KVBatch(d["q_off"], d["kv_len"], d["table"]), d)

    def values(self, name):
        """Keys or values as 64-bit numbers, [pages][page][Hkv][D]."""
        t = getattr(self, name)
        if not self.f8:
            return t.double().numpy()
        return around.E4M3[t.numpy()] * getattr(self, name + "_scale").double().numpy()[..., None]

    def place(self, b, pos):
        """(page, slot) of a position, or None if it is not there."""
        if pos < 0 or pos >= self.max_pages * self.page:
            return None
        p = int(self.table[b, pos // self.page])
        return (p, pos % self.page) if 0 <= p < self.pages else None

    def sequence(self, b):
        """(keys, values [L][Hkv][D], seen [L]) of sequence b in 64 bits."""
        L = max(0, min(int(self.kv_len[b]), self.max_pages * self.page))
        k, v = np.zeros((L, self.Hkv, self.D)), np.zeros((L, self.Hkv, self.D))
        seen = np.zeros(L, bool)
        kk, vv = self.values("k"), self.values("v")
        for pos in range(L):
            where = self.place(b, pos)
            if where:
                k[pos], v[pos], seen[pos] = kk[where], vv[where], True
        return k, v, seen

    def positions(self, b):
        new = self.rows[b][0]
        return np.arange(int(self.kv_len[b]) - new, int(self.kv_len[b]))
